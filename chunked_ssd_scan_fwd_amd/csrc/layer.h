// Declarations shared by the kernels of a linear-attention layer (layer_*.hip)
// and their host-side checks (layer_validate.cpp).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ssd.h"

namespace layer {

constexpr int64_t kMaxHeadDim = 256;
constexpr int64_t kMaxCount = int64_t(1) << 24;   // sequences, slots, entries, row strides

// Blocks of `threads` threads that one launch may have: a grid's threads are
// counted in 32 bits.
constexpr int64_t max_blocks(int threads) { return ((int64_t(1) << 32) - 1) / threads; }

int check_dtype(int dtype);
int check_lin(const lin_shape *s, bool step);
// The strides to use (dense ones where `st` is null) for `rows` rows, or
// SSD_ERR_SHAPE where they are out of range or let values of y overlap.
int resolve_strides(const lin_shape *s, const lin_strides *st, lin_strides *out, int64_t rows);
int check_gn(const gn_shape *s, int act);
int check_cache(const state_cache_shape *s);
inline bool misaligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
inline unsigned dtype_size(int dtype) { return dtype == LAYER_F32 ? 4u : 2u; }

}  // namespace layer
