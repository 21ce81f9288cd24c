// Device-side helpers of the linear-attention layer's kernels: element types
// and checks of the callers' index arrays.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "layer.h"

namespace layer {

typedef __bf16 bf16;
typedef _Float16 f16;

// Both conversions round to nearest, ties to even (v_cvt_pk_bf16_f32, v_cvt_f16_f32).
template <typename T>
__device__ __forceinline__ float to_f(T x) { return (float)x; }
template <typename T>
__device__ __forceinline__ T from_f(float x) { return (T)x; }

// N elements that follow one another, loaded or stored at once.
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

// A log decay of -inf (the state is forgotten) as a finite number, so that
// differences of sums of log decays stay finite: e^-10000 is 0 in float32,
// also beside any growth that does not overflow by itself.
__device__ __forceinline__ float clamp_decay(float la) { return la < -1e4f ? -1e4f : la; }

// The index of pair i: ids[i], or i where there is no array.
__device__ __forceinline__ int index_of(const int32_t *ids, int i) { return ids ? ids[i] : i; }

inline int launch_status() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_DEVICE; }

// Runs BODY with T the element type that `dtype` names.
#define LAYER_DISPATCH(DTYPE, ...)                                 \
    do {                                                           \
        if ((DTYPE) == LAYER_BF16) { using T = layer::bf16; __VA_ARGS__; } \
        else if ((DTYPE) == LAYER_F16) { using T = layer::f16; __VA_ARGS__; } \
        else { using T = float; __VA_ARGS__; }                            \
    } while (0)

}  // namespace layer
