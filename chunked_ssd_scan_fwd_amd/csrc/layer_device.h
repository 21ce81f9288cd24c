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

typedef float f32x4 __attribute__((ext_vector_type(4)));

// A piece of a state.  STREAM: non-temporal, past the caches.
template <int N, bool STREAM>
__device__ __forceinline__ Vec<float, N> load_state(const float *p)
{
    if constexpr (STREAM && N == 4)
        return __builtin_bit_cast(Vec<float, 4>, __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p)));
    else
        return *reinterpret_cast<const Vec<float, N> *>(p);
}
template <int N, bool STREAM>
__device__ __forceinline__ void store_state(float *p, const Vec<float, N> &x)
{
    if constexpr (STREAM && N == 4)
        __builtin_nontemporal_store(__builtin_bit_cast(f32x4, x), reinterpret_cast<f32x4 *>(p));
    else
        *reinterpret_cast<Vec<float, N> *>(p) = x;
}

// Looks for other rows of row n's slot: whether an earlier one has it, and
// the next later one (N if none).  All rows are looked at by every wave, 256
// at a time, which is one load's latency.
__device__ __forceinline__ void same_slot(const int32_t *slots, int N, int n, int sl, bool &before, int &next)
{
    const int lane = threadIdx.x & 63;
    before = false;
    next = N;
    for (int j0 = 0; j0 < N; j0 += 256) {
        bool same[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + 64 * u + lane;
            same[u] = j < N && slots[j < N ? j : 0] == sl;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + 64 * u + lane;
            before = before || __ballot(same[u] && j < n) != 0;
            const unsigned long long later = __ballot(same[u] && j > n);
            if (later != 0 && next == N) next = j0 + 64 * u + __ffsll(later) - 1;
        }
    }
}

inline int launch_status() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_DEVICE; }

// Runs BODY with T the element type that `dtype` names.
#define LAYER_DISPATCH(DTYPE, ...)                                 \
    do {                                                           \
        if ((DTYPE) == LAYER_BF16) { using T = layer::bf16; __VA_ARGS__; } \
        else if ((DTYPE) == LAYER_F16) { using T = layer::f16; __VA_ARGS__; } \
        else { using T = float; __VA_ARGS__; }                            \
    } while (0)

}  // namespace layer
