// States to a cache in 8 bits and back.  A block of 32 values x of a state's
// row becomes e4m3 numbers of x 2^-s, with s the least exponent for which the
// block's largest magnitude stays within 448 2^s.  The scale is a power of
// two, so the only rounding is that to e4m3.
//
// One pass: 5 bytes and 1/32 move for each value, which bounds both kernels.
#include "layer_device.h"

namespace layer {

constexpr int CT = 256;

struct CacheArgs {
    const int32_t *src, *dst;   // slots and entries, or the other way round
    int n, nsrc, ndst, dk, dv, nb;
    int64_t rows;               // H * dk
    int64_t per;                // blocks of a state: H * dk * nb
    int chunks;                 // thread blocks of a pair
};

// Whether pair i is to be copied: its destination exists, and no later pair
// has the same one.
__device__ __forceinline__ bool takes(const CacheArgs &a, int i, int &src, int &dst)
{
    src = index_of(a.src, i);
    dst = index_of(a.dst, i);
    if (src < 0 || dst < 0 || dst >= a.ndst) return false;
    if (!a.dst) return true;
    for (int j0 = i + 1; j0 < a.n; j0 += 64) {
        const int j = j0 + (int)(threadIdx.x & 63);
        const bool again = j < a.n && a.dst[j] == dst && index_of(a.src, j) >= 0;
        if (__ballot(again) != 0) return false;
    }
    return true;
}

// Four lanes' worth of a block: one thread holds 4 of its values, 8 threads
// the block.
__global__ __launch_bounds__(CT) void k_state_pack(CacheArgs a, const float *states, uint8_t *cache, uint8_t *scales)
{
    const int i = blockIdx.x / a.chunks;
    int src, dst;
    if (!takes(a, i, src, dst)) return;
    const int64_t b = ((int64_t)(blockIdx.x % a.chunks) * CT + threadIdx.x) / 8;   // block of the state
    if (b >= a.per) return;   // the 8 threads of a block leave together
    const int part = threadIdx.x & 7;
    const int64_t row = b / a.nb;
    const int col = (int)(b % a.nb) * STATE_CACHE_BLOCK + part * 4;
    const int64_t at = row * a.dv + col, state = a.rows * a.dv;
    float x[4];
    float big = 0.f;
    bool bad = src >= a.nsrc;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = !bad && col + e < a.dv ? states[src * state + at + e] : 0.f;
        big = fmaxf(big, fabsf(x[e]));
        bad = bad || !(fabsf(x[e]) < __builtin_inff());
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2) {
        big = fmaxf(big, __shfl_xor(big, d));
        bad = __shfl_xor((int)bad, d) | (int)bad;
    }
    // big = m 2^e with m in [1/2, 1): 448 = 7/8 2^9
    int ex;
    const float m = frexpf(big, &ex);
    int s = m <= 0.875f ? ex - 9 : ex - 8;
    if (big == 0.f || s < -127) s = -127;
    unsigned word = 0x7f7f7f7fu;   // four NaN
    if (!bad) {
        word = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(x[0], -s), ldexpf(x[1], -s), 0, false);
        word = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(x[2], -s), ldexpf(x[3], -s), word, true);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < a.dv) cache[dst * state + at + e] = (uint8_t)(word >> (8 * e));
    if (part == 0) scales[dst * a.per + b] = bad ? 255 : (uint8_t)(s + 127);
}

__global__ __launch_bounds__(CT) void k_state_unpack(CacheArgs a, const uint8_t *cache, const uint8_t *scales,
                                                     float *states)
{
    const int i = blockIdx.x / a.chunks;
    int src, dst;
    if (!takes(a, i, src, dst)) return;
    const int64_t b = ((int64_t)(blockIdx.x % a.chunks) * CT + threadIdx.x) / 8;
    if (b >= a.per) return;
    const int64_t row = b / a.nb;
    const int col = (int)(b % a.nb) * STATE_CACHE_BLOCK + (threadIdx.x & 7) * 4;
    const int64_t at = row * a.dv + col, state = a.rows * a.dv;
    const bool none = src >= a.nsrc;
    unsigned word = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (!none && col + e < a.dv) word |= (unsigned)cache[src * state + at + e] << (8 * e);
    const int sb = none ? 255 : scales[src * a.per + b];
    float x[4];
    x[0] = __builtin_amdgcn_cvt_f32_fp8(word, 0);
    x[1] = __builtin_amdgcn_cvt_f32_fp8(word, 1);
    x[2] = __builtin_amdgcn_cvt_f32_fp8(word, 2);
    x[3] = __builtin_amdgcn_cvt_f32_fp8(word, 3);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < a.dv) states[dst * state + at + e] = sb == 255 ? __builtin_nanf("") : ldexpf(x[e], sb - 127);
}

// Fills the arguments; SSD_ERR_SHAPE for a grid that is too large.
static int cache_args(const state_cache_shape &s, const int32_t *src, int64_t nsrc, const int32_t *dst, int64_t ndst,
                      CacheArgs *a, unsigned *grid)
{
    a->src = src;
    a->dst = dst;
    a->n = (int)s.n;
    a->nsrc = (int)nsrc;
    a->ndst = (int)ndst;
    a->dk = (int)s.dk;
    a->dv = (int)s.dv;
    a->nb = (int)((s.dv + STATE_CACHE_BLOCK - 1) / STATE_CACHE_BLOCK);
    a->rows = s.H * s.dk;
    a->per = a->rows * a->nb;
    const int64_t chunks = (a->per * 8 + CT - 1) / CT;
    a->chunks = (int)chunks;
    if (s.n > ((int64_t(1) << 31) - 1) / chunks) return SSD_ERR_SHAPE;
    *grid = (unsigned)(s.n * chunks);
    return SSD_OK;
}

}  // namespace layer

using namespace layer;

extern "C" int state_pack(const state_cache_shape *shape, const float *states, const int32_t *slots,
                          const int32_t *entries, uint8_t *cache, uint8_t *scales, void *stream)
{
    int rc = check_cache(shape);
    if (rc != SSD_OK) return rc;
    const state_cache_shape &s = *shape;
    if ((!slots && s.n > s.slots) || (!entries && s.n > s.entries)) return SSD_ERR_SHAPE;
    CacheArgs a;
    unsigned grid = 0;
    rc = cache_args(s, slots, s.slots, entries, s.entries, &a, &grid);
    if (rc != SSD_OK) return rc;
    if (s.n == 0 || s.entries == 0) return SSD_OK;
    if ((s.slots > 0 && !states) || !cache || !scales) return SSD_ERR_NULL;
    if (misaligned(states, 4) || misaligned(slots, 4) || misaligned(entries, 4)) return SSD_ERR_ALIGN;
    k_state_pack<<<dim3(grid), dim3(CT), 0, static_cast<hipStream_t>(stream)>>>(a, states, cache, scales);
    return launch_status();
}

extern "C" int state_unpack(const state_cache_shape *shape, const uint8_t *cache, const uint8_t *scales,
                            const int32_t *entries, const int32_t *slots, float *states, void *stream)
{
    int rc = check_cache(shape);
    if (rc != SSD_OK) return rc;
    const state_cache_shape &s = *shape;
    if ((!slots && s.n > s.slots) || (!entries && s.n > s.entries)) return SSD_ERR_SHAPE;
    CacheArgs a;
    unsigned grid = 0;
    rc = cache_args(s, entries, s.entries, slots, s.slots, &a, &grid);
    if (rc != SSD_OK) return rc;
    if (s.n == 0 || s.slots == 0) return SSD_OK;
    if (!states || (s.entries > 0 && (!cache || !scales))) return SSD_ERR_NULL;
    if (misaligned(states, 4) || misaligned(slots, 4) || misaligned(entries, 4)) return SSD_ERR_ALIGN;
    k_state_unpack<<<dim3(grid), dim3(CT), 0, static_cast<hipStream_t>(stream)>>>(a, cache, scales, states);
    return launch_status();
}
