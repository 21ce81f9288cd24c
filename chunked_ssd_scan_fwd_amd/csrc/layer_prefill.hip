// The scalar-decay scan of a packed batch over a pool of states.
#include "layer_device.h"

namespace layer {

struct PrefillArgs {
    const void *q, *k, *v;
    const float *la;
    const int32_t *cu, *slots, *carry;
    float *states;
    void *y;
    int64_t la_t;
    lin_strides st;
    int T, N, G, H, dk, dv, nslots, tiles;
};

constexpr int PT = 256;

// The recurrence step by step: 64 columns of a head's state, a quarter of
// its rows in each wave.
template <typename T>
__global__ __launch_bounds__(PT) void k_lin_prefill(PrefillArgs a)
{
    __shared__ float red[2][PT / 64][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int tile = blockIdx.x % a.tiles, h = blockIdx.x / a.tiles % a.H, n = blockIdx.x / (a.tiles * a.H);
    const int g = h / (a.H / a.G), col = tile * 64 + lane;
    const bool on = col < a.dv;
    const int begin = min(max(a.cu[n], 0), a.T), end = min(max(a.cu[n + 1], begin), a.T);
    const int sl = index_of(a.slots, n);
    bool bad = sl >= a.nslots;
    if (a.slots && sl >= 0)
        for (int j = 0; j < n && !bad; ++j) bad = a.slots[j] == sl;
    T *y = static_cast<T *>(a.y) + h * a.st.y_h;
    if (bad) {
        for (int t = begin + wave; t < end; t += PT / 64)
            if (on) y[t * a.st.y_t + col] = from_f<T>(__builtin_nanf(""));
        return;
    }
    float *S = sl < 0 ? nullptr : a.states + ((int64_t)sl * a.H + h) * a.dk * a.dv + col;
    const bool read = S && (!a.carry || a.carry[n] != 0);
    const int per = (a.dk + 3) / 4, r0 = wave * per, r1 = min(r0 + per, a.dk);
    float s[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) s[i] = read && on && r0 + i < r1 ? S[(int64_t)(r0 + i) * a.dv] : 0.f;
    for (int t = begin; t < end; ++t) {
        const T *q = static_cast<const T *>(a.q) + t * a.st.q_t + g * a.st.q_g;
        const T *k = static_cast<const T *>(a.k) + t * a.st.k_t + g * a.st.k_g;
        const float v = on ? to_f(static_cast<const T *>(a.v)[t * a.st.v_t + h * a.st.v_h + col]) : 0.f;
        const float dec = expf(a.la[(a.la_t ? t * a.la_t : 0) + h]);
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (r0 + i < r1) {
                s[i] = dec * s[i] + to_f(k[r0 + i]) * v;
                o += to_f(q[r0 + i]) * s[i];
            }
        red[t & 1][wave][lane] = o;
        __syncthreads();
        if (wave == 0 && on)
            y[t * a.st.y_t + col] = from_f<T>(red[t & 1][0][lane] + red[t & 1][1][lane] + red[t & 1][2][lane] +
                                              red[t & 1][3][lane]);
    }
    if (S && on)
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (r0 + i < r1) S[(int64_t)(r0 + i) * a.dv] = s[i];
}

}  // namespace layer

using namespace layer;

extern "C" size_t lin_prefill_workspace_size(const lin_shape *shape, int64_t max_seqlen)
{
    if (check_lin(shape, false) != SSD_OK || max_seqlen < 0) return (size_t)-1;
    return 0;
}

extern "C" int lin_prefill(const lin_shape *shape, int dtype, const lin_strides *strides, const void *q,
                           const void *k, const void *v, const float *log_decay, int64_t decay_stride,
                           const int32_t *cu_seqlens, const int32_t *slots, const int32_t *carry,
                           int64_t max_seqlen, float *states, void *y, void *workspace, size_t workspace_bytes,
                           void *stream)
{
    int rc = check_lin(shape, false);
    if (rc == SSD_OK) rc = check_dtype(dtype);
    if (rc != SSD_OK) return rc;
    const lin_shape &s = *shape;
    PrefillArgs a;
    rc = resolve_strides(shape, strides, &a.st, s.T);
    if (rc != SSD_OK) return rc;
    if (decay_stride < 0 || decay_stride >= kMaxCount || max_seqlen < 0) return SSD_ERR_SHAPE;
    if (!slots && s.N > s.slots) return SSD_ERR_SHAPE;
    if (s.N == 0) return SSD_OK;
    if (!cu_seqlens || (s.slots > 0 && !states)) return SSD_ERR_NULL;
    if (s.T > 0 && (!q || !k || !v || !log_decay || !y)) return SSD_ERR_NULL;
    const unsigned e = dtype_size(dtype);
    if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(y, e) || misaligned(log_decay, 4) ||
        misaligned(slots, 4) || misaligned(states, 4) || misaligned(cu_seqlens, 4) || misaligned(carry, 4))
        return SSD_ERR_ALIGN;
    (void)workspace;
    (void)workspace_bytes;
    a.q = q;
    a.k = k;
    a.v = v;
    a.la = log_decay;
    a.la_t = decay_stride;
    a.cu = cu_seqlens;
    a.slots = slots;
    a.carry = carry;
    a.states = states;
    a.y = y;
    a.T = (int)s.T;
    a.N = (int)s.N;
    a.G = (int)s.G;
    a.H = (int)s.H;
    a.dk = (int)s.dk;
    a.dv = (int)s.dv;
    a.nslots = (int)s.slots;
    a.tiles = (a.dv + 63) / 64;
    hipStream_t st = static_cast<hipStream_t>(stream);
    LAYER_DISPATCH(dtype, (k_lin_prefill<T><<<dim3((unsigned)((int64_t)a.N * a.H * a.tiles)), dim3(PT), 0, st>>>(a)));
    return launch_status();
}
