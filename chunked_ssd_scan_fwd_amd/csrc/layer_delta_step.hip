// One step of the gated delta rule for each running sequence:
//   u = beta (v - a S^T k),   S <- a S + k u^T,   y = S^T q,   a = e^{log_decay}
// S in float32, in place.
//
// S is read and written once (8 dk dv bytes for each row and head; q, k, v and
// y are 1/dk of that), so memory bounds it, and for a few rows the latency of
// two dependent loads (slot, then state).  u needs all of a column before any
// of it can be written, so a block keeps its columns in registers, and y is
// taken from the same pass over them: S'^T q = a S^T q + (k . q) u.
//
// The states go past the caches: by a next step the other layers' have taken
// their place.  Over 3 GB of layers, each with 16 rows of 16 heads of 128 x 128,
// 7.8 us a call, and through the caches 10.7; with 128 rows 49 and 59.  A small
// model, whose states all stay in the last cache, gains too: 117 MB of layers of
// 16 rows 8.4 and 9.8, 34 MB of layers of one row of 8 heads 3.8 and 4.3.
//
// Captured calls on such layers, 256 rows (537 MB): 96 us, 5.6 TB/s.  One after
// the other from Python, with new inputs, 109 us (4.9 TB/s).
#include "layer_device.h"
#include "ssd_internal.h"

namespace layer {

constexpr int DT = 256;   // threads of a block

struct DeltaStepArgs {
    const void *q, *k, *v;
    const float *la, *beta;
    const int32_t *slots;
    float *states;
    void *y;
    int64_t la_n, beta_n;   // row strides; la_n 0 for one decay for each head
    lin_strides st;
    int N, G, H, dk, dv, nslots, tiles;
};

// One block takes TV = CL * VEC columns of one head's state for one row: CL
// threads across a row of the state, DT / CL rows at a time, NR times.
template <typename T, int VEC, int CL, int NR>
__global__ __launch_bounds__(DT) void k_delta_step(DeltaStepArgs a)
{
    constexpr int TV = CL * VEC, R = DT / CL, W = DT / 64;
    typedef Vec<float, VEC> V;
    __shared__ float qs[NR * R], ks[NR * R], red[2][W][TV], dots[W];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int tile = blockIdx.x % a.tiles;
    const int h = blockIdx.x / a.tiles % a.H;
    int n = blockIdx.x / (a.tiles * a.H);
    const int g = h / (a.H / a.G);
    const int c0 = tile * TV, col = tid % CL * VEC, r0 = tid / CL;
    const bool on = c0 + col < a.dv;   // VEC > 1 only where dv is a multiple of it
    const int sl = index_of(a.slots, n);
    if (sl < 0) return;
    T *yb = static_cast<T *>(a.y) + h * a.st.y_h + c0;
    if (sl >= a.nslots) {
        if (tid < TV && c0 + tid < a.dv) yb[n * a.st.y_t + tid] = from_f<T>(__builtin_nanf(""));
        return;
    }
    float *S = a.states + ((int64_t)sl * a.H + h) * a.dk * a.dv + c0 + col;
    V x[NR];
#pragma unroll
    for (int u = 0; u < NR; ++u) {
        const int r = r0 + u * R;
        x[u] = V{};
        if (on && r < a.dk) x[u] = load_state<VEC, true>(S + (int64_t)r * a.dv);
    }
    bool before = false;
    int next = a.N;
    if (a.slots) same_slot(a.slots, a.N, n, sl, before, next);
    if (before) return;   // the block of the slot's first row takes all of them
    while (true) {
        const T *q = static_cast<const T *>(a.q) + n * a.st.q_t + g * a.st.q_g;
        const T *k = static_cast<const T *>(a.k) + n * a.st.k_t + g * a.st.k_g;
        const T *v = static_cast<const T *>(a.v) + n * a.st.v_t + h * a.st.v_h + c0 + col;
        for (int r = tid; r < NR * R; r += DT) {
            qs[r] = r < a.dk ? to_f(q[r]) : 0.f;
            ks[r] = r < a.dk ? to_f(k[r]) : 0.f;
        }
        float vv[VEC], sk[VEC] = {}, sq[VEC] = {}, kq = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) vv[i] = on ? to_f(v[i]) : 0.f;
        const float dec = expf(a.la[(a.la_n ? n * a.la_n : 0) + h]), beta = a.beta[n * a.beta_n + h];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < NR; ++u) {
            const float kr = ks[r0 + u * R], qr = qs[r0 + u * R];
            kq += kr * qr;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sk[i] += kr * x[u].v[i];
                sq[i] += qr * x[u].v[i];
            }
        }
        // over the rows: the lanes CL apart, then the waves
#pragma unroll
        for (int d = CL; d < 64; d *= 2) {
            kq += __shfl_xor(kq, d);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sk[i] += __shfl_xor(sk[i], d);
                sq[i] += __shfl_xor(sq[i], d);
            }
        }
        if ((tid & 63) < CL) {
            if ((tid & 63) == 0) dots[wave] = kq;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                red[0][wave][col + i] = sk[i];
                red[1][wave][col + i] = sq[i];
            }
        }
        __syncthreads();
        kq = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) kq += dots[w];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float s = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                s += red[0][w][col + i];
                y += red[1][w][col + i];
            }
            const float uu = beta * (vv[i] - dec * s);
            if (on && r0 == 0) yb[n * a.st.y_t + col + i] = from_f<T>(dec * y + kq * uu);
#pragma unroll
            for (int u = 0; u < NR; ++u) x[u].v[i] = dec * x[u].v[i] + ks[r0 + u * R] * uu;
        }
        if (next >= a.N) break;
        n = next;
        bool b;
        same_slot(a.slots, a.N, n, sl, b, next);
        __syncthreads();   // qs, ks and red are free again
    }
#pragma unroll
    for (int u = 0; u < NR; ++u) {
        const int r = r0 + u * R;
        if (on && r < a.dk) store_state<VEC, true>(S + (int64_t)r * a.dv, x[u]);
    }
}

template <typename T, int VEC, int CL>
static void launch_rows(DeltaStepArgs &a, hipStream_t st)
{
    constexpr int R = DT / CL;
    a.tiles = (a.dv + CL * VEC - 1) / (CL * VEC);
    const dim3 grid((unsigned)((int64_t)a.N * a.H * a.tiles));
    if (a.dk <= 64)
        k_delta_step<T, VEC, CL, 64 / R><<<grid, dim3(DT), 0, st>>>(a);
    else if (a.dk <= 128)
        k_delta_step<T, VEC, CL, 128 / R><<<grid, dim3(DT), 0, st>>>(a);
    else
        k_delta_step<T, VEC, CL, 256 / R><<<grid, dim3(DT), 0, st>>>(a);
}

// Columns of a block: 64 where that makes a block for every CU, else 32.  (16
// heads of 128 x 128, captured: 64 rows 24.6 us with 64, 27.7 with 32, 256 rows
// 96 and 104; one row of 8 heads 4.1 and 3.8.)
template <typename T>
static void launch_delta_step(DeltaStepArgs &a, int cus, hipStream_t st)
{
    if (a.dv % 4 != 0 || misaligned(a.states, 16)) return launch_rows<T, 1, 32>(a, st);
    if (a.dv > 32 && (int64_t)a.N * a.H * ((a.dv + 63) / 64) >= cus) return launch_rows<T, 4, 16>(a, st);
    return launch_rows<T, 4, 8>(a, st);
}

}  // namespace layer

using namespace layer;

extern "C" int delta_step(const lin_shape *shape, int dtype, const lin_strides *strides, const void *q, const void *k,
                          const void *v, const float *log_decay, int64_t decay_stride, const float *beta,
                          int64_t beta_stride, const int32_t *slots, float *states, void *y, void *stream)
{
    int rc = check_delta(shape, true);
    if (rc == SSD_OK) rc = check_dtype(dtype);
    if (rc != SSD_OK) return rc;
    const lin_shape &s = *shape;
    DeltaStepArgs a;
    rc = resolve_strides(shape, strides, &a.st, s.N);
    if (rc != SSD_OK) return rc;
    if (decay_stride < 0 || decay_stride >= kMaxCount || beta_stride < 0 || beta_stride >= kMaxCount)
        return SSD_ERR_SHAPE;
    if (!slots && s.N > s.slots) return SSD_ERR_SHAPE;
    if (s.N == 0) return SSD_OK;
    if (!q || !k || !v || !log_decay || !beta || !y || (s.slots > 0 && !states)) return SSD_ERR_NULL;
    const unsigned e = dtype_size(dtype);
    if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(y, e) || misaligned(log_decay, 4) ||
        misaligned(beta, 4) || misaligned(slots, 4) || misaligned(states, 4))
        return SSD_ERR_ALIGN;
    a.q = q;
    a.k = k;
    a.v = v;
    a.la = log_decay;
    a.la_n = decay_stride;
    a.beta = beta;
    a.beta_n = beta_stride;
    a.slots = slots;
    a.states = states;
    a.y = y;
    a.N = (int)s.N;
    a.G = (int)s.G;
    a.H = (int)s.H;
    a.dk = (int)s.dk;
    a.dv = (int)s.dv;
    a.nslots = (int)s.slots;
    LAYER_DISPATCH(dtype, launch_delta_step<T>(a, ssd::device_cus(), static_cast<hipStream_t>(stream)));
    return launch_status();
}
