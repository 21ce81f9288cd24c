// One step of the scalar-decay scan for each running sequence:
//   S <- e^{log_decay} S + k v^T,   y = S^T q,   S in float32, in place.
//
// Every state is read and written once (8 dk dv bytes for each row and head;
// q, k, v and y are 1/dk of that), so memory bounds it, and for a few rows
// the latency of two dependent loads (slot, then state).
#include "layer_device.h"
#include "ssd_internal.h"

namespace layer {

constexpr int ST = 256;   // threads of a block

struct StepArgs {
    const void *q, *k, *v;
    const float *la;
    const int32_t *slots;
    float *states;
    void *y;
    int64_t la_n;         // row stride of log_decay, 0 for one decay for each head
    lin_strides st;
    int N, G, H, dk, dv, nslots, tiles;
};

// One block takes TV = CL * VEC columns of one head's state for one row: CL
// threads across a row of the state, ST / CL rows at a time.
template <typename T, int VEC, int CL, bool STREAM>
__global__ __launch_bounds__(ST) void k_lin_step(StepArgs a)
{
    constexpr int TV = CL * VEC, R = ST / CL;
    typedef Vec<float, VEC> V;
    __shared__ float qs[kMaxHeadDim], ks[kMaxHeadDim], red[ST / 64][TV];
    const int tid = threadIdx.x;
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
    bool before = false;
    int next = a.N;
    if (a.slots) same_slot(a.slots, a.N, n, sl, before, next);
    if (before) return;   // the block of the slot's first row takes all of them
    float *S = a.states + ((int64_t)sl * a.H + h) * a.dk * a.dv + c0 + col;
    while (true) {
        const T *q = static_cast<const T *>(a.q) + n * a.st.q_t + g * a.st.q_g;
        const T *k = static_cast<const T *>(a.k) + n * a.st.k_t + g * a.st.k_g;
        const T *v = static_cast<const T *>(a.v) + n * a.st.v_t + h * a.st.v_h + c0 + col;
        for (int r = tid; r < a.dk; r += ST) {
            qs[r] = to_f(q[r]);
            ks[r] = to_f(k[r]);
        }
        float vv[VEC], y[VEC] = {};
#pragma unroll
        for (int i = 0; i < VEC; ++i) vv[i] = on ? to_f(v[i]) : 0.f;
        const float dec = expf(a.la[(a.la_n ? n * a.la_n : 0) + h]);
        __syncthreads();
        if (on) {
#pragma unroll 8
            for (int r = r0; r < a.dk; r += R) {
                V x = load_state<VEC, STREAM>(S + (int64_t)r * a.dv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    x.v[i] = dec * x.v[i] + ks[r] * vv[i];
                    y[i] += qs[r] * x.v[i];
                }
                store_state<VEC, STREAM>(S + (int64_t)r * a.dv, x);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
            for (int d = CL; d < 64; d *= 2) y[i] += __shfl_xor(y[i], d);
            if ((tid & 63) < CL) red[tid >> 6][col + i] = y[i];
        }
        __syncthreads();
        if (tid < TV && c0 + tid < a.dv) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < ST / 64; ++w) s += red[w][tid];
            yb[n * a.st.y_t + tid] = from_f<T>(s);
        }
        if (next >= a.N) break;
        n = next;
        bool b;
        same_slot(a.slots, a.N, n, sl, b, next);
        __syncthreads();   // qs, ks and red are free again
    }
}

// Columns of a block: as many as dv has, up to 128, so that no thread is
// idle (24 heads of 64 columns: 91 us with 64, 97 with 128); fewer while
// there is no block for every CU (one row of 8 heads of 128 x 128: 4.2 us with
// 32, 5.9 with 128).
//
// States of more than 128 MiB in a call go past the caches: 256 rows of 24
// heads of 128 x 64 (201 MB) took 84 us so and 91 otherwise where other data
// passed in between, as other layers' does; the same states alone and again,
// 82 and 62.
template <typename T>
static void launch_step(StepArgs &a, int cus, hipStream_t st)
{
    const auto go = [&](auto kernel, int tv) {
        a.tiles = (a.dv + tv - 1) / tv;
        kernel<<<dim3((unsigned)((int64_t)a.N * a.H * a.tiles)), dim3(ST), 0, st>>>(a);
    };
    if (a.dv % 4 != 0 || misaligned(a.states, 16)) return go(k_lin_step<T, 1, 64, false>, 64);
    const auto blocks = [&](int tv) { return (int64_t)a.N * a.H * ((a.dv + tv - 1) / tv); };
    const bool stream = (int64_t)a.N * a.H * a.dk * a.dv * 4 > (int64_t(128) << 20);
    if (a.dv > 64 && blocks(128) >= cus)
        return stream ? go(k_lin_step<T, 4, 32, true>, 128) : go(k_lin_step<T, 4, 32, false>, 128);
    if (a.dv > 32 && blocks(64) >= cus)
        return stream ? go(k_lin_step<T, 4, 16, true>, 64) : go(k_lin_step<T, 4, 16, false>, 64);
    return stream ? go(k_lin_step<T, 4, 8, true>, 32) : go(k_lin_step<T, 4, 8, false>, 32);
}

}  // namespace layer

using namespace layer;

extern "C" int lin_step(const lin_shape *shape, int dtype, const lin_strides *strides, const void *q, const void *k,
                        const void *v, const float *log_decay, int64_t decay_stride, const int32_t *slots,
                        float *states, void *y, void *stream)
{
    int rc = check_lin(shape, true);
    if (rc == SSD_OK) rc = check_dtype(dtype);
    if (rc != SSD_OK) return rc;
    const lin_shape &s = *shape;
    StepArgs a;
    rc = resolve_strides(shape, strides, &a.st, s.N);
    if (rc != SSD_OK) return rc;
    if (decay_stride < 0 || decay_stride >= kMaxCount) return SSD_ERR_SHAPE;
    if (!slots && s.N > s.slots) return SSD_ERR_SHAPE;
    if (s.N == 0) return SSD_OK;
    if (!q || !k || !v || !log_decay || !y || (s.slots > 0 && !states)) return SSD_ERR_NULL;
    const unsigned e = dtype_size(dtype);
    if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(y, e) || misaligned(log_decay, 4) ||
        misaligned(slots, 4) || misaligned(states, 4))
        return SSD_ERR_ALIGN;
    a.q = q;
    a.k = k;
    a.v = v;
    a.la = log_decay;
    a.la_n = decay_stride;
    a.slots = slots;
    a.states = states;
    a.y = y;
    a.N = (int)s.N;
    a.G = (int)s.G;
    a.H = (int)s.H;
    a.dk = (int)s.dk;
    a.dv = (int)s.dv;
    a.nslots = (int)s.slots;
    LAYER_DISPATCH(dtype, launch_step<T>(a, ssd::device_cus(), static_cast<hipStream_t>(stream)));
    return launch_status();
}
