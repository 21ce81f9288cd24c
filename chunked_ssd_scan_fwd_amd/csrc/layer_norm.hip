// Group norm, channels last, with an activation on the normalised value or
// on a gate, and its gradient.  For sample n and run of channels j, over
// M = L C / groups values:
//   mu = sum x / M,  rstd = (sum (x - mu)^2 / M + eps)^(-1/2),
//   xh = (x - mu) rstd,  z = xh weight + bias,  y = act(z) or z act(gate).
// With dz = dy act'(z) or dy act(gate), and d = dz weight:
//   dx = rstd (d - mean(d) - xh mean(d xh)),
//   dgate = dy z act'(gate),  dweight = sum dz xh,  dbias = sum dz.
// act is SiLU: act(u) = u s, act'(u) = s (1 + u (1 - s)), s = 1 / (1 + e^-u).
//
// Memory bounds all of it.  Two ways through the data:
//
// * A sample's run of M values that fits the registers of its threads (up to
//   64 lanes of a wave, or one block) is read once: k_gn_fwd_held and
//   k_gn_bwd_held.  The threads of a block keep their channels from sample to
//   sample, so the backward sums dweight and dbias in registers.
// * Longer runs are cut into parts of rows.  k_gn_sums reads them once for
//   each channel's sums over a part, k_gn_mid joins these for each run, and
//   k_gn_apply reads the data again.
//
// k_gn_wsum, or k_gn_mid's last blocks, add up the parts of dweight and dbias
// in a fixed order.
#include "layer_device.h"
#include "ssd_internal.h"

namespace layer {

constexpr int GT = 512;   // threads of a block
constexpr int HELD = 4;   // most pieces of a run that a thread holds

struct GnArgs {
    const void *x, *gate, *dy;
    const float *w, *b;
    void *y, *dx, *dgate;
    float *stats, *dw, *db;
    float *part;        // held: [nparts][2][C]; cut: [N][nparts][2][C]
    float *mean;        // cut, backward: [N][groups][2], mean(d) and mean(d xh)
    int64_t N, ldx, ldg, ldy;
    int64_t nparts, per;   // cut: parts of a sample, rows of a part
    int64_t block0;        // cut: the launch's first of the blocks
    int L, C, groups, cg;
    float eps;
    bool silu;
    // held: 2^lw threads to a run; gs runs of one sample side by side in a
    // block (of sets blocks for all of them), rpb samples; a run's rows have
    // ppr pieces, the run has `pieces`
    int lw, gs, rpb, sets, ppr, pieces;
};

struct Act {
    float f, df;   // act(u) and act'(u)
};
__device__ __forceinline__ Act act(float u, bool silu)
{
    if (!silu) return {u, 1.f};
    const float s = __builtin_amdgcn_rcpf(1.f + __expf(-u));
    return {u * s, s * (1.f + u * (1.f - s))};
}

template <typename T, int VE>
__device__ __forceinline__ Vec<T, VE> load(const T *p, bool on)
{
    Vec<T, VE> r = {};
    if (on) r = *reinterpret_cast<const Vec<T, VE> *>(p);
    return r;
}
// The same for what is read once by the whole call: a non-temporal load.
// The forward on 16384 rows of 2048 took 40 us with it and 51 without; the
// backward, whose second tensor pair crowds the caches anyway, 25 both ways.
template <typename T, int VE>
__device__ __forceinline__ Vec<T, VE> load_once(const T *p, bool on)
{
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    if constexpr (sizeof(Vec<T, VE>) == 16) {
        u32x4 r = {};
        if (on) r = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
        return __builtin_bit_cast(Vec<T, VE>, r);
    } else {
        return load<T, VE>(p, on);
    }
}
// weight or bias of VE channels
template <int VE>
__device__ __forceinline__ void channels(float (&to)[VE], const float *p, float none, bool on)
{
#pragma unroll
    for (int i = 0; i < VE; ++i) to[i] = p && on ? p[i] : none;
}

// Sum over a run's 2^lw threads, in each of them: up to a wave's lanes, or the
// whole block (then every thread of the block calls it).
__device__ __forceinline__ void run_sum(float &a, float &b, int lw, float (&red)[2][GT / 64])
{
    const int lanes = lw > 6 ? 6 : lw;
    for (int d = 1; d < 1 << lanes; d *= 2) {
        a += __shfl_xor(a, d);
        b += __shfl_xor(b, d);
    }
    if (lw <= 6) return;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        red[0][threadIdx.x >> 6] = a;
        red[1][threadIdx.x >> 6] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < GT / 64; ++w) {
        a += red[0][w];
        b += red[1][w];
    }
}

// Where a thread of the held kernels works: run `run` of every rpb-th sample
// from `first` on, piece k at row l[k] and channel c[k] of the sample.
template <int VE, int K>
struct Held {
    int run, first, c[K], l[K];
    bool on[K];
    __device__ __forceinline__ explicit Held(const GnArgs &a)
    {
        const int set = blockIdx.x % a.sets, slot = threadIdx.x >> a.lw, j = threadIdx.x & ((1 << a.lw) - 1);
        const int rs = slot / a.gs, g = set * a.gs + slot % a.gs;
        const bool live = rs < a.rpb && g < a.groups;
        run = live ? g : -1;
        first = blockIdx.x / a.sets * a.rpb + rs;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int p = j + (k << a.lw);
            on[k] = live && p < a.pieces;
            l[k] = p / a.ppr;
            c[k] = g * a.cg + p % a.ppr * VE;
        }
    }
};

template <typename T, int VE, int K>
__global__ __launch_bounds__(GT) void k_gn_fwd_held(GnArgs a)
{
    __shared__ float red[2][GT / 64];
    const Held<VE, K> h(a);
    if (h.run < 0) return;   // a run's threads leave together
    const int64_t step = (int64_t)(gridDim.x / a.sets) * a.rpb;
    const float inv = 1.f / ((float)a.L * (float)a.cg);
    const bool first = (threadIdx.x & ((1 << a.lw) - 1)) == 0;
    float w[K][VE], b[K][VE];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        channels<VE>(w[k], a.w ? a.w + h.c[k] : nullptr, 1.f, h.on[k]);
        channels<VE>(b[k], a.b ? a.b + h.c[k] : nullptr, 0.f, h.on[k]);
    }
    for (int64_t n = h.first; n < a.N; n += step) {
        Vec<T, VE> x[K], gt[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t row = n * a.L + h.l[k];
            x[k] = load_once<T, VE>(static_cast<const T *>(a.x) + row * a.ldx + h.c[k], h.on[k]);
            if (a.gate) gt[k] = load_once<T, VE>(static_cast<const T *>(a.gate) + row * a.ldg + h.c[k], h.on[k]);
        }
        float s = 0.f, none = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VE; ++i) s += to_f(x[k].v[i]);   // absent ones are 0
        run_sum(s, none, a.lw, red);
        const float mu = s * inv;
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float d = to_f(x[k].v[i]) - mu;
                q += h.on[k] ? d * d : 0.f;
            }
        run_sum(q, none, a.lw, red);
        const float rstd = 1.f / sqrtf(q * inv + a.eps);
        if (first) {
            float *st = a.stats + 2 * (n * a.groups + h.run);
            st[0] = mu;
            st[1] = rstd;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!h.on[k]) continue;
            Vec<T, VE> y;
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float z = (to_f(x[k].v[i]) - mu) * rstd * w[k][i] + b[k][i];
                y.v[i] = from_f<T>(a.gate ? z * act(to_f(gt[k].v[i]), a.silu).f : act(z, a.silu).f);
            }
            *reinterpret_cast<Vec<T, VE> *>(static_cast<T *>(a.y) + (n * a.L + h.l[k]) * a.C + h.c[k]) = y;
        }
    }
}

struct GnGrad {
    float xh, dz, dgate;
};

// The parts of the gradient that belong to one value.
__device__ __forceinline__ GnGrad gn_grad(float x, float mu, float rstd, float w, float b, bool gated, float gate,
                                          float dy, bool silu)
{
    GnGrad r;
    r.xh = (x - mu) * rstd;
    const float z = r.xh * w + b;
    const Act t = act(gated ? gate : z, silu);
    r.dz = dy * (gated ? t.f : t.df);
    r.dgate = dy * z * t.df;
    return r;
}

// Adds up what the threads of a block hold of dweight or dbias, in a fixed
// order, into the block's row of `part`: `held` lists it by thread slot and
// piece; a channel's values are those of its run's rows and of the block's
// samples.  As many threads take a channel as there are for all.
template <int VE, int K>
__device__ __forceinline__ void held_part(const GnArgs &a, const float (&v)[K][VE], float *held, float *sub, float *to)
{
    const int W = 1 << a.lw;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VE; ++i) held[((threadIdx.x >> a.lw) * K * W + k * W + (threadIdx.x & (W - 1))) * VE + i] = v[k][i];
    __syncthreads();
    const int set = blockIdx.x % a.sets, cb = min(a.gs, a.groups - set * a.gs) * a.cg;   // the block's channels
    int ns = 1;
    while (ns * 2 * cb <= GT) ns *= 2;
    const int terms = a.rpb * a.L;
    for (int c0 = 0; c0 < cb; c0 += GT / ns) {
        const int c = c0 + (int)threadIdx.x / ns, s = threadIdx.x % ns;
        float t = 0.f;
        if (c < cb) {
            const int g = c / a.cg, ch = c % a.cg;
            for (int e = s; e < terms; e += ns) {
                const int rs = e / a.L, l = e % a.L;
                t += held[((rs * a.gs + g) * K * W + l * a.ppr + ch / VE) * VE + ch % VE];
            }
        }
        sub[threadIdx.x] = t;
        __syncthreads();
        if (s == 0 && c < cb) {
            for (int i = 1; i < ns; ++i) t += sub[threadIdx.x + i];
            to[set * a.gs * a.cg + c] = t;
        }
        __syncthreads();
    }
}

template <typename T, int VE, int K>
__global__ __launch_bounds__(GT) void k_gn_bwd_held(GnArgs a)
{
    __shared__ float red[2][GT / 64], held[GT * VE * K], sub[GT];
    const Held<VE, K> h(a);
    const int64_t step = (int64_t)(gridDim.x / a.sets) * a.rpb;
    const float inv = 1.f / ((float)a.L * (float)a.cg);
    float aw[K][VE] = {}, ab[K][VE] = {}, w[K][VE], b[K][VE];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        channels<VE>(w[k], a.w ? a.w + h.c[k] : nullptr, 1.f, h.on[k]);
        channels<VE>(b[k], a.b ? a.b + h.c[k] : nullptr, 0.f, h.on[k]);
    }
    if (h.run >= 0 && h.first < a.N) {
        // what one sample's run takes, fetched while the one before is worked on
        struct Row {
            Vec<T, VE> x[K], gt[K], dy[K];
            float mu, rstd;
        } r, ahead;
        const auto fetch = [&](Row &to, int64_t n) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int64_t row = n * a.L + h.l[k];
                to.x[k] = load<T, VE>(static_cast<const T *>(a.x) + row * a.ldx + h.c[k], h.on[k]);
                to.dy[k] = load<T, VE>(static_cast<const T *>(a.dy) + row * a.ldy + h.c[k], h.on[k]);
                if (a.gate) to.gt[k] = load<T, VE>(static_cast<const T *>(a.gate) + row * a.ldg + h.c[k], h.on[k]);
            }
            const float *st = a.stats + 2 * (n * a.groups + h.run);
            to.mu = st[0];
            to.rstd = st[1];
        };
        fetch(r, h.first);
        for (int64_t n = h.first; n < a.N; n += step) {
            fetch(ahead, n + step < a.N ? n + step : n);
            const float mu = r.mu, rstd = r.rstd;
            float xh[K][VE], d[K][VE], s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Vec<T, VE> dg;
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const GnGrad t = gn_grad(to_f(r.x[k].v[i]), mu, rstd, w[k][i], b[k][i], a.gate != nullptr,
                                             a.gate ? to_f(r.gt[k].v[i]) : 0.f, to_f(r.dy[k].v[i]), a.silu);
                    const float dz = h.on[k] ? t.dz : 0.f;
                    xh[k][i] = h.on[k] ? t.xh : 0.f;
                    d[k][i] = dz * w[k][i];
                    s1 += d[k][i];
                    s2 += d[k][i] * xh[k][i];
                    aw[k][i] += dz * xh[k][i];
                    ab[k][i] += dz;
                    dg.v[i] = from_f<T>(t.dgate);
                }
                if (a.dgate && h.on[k])
                    *reinterpret_cast<Vec<T, VE> *>(static_cast<T *>(a.dgate) + (n * a.L + h.l[k]) * a.C + h.c[k]) = dg;
            }
            r = ahead;
            if (!a.dx) continue;
            run_sum(s1, s2, a.lw, red);
            const float m1 = s1 * inv, m2 = s2 * inv;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!h.on[k]) continue;
                Vec<T, VE> dx;
#pragma unroll
                for (int i = 0; i < VE; ++i) dx.v[i] = from_f<T>(rstd * (d[k][i] - m1 - xh[k][i] * m2));
                *reinterpret_cast<Vec<T, VE> *>(static_cast<T *>(a.dx) + (n * a.L + h.l[k]) * a.C + h.c[k]) = dx;
            }
        }
    }
    if (!a.part) return;
    float *part = a.part + 2 * (int64_t)(blockIdx.x / a.sets) * a.C;
    held_part<VE, K>(a, aw, held, sub, part);
    held_part<VE, K>(a, ab, held, sub, part + a.C);
}

// ---- runs that are cut into parts of rows
//
// A block takes a part of a sample: cp threads side by side on a row's
// pieces (of tiles of GT of them), GT / cp rows at a time.

template <int VE>
struct Cut {
    int64_t n, part;
    int c, r0, rp, l0, l1;   // channel, first row, rows at a time; the part's rows
    bool on;
    __device__ __forceinline__ explicit Cut(const GnArgs &a)
    {
        const int64_t block = a.block0 + blockIdx.x;
        const int cp = min(a.C / VE, GT), tiles = (a.C / VE + GT - 1) / GT;
        const int tile = (int)(block % tiles);
        part = block / tiles % a.nparts;
        n = block / tiles / a.nparts;
        rp = GT / cp;
        c = (tile * GT + (int)threadIdx.x % cp) * VE;
        r0 = threadIdx.x / cp;
        on = r0 < rp && c < a.C;
        l0 = (int)(part * a.per);
        l1 = (int)min((part + 1) * a.per, (int64_t)a.L);
    }
};

// A part's sums for each channel.  Forward: mean and sum of squares about it,
// formed from differences to the thread's first value, so that a mean far
// from zero costs no accuracy.  Backward: sums of dz and dz xh.
template <typename T, int VE, bool BWD>
__global__ __launch_bounds__(GT) void k_gn_sums(GnArgs a)
{
    __shared__ float red[2][VE][GT], cnt[GT];
    const Cut<VE> p(a);
    float s[2][VE] = {}, x0[VE] = {}, w[VE], b[VE], mu[VE], rstd[VE];
    int rows = 0;
    if (p.on) {
        if (BWD) {
            channels<VE>(w, a.w ? a.w + p.c : nullptr, 1.f, true);
            channels<VE>(b, a.b ? a.b + p.c : nullptr, 0.f, true);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float *st = a.stats + 2 * (p.n * a.groups + (p.c + i) / a.cg);
                mu[i] = st[0];
                rstd[i] = st[1];
            }
        }
        if (!BWD && p.l0 + p.r0 < p.l1) {
            const Vec<T, VE> x =
                load<T, VE>(static_cast<const T *>(a.x) + (p.n * a.L + p.l0 + p.r0) * a.ldx + p.c, true);
#pragma unroll
            for (int i = 0; i < VE; ++i) x0[i] = to_f(x.v[i]);
        }
#pragma unroll 4
        for (int l = p.l0 + p.r0; l < p.l1; l += p.rp) {
            const int64_t row = p.n * a.L + l;
            const Vec<T, VE> x = load<T, VE>(static_cast<const T *>(a.x) + row * a.ldx + p.c, true);
            Vec<T, VE> dy = {}, gt = {};
            if (BWD) {
                dy = load<T, VE>(static_cast<const T *>(a.dy) + row * a.ldy + p.c, true);
                if (a.gate) gt = load<T, VE>(static_cast<const T *>(a.gate) + row * a.ldg + p.c, true);
            }
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                if (BWD) {
                    const GnGrad r = gn_grad(to_f(x.v[i]), mu[i], rstd[i], w[i], b[i], a.gate != nullptr,
                                             to_f(gt.v[i]), to_f(dy.v[i]), a.silu);
                    s[0][i] += r.dz * r.xh;
                    s[1][i] += r.dz;
                } else {
                    const float d = to_f(x.v[i]) - x0[i];
                    s[0][i] += d;
                    s[1][i] += d * d;
                }
            }
            ++rows;
        }
    }
    if (!BWD && rows > 0)
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const float m = s[0][i] / (float)rows;
            s[1][i] = fmaxf(s[1][i] - m * s[0][i], 0.f) + 0.f * s[1][i];   // and a NaN stays one
            s[0][i] = x0[i] + m;
        }
    // join the threads of a column of rows, pairs in a fixed order
    const int cp = min(a.C / VE, GT);
    float count = (float)rows;
    int half = 1;
    while (half < p.rp) half *= 2;
    for (half /= 2; half > 0; half /= 2) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            red[0][i][threadIdx.x] = s[0][i];
            red[1][i][threadIdx.x] = s[1][i];
        }
        cnt[threadIdx.x] = count;
        __syncthreads();
        const int other = threadIdx.x + half * cp;
        if (p.r0 < half && p.r0 + half < p.rp) {
            const float k = cnt[other];
            if (BWD || k > 0.f) {
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float u = red[0][i][other], v = red[1][i][other];
                    if (BWD) {
                        s[0][i] += u;
                        s[1][i] += v;
                    } else {   // rows go to the lower threads first, so this one has some
                        const float d = u - s[0][i], f = k / (count + k);
                        s[0][i] += d * f;
                        s[1][i] += v + d * d * count * f;
                    }
                }
                count += k;
            }
        }
    }
    if (p.on && p.r0 == 0) {
        float *to = a.part + (p.n * a.nparts + p.part) * 2 * a.C + p.c;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            to[i] = s[0][i];
            to[a.C + i] = s[1][i];
        }
    }
}

// Joins a run's parts and channels: forward, its statistics; backward,
// mean(d) and mean(d xh).
template <bool BWD>
__device__ __forceinline__ void gn_join(const GnArgs &a, int64_t run, float (&red)[2][GT / 64])
{
    const int64_t n = run / a.groups;
    const int c0 = (int)(run % a.groups) * a.cg;
    const float *part = a.part + n * a.nparts * 2 * a.C + c0;
    const int64_t items = a.nparts * a.cg;
    const float inv = 1.f / ((float)a.L * (float)a.cg);
    float s = 0.f, t = 0.f;
    if (BWD) {
        for (int64_t e = threadIdx.x; e < items; e += GT) {
            const int c = (int)(e % a.cg);
            const float *p = part + e / a.cg * 2 * a.C + c;
            const float w = a.w ? a.w[c0 + c] : 1.f;
            t += p[0] * w;
            s += p[a.C] * w;
        }
        run_sum(s, t, 9, red);
        s *= inv;
        t *= inv;
    } else {
        const auto rows = [&](int64_t k) { return (float)(min((k + 1) * a.per, (int64_t)a.L) - k * a.per); };
        const float base = part[0];
        float none = 0.f;
        for (int64_t e = threadIdx.x; e < items; e += GT) {
            const int64_t k = e / a.cg;
            s += rows(k) * (part[k * 2 * a.C + e % a.cg] - base);
        }
        run_sum(s, none, 9, red);
        s = base + s * inv;
        for (int64_t e = threadIdx.x; e < items; e += GT) {
            const int64_t k = e / a.cg;
            const float *p = part + k * 2 * a.C + e % a.cg;
            const float d = p[0] - s;
            t += p[a.C] + rows(k) * d * d;
        }
        run_sum(t, none, 9, red);
        t = 1.f / sqrtf(t * inv + a.eps);
    }
    if (threadIdx.x == 0) {
        float *to = (BWD ? a.mean : a.stats) + 2 * run;
        to[0] = s;
        to[1] = t;
    }
}

// dweight and dbias: sums of `rows` rows of 2 C partial sums, in a fixed
// order and in 64 bits (there may be millions of rows); columns 32 `block`
// on, 16 threads to a column.
__device__ __forceinline__ void gn_wsum(const GnArgs &a, int64_t rows, int64_t block, double (&red)[GT])
{
    const int64_t e = block * 32 + (threadIdx.x & 31);
    double s = 0.0;
    if (e < 2 * (int64_t)a.C) {
#pragma unroll 8
        for (int64_t p = threadIdx.x >> 5; p < rows; p += GT / 32) s += (double)a.part[2 * p * a.C + e];
    }
    red[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x < 32 && e < 2 * (int64_t)a.C) {
        for (int k = 1; k < GT / 32; ++k) s += red[threadIdx.x + 32 * k];
        float *to = e < a.C ? a.dw : a.db;
        if (to) to[e < a.C ? e : e - a.C] = (float)s;
    }
}

__global__ __launch_bounds__(GT) void k_gn_wsum(GnArgs a, int64_t rows)
{
    __shared__ double red[GT];
    gn_wsum(a, rows, blockIdx.x, red);
}

// The joined runs, in `joins` blocks; the blocks after them, in the backward,
// add up dweight and dbias from the same partial sums.
template <bool BWD>
__global__ __launch_bounds__(GT) void k_gn_mid(GnArgs a, unsigned joins, int64_t rows)
{
    __shared__ float red[2][GT / 64];
    __shared__ double wide[GT];
    if (blockIdx.x >= joins) return gn_wsum(a, rows, blockIdx.x - joins, wide);
    for (int64_t run = blockIdx.x; run < a.N * a.groups; run += joins) gn_join<BWD>(a, run, red);
}

template <typename T, int VE, bool BWD>
__global__ __launch_bounds__(GT) void k_gn_apply(GnArgs a)
{
    const Cut<VE> p(a);
    if (!p.on) return;
    float w[VE], b[VE], mu[VE], rstd[VE], m1[VE], m2[VE];
    channels<VE>(w, a.w ? a.w + p.c : nullptr, 1.f, true);
    channels<VE>(b, a.b ? a.b + p.c : nullptr, 0.f, true);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        const int64_t run = 2 * (p.n * a.groups + (p.c + i) / a.cg);
        mu[i] = a.stats[run];
        rstd[i] = a.stats[run + 1];
        m1[i] = BWD ? a.mean[run] : 0.f;
        m2[i] = BWD ? a.mean[run + 1] : 0.f;
    }
#pragma unroll 2
    for (int l = p.l0 + p.r0; l < p.l1; l += p.rp) {
        const int64_t row = p.n * a.L + l;
        const Vec<T, VE> x = load<T, VE>(static_cast<const T *>(a.x) + row * a.ldx + p.c, true);
        Vec<T, VE> gt = {}, dy = {}, y, dg;
        if (a.gate) gt = load<T, VE>(static_cast<const T *>(a.gate) + row * a.ldg + p.c, true);
        if (BWD) dy = load<T, VE>(static_cast<const T *>(a.dy) + row * a.ldy + p.c, true);
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            if (BWD) {
                const GnGrad r = gn_grad(to_f(x.v[i]), mu[i], rstd[i], w[i], b[i], a.gate != nullptr, to_f(gt.v[i]),
                                         to_f(dy.v[i]), a.silu);
                y.v[i] = from_f<T>(rstd[i] * (r.dz * w[i] - m1[i] - r.xh * m2[i]));
                dg.v[i] = from_f<T>(r.dgate);
            } else {
                const float z = (to_f(x.v[i]) - mu[i]) * rstd[i] * w[i] + b[i];
                y.v[i] = from_f<T>(a.gate ? z * act(to_f(gt.v[i]), a.silu).f : act(z, a.silu).f);
            }
        }
        T *to = static_cast<T *>(BWD ? a.dx : a.y);
        if (to) *reinterpret_cast<Vec<T, VE> *>(to + row * a.C + p.c) = y;
        if (BWD && a.dgate) *reinterpret_cast<Vec<T, VE> *>(static_cast<T *>(a.dgate) + row * a.C + p.c) = dg;
    }
}

// Statistics of samples without rows.
__global__ void k_gn_zero(float *p, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * GT + threadIdx.x; i < n; i += (int64_t)gridDim.x * GT) p[i] = 0.f;
}

// ---- host side

struct GnPlan {
    bool held = false;
    int ve = 1, k = 1;
    int64_t blocks = 0;
    size_t mean = 0, total = 0;   // workspace: partial sums, then the runs' means
};

// Elements that every row of every tensor allows to be moved at once.
static int widest(const GnArgs &a, int dtype, int64_t run)
{
    const int64_t e = dtype_size(dtype);
    for (int ve = 16 / (int)e; ve > 1; ve /= 2) {
        if (e == 2 && ve == 4) continue;   // 16 bytes, 4 bytes or one at a time
        if (e == 4 && ve == 2) continue;
        bool fits = run % ve == 0 && a.C % ve == 0;
        for (const void *p : {a.x, a.gate, a.dy, (const void *)a.y, (const void *)a.dx, (const void *)a.dgate})
            fits = fits && !misaligned(p, (unsigned)(ve * e));
        fits = fits && a.ldx % ve == 0 && (!a.gate || a.ldg % ve == 0) && (!a.dy || a.ldy % ve == 0);
        if (fits) return ve;
    }
    return 1;
}

// Chooses the kernels and fills in the arguments that go with them.  The
// workspace does not depend on the pointers' alignment: sizes come from `ve`
// as given, and every `ve` of a shape needs no more than one at a time does.
static GnPlan plan_gn(GnArgs &a, bool bwd, int ve_run, int ve_row, int64_t esize, int cus)
{
    GnPlan P;
    const int64_t M = (int64_t)a.L * a.cg, pieces = M / ve_run;
    // A wave holds runs of up to 64 HELD pieces (1000 x 32 x 320 in 32 groups
    // took 26 us so, and 101 cut), beside its neighbours, so that they share
    // the lines they fetch.  One that takes a whole block is held only where
    // its rows fill lines: blocks of neighbouring runs sit on different dies,
    // and each would fetch the others' part of a line (64 x 1024 x 512 in 32
    // groups took 106 us so, and 51 cut).
    P.held = pieces <= 64 * HELD || (pieces <= (int64_t)GT * HELD && (a.L == 1 || a.cg * esize >= 256));
    if (P.held) {
        // One piece to a thread while a wave's lanes suffice: the backward of
        // 5001 x 1536 took 25 us so, and 37 with two (more registers, fewer
        // waves); the forward took the same.
        a.pieces = (int)pieces;
        a.ppr = a.cg / ve_run;
        int lw = 0;
        while (lw < 6 && (int64_t(1) << lw) < pieces) ++lw;
        if ((int64_t(HELD) << lw) < pieces) lw = 9;
        const int64_t k = (pieces + (1 << lw) - 1) >> lw;
        P.k = k <= 1 ? 1 : k <= 2 ? 2 : 4;
        a.lw = lw;
        const int slots = GT >> lw;
        a.gs = a.groups < slots ? a.groups : slots;
        a.rpb = slots / a.gs;
        a.sets = (a.groups + a.gs - 1) / a.gs;
        // Blocks go on from sample to sample with their weights, and the
        // backward's with their sums, of which each leaves a row: 8 and 2 for
        // each CU (the backward took 25 us so, 32 with 4 and 27 with 1).
        int64_t rows = (a.N + a.rpb - 1) / a.rpb;
        const int64_t most = ((bwd ? 2 : 8) * int64_t(cus) + a.sets - 1) / a.sets;
        if (rows > most) rows = most;
        P.blocks = rows * a.sets;
        a.nparts = rows;
        P.ve = ve_run;
        P.total = bwd ? (size_t)rows * 2 * a.C * sizeof(float) : 0;
        return P;
    }
    P.ve = ve_row;
    const int64_t tiles = (a.C / P.ve + GT - 1) / GT;
    int64_t parts = (2 * int64_t(cus) + a.N * tiles - 1) / (a.N * tiles);
    const int64_t most = (a.L + 15) / 16;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    a.per = (a.L + parts - 1) / parts;
    a.nparts = (a.L + a.per - 1) / a.per;
    P.blocks = a.N * a.nparts * tiles;   // parts and channel tiles of all samples
    P.mean = (size_t)(a.N * a.nparts) * 2 * a.C * sizeof(float);
    P.total = P.mean + (bwd ? (size_t)(a.N * a.groups) * 2 * sizeof(float) : 0);
    return P;
}

// The workspace for any alignment and type.
static size_t gn_workspace_of(const gn_shape &s, bool bwd, int cus)
{
    if (s.N == 0 || s.L == 0) return 0;
    size_t most = 0;
    for (int run : {8, 4, 2, 1})
        for (int row : {8, 4, 2, 1}) {
            if ((s.C / s.groups) % run != 0 || s.C % row != 0) continue;
            GnArgs a{};
            a.N = s.N;
            a.L = (int)s.L;
            a.C = (int)s.C;
            a.groups = (int)s.groups;
            a.cg = (int)(s.C / s.groups);
            for (int64_t e : {2, 4}) {
                const GnPlan P = plan_gn(a, bwd, run, row, e, cus);
                if (P.total > most) most = P.total;
            }
        }
    return most;
}

// Working that out takes microseconds, so a thread remembers its last shapes.
static size_t gn_workspace(const gn_shape &s, bool bwd)
{
    struct Known {
        gn_shape s{-1, 0, 0, 0};
        int cus = 0;
        size_t bytes = 0;
    };
    static thread_local Known known[2][8];
    const int cus = ssd::device_cus();
    Known &k = known[bwd][(s.N ^ s.L ^ s.C >> 3 ^ s.groups) & 7];
    if (k.s.N != s.N || k.s.L != s.L || k.s.C != s.C || k.s.groups != s.groups || k.cus != cus) {
        k.s = s;
        k.cus = cus;
        k.bytes = gn_workspace_of(s, bwd, cus);
    }
    return k.bytes;
}

static int gn_args(const gn_shape &s, int64_t ldx, int64_t ldg, int64_t ldy, GnArgs *a)
{
    *a = GnArgs{};
    if (ldx < 0 || ldg < 0 || ldy < 0 || ldx >= kMaxCount || ldg >= kMaxCount || ldy >= kMaxCount) return SSD_ERR_SHAPE;
    a->N = s.N;
    a->L = (int)s.L;
    a->C = (int)s.C;
    a->groups = (int)s.groups;
    a->cg = (int)(s.C / s.groups);
    a->ldx = ldx ? ldx : s.C;
    a->ldg = ldg ? ldg : s.C;
    a->ldy = ldy ? ldy : s.C;
    return SSD_OK;
}

// Runs BODY with constants VE and K for the plan's.
#define GN_DISPATCH(P, ...)                                                              \
    do {                                                                                  \
        constexpr int FULL = 16 / (int)sizeof(T), PART = sizeof(T) == 2 ? 2 : 1;           \
        if ((P).ve == FULL) { constexpr int VE = FULL; __VA_ARGS__; }                             \
        else if ((P).ve == PART) { constexpr int VE = PART; __VA_ARGS__; }                        \
        else { constexpr int VE = 1; __VA_ARGS__; }                                               \
    } while (0)
#define GN_DISPATCH_K(P, ...)                       \
    do {                                             \
        if ((P).k == 1) { constexpr int K = 1; __VA_ARGS__; } \
        else if ((P).k == 2) { constexpr int K = 2; __VA_ARGS__; } \
        else { constexpr int K = 4; __VA_ARGS__; }          \
    } while (0)

// `wanted`: dweight and dbias; the held backward leaves their last sums to
// k_gn_wsum.
template <typename T>
static void run_gn(GnArgs a, const GnPlan &P, bool bwd, bool wanted, hipStream_t st)
{
    const dim3 blk(GT);
    const int64_t runs = a.N * a.groups, most = max_blocks(GT) / 2;
    const unsigned joins = (unsigned)(runs < most ? runs : most), sums = (unsigned)((2 * a.C + 31) / 32);
    // all blocks, in as many launches as it takes
    const auto all = [&](auto kernel) {
        for (a.block0 = 0; a.block0 < P.blocks; a.block0 += most) {
            const int64_t left = P.blocks - a.block0;
            kernel<<<dim3((unsigned)(left < most ? left : most)), blk, 0, st>>>(a);
        }
    };
    GN_DISPATCH(P, {
        if (P.held) {
            GN_DISPATCH_K(P, {
                if (bwd)
                    all(k_gn_bwd_held<T, VE, K>);
                else
                    all(k_gn_fwd_held<T, VE, K>);
            });
            if (wanted) k_gn_wsum<<<dim3(sums), blk, 0, st>>>(a, a.nparts);
        } else if (bwd) {
            all(k_gn_sums<T, VE, true>);
            k_gn_mid<true><<<dim3(joins + (wanted ? sums : 0)), blk, 0, st>>>(a, joins, a.N * a.nparts);
            if (a.dx || a.dgate) all(k_gn_apply<T, VE, true>);
        } else {
            all(k_gn_sums<T, VE, false>);
            k_gn_mid<false><<<dim3(joins), blk, 0, st>>>(a, joins, 0);
            all(k_gn_apply<T, VE, false>);
        }
    });
}

}  // namespace layer

using namespace layer;

extern "C" size_t gn_fwd_workspace_size(const gn_shape *shape)
{
    return check_gn(shape, GN_ACT_NONE) != SSD_OK ? (size_t)-1 : gn_workspace(*shape, false);
}

extern "C" size_t gn_bwd_workspace_size(const gn_shape *shape)
{
    return check_gn(shape, GN_ACT_NONE) != SSD_OK ? (size_t)-1 : gn_workspace(*shape, true);
}

extern "C" int gn_fwd(const gn_shape *shape, int dtype, int act, float eps, const void *x, int64_t ld_x,
                      const float *weight, const float *bias, const void *gate, int64_t ld_gate, void *y,
                      float *stats, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = check_gn(shape, act);
    if (rc == SSD_OK) rc = check_dtype(dtype);
    if (rc != SSD_OK) return rc;
    const gn_shape &s = *shape;
    GnArgs a;
    rc = gn_args(s, ld_x, ld_gate, 0, &a);
    if (rc != SSD_OK) return rc;
    if (!(eps >= 0.f)) return SSD_ERR_SHAPE;
    if (s.N == 0) return SSD_OK;
    if (!stats || (s.L > 0 && (!x || !y))) return SSD_ERR_NULL;
    const unsigned e = dtype_size(dtype);
    if (misaligned(x, e) || misaligned(gate, e) || misaligned(y, e) || misaligned(weight, 4) || misaligned(bias, 4) ||
        misaligned(stats, 4))
        return SSD_ERR_ALIGN;
    const size_t need = gn_workspace(s, false);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (need > 0 && !workspace) return SSD_ERR_NULL;
    if (need > 0 && misaligned(workspace, 16)) return SSD_ERR_ALIGN;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (s.L == 0) {
        const int64_t n = 2 * s.N * s.groups;
        const int64_t blocks = (n + GT - 1) / GT, most = max_blocks(GT);
        k_gn_zero<<<dim3((unsigned)(blocks < most ? blocks : most)), dim3(GT), 0, st>>>(stats, n);
        return launch_status();
    }
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.gate = gate;
    a.y = y;
    a.stats = stats;
    a.eps = eps;
    a.silu = act == GN_ACT_SILU;
    a.part = static_cast<float *>(workspace);
    const GnPlan P = plan_gn(a, false, widest(a, dtype, a.cg), widest(a, dtype, a.C), dtype_size(dtype), ssd::device_cus());
    LAYER_DISPATCH(dtype, run_gn<T>(a, P, false, false, st));
    return launch_status();
}

extern "C" int gn_bwd(const gn_shape *shape, int dtype, int act, const void *x, int64_t ld_x, const float *weight,
                      const float *bias, const void *gate, int64_t ld_gate, const float *stats, const void *dy,
                      int64_t ld_dy, void *dx, float *dweight, float *dbias, void *dgate, void *workspace,
                      size_t workspace_bytes, void *stream)
{
    int rc = check_gn(shape, act);
    if (rc == SSD_OK) rc = check_dtype(dtype);
    if (rc != SSD_OK) return rc;
    const gn_shape &s = *shape;
    GnArgs a;
    rc = gn_args(s, ld_x, ld_gate, ld_dy, &a);
    if (rc != SSD_OK) return rc;
    if (dgate && !gate) return SSD_ERR_NULL;
    const bool work = s.N > 0 && s.L > 0;
    if (work && (!x || !dy || !stats)) return SSD_ERR_NULL;
    const unsigned e = dtype_size(dtype);
    if (misaligned(x, e) || misaligned(gate, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(dgate, e) ||
        misaligned(weight, 4) || misaligned(bias, 4) || misaligned(stats, 4) || misaligned(dweight, 4) ||
        misaligned(dbias, 4))
        return SSD_ERR_ALIGN;
    const size_t need = gn_workspace(s, true);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (need > 0 && !workspace) return SSD_ERR_NULL;
    if (need > 0 && misaligned(workspace, 16)) return SSD_ERR_ALIGN;
    hipStream_t st = static_cast<hipStream_t>(stream);
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.gate = gate;
    a.dy = dy;
    a.stats = const_cast<float *>(stats);
    a.dx = dx;
    a.dgate = dgate;
    a.dw = dweight;
    a.db = dbias;
    a.silu = act == GN_ACT_SILU;
    const bool wanted = dweight || dbias;
    a.part = static_cast<float *>(workspace);
    if (work) {
        const GnPlan P = plan_gn(a, true, widest(a, dtype, a.cg), widest(a, dtype, a.C), dtype_size(dtype), ssd::device_cus());
        a.mean = reinterpret_cast<float *>(static_cast<char *>(workspace) + P.mean);
        if (P.held && !wanted) a.part = nullptr;
        if (wanted || dx || dgate) LAYER_DISPATCH(dtype, run_gn<T>(a, P, true, wanted, st));
    } else if (wanted) {
        k_gn_wsum<<<dim3((unsigned)((2 * s.C + 31) / 32)), dim3(GT), 0, st>>>(a, 0);   // sums of nothing
    }
    return launch_status();
}
