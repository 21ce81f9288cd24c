// Group norm, channels last, with an activation on the normalised value or
// on a gate, and its gradient.  For sample n and run of channels j, over
// M = L C / groups values:
//   mu = sum x / M,  rstd = (sum (x - mu)^2 / M + eps)^(-1/2),
//   xh = (x - mu) rstd,  z = xh weight + bias,  y = act(z) or z act(gate).
// With dz = dy act'(z) or dy act(gate), and d = dz weight:
//   dx = rstd (d - mean(d) - xh mean(d xh)),
//   dgate = dy z act'(gate),  dweight = sum dz xh,  dbias = sum dz.
// act is SiLU: act(u) = u s, act'(u) = s (1 + u (1 - s)), s = 1 / (1 + e^-u).
#include "layer_device.h"

namespace layer {

constexpr int GT = 256;   // threads of a block

struct GnArgs {
    const void *x, *gate, *dy;
    const float *w, *b;
    void *y, *dx, *dgate;
    float *stats, *dw, *db, *part;
    int64_t N, ldx, ldg, ldy, nparts;
    int L, C, groups, cg;
    float eps;
};

__device__ __forceinline__ float sigmoid(float u) { return 1.f / (1.f + expf(-u)); }

// Sum over the block, in every thread.
__device__ __forceinline__ float block_sum(float x, float *red)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < GT / 64; ++w) s += red[w];
    return s;
}

// One block for a sample's run of channels.
template <typename T>
__global__ __launch_bounds__(GT) void k_gn_fwd(GnArgs a, bool silu)
{
    __shared__ float red[GT / 64];
    const int64_t n = blockIdx.x / a.groups;
    const int c0 = (int)(blockIdx.x % a.groups) * a.cg;
    const int64_t M = (int64_t)a.L * a.cg;
    const T *x = static_cast<const T *>(a.x) + n * a.L * a.ldx + c0;
    const auto each = [&](auto f) {
        for (int64_t e = threadIdx.x; e < M; e += GT) f(e / a.cg, (int)(e % a.cg));
    };
    float s = 0.f;
    each([&](int64_t l, int c) { s += to_f(x[l * a.ldx + c]); });
    const float mu = block_sum(s, red) / (float)M;
    s = 0.f;
    each([&](int64_t l, int c) {
        const float d = to_f(x[l * a.ldx + c]) - mu;
        s += d * d;
    });
    const float rstd = 1.f / sqrtf(block_sum(s, red) / (float)M + a.eps);
    if (threadIdx.x == 0) {
        a.stats[2 * blockIdx.x] = mu;
        a.stats[2 * blockIdx.x + 1] = rstd;
    }
    T *y = static_cast<T *>(a.y) + n * a.L * a.C + c0;
    const T *gate = a.gate ? static_cast<const T *>(a.gate) + n * a.L * a.ldg + c0 : nullptr;
    each([&](int64_t l, int c) {
        const float z = (to_f(x[l * a.ldx + c]) - mu) * rstd * (a.w ? a.w[c0 + c] : 1.f) + (a.b ? a.b[c0 + c] : 0.f);
        const float u = gate ? to_f(gate[l * a.ldg + c]) : z;
        const float act = silu ? u * sigmoid(u) : u;
        y[l * a.C + c] = from_f<T>(gate ? z * act : act);
    });
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
    const float z = r.xh * w + b, u = gated ? gate : z;
    const float s = silu ? sigmoid(u) : 1.f;
    const float d = silu ? s * (1.f + u * (1.f - s)) : 1.f;
    r.dz = gated ? dy * (u * s) : dy * d;
    r.dgate = dy * z * d;
    return r;
}

template <typename T>
__global__ __launch_bounds__(GT) void k_gn_bwd(GnArgs a, bool silu)
{
    __shared__ float red[GT / 64];
    const int64_t n = blockIdx.x / a.groups;
    const int c0 = (int)(blockIdx.x % a.groups) * a.cg;
    const int64_t M = (int64_t)a.L * a.cg;
    const T *x = static_cast<const T *>(a.x) + n * a.L * a.ldx + c0;
    const T *dy = static_cast<const T *>(a.dy) + n * a.L * a.ldy + c0;
    const T *gate = a.gate ? static_cast<const T *>(a.gate) + n * a.L * a.ldg + c0 : nullptr;
    const float mu = a.stats[2 * blockIdx.x], rstd = a.stats[2 * blockIdx.x + 1];
    const auto each = [&](auto f) {
        for (int64_t e = threadIdx.x; e < M; e += GT) {
            const int64_t l = e / a.cg;
            const int c = (int)(e % a.cg);
            const float w = a.w ? a.w[c0 + c] : 1.f;
            f(l, c, w, gn_grad(to_f(x[l * a.ldx + c]), mu, rstd, w, a.b ? a.b[c0 + c] : 0.f, gate != nullptr,
                               gate ? to_f(gate[l * a.ldg + c]) : 0.f, to_f(dy[l * a.ldy + c]), silu));
        }
    };
    float s1 = 0.f, s2 = 0.f;
    each([&](int64_t, int, float w, const GnGrad &r) {
        s1 += r.dz * w;
        s2 += r.dz * w * r.xh;
    });
    const float m1 = block_sum(s1, red) / (float)M, m2 = block_sum(s2, red) / (float)M;
    T *dx = a.dx ? static_cast<T *>(a.dx) + n * a.L * a.C + c0 : nullptr;
    T *dg = a.dgate ? static_cast<T *>(a.dgate) + n * a.L * a.C + c0 : nullptr;
    each([&](int64_t l, int c, float w, const GnGrad &r) {
        if (dx) dx[l * a.C + c] = from_f<T>(rstd * (r.dz * w - m1 - r.xh * m2));
        if (dg) dg[l * a.C + c] = from_f<T>(r.dgate);
    });
}

// Partial sums of dweight and dbias: 64 channels, every nparts-th row.
template <typename T>
__global__ __launch_bounds__(GT) void k_gn_wpart(GnArgs a, bool silu)
{
    __shared__ float red[2][GT];
    const int c = blockIdx.x * 64 + (threadIdx.x & 63);
    float sw = 0.f, sb = 0.f;
    if (c < a.C) {
        const float w = a.w ? a.w[c] : 1.f, b = a.b ? a.b[c] : 0.f;
        for (int64_t r = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); r < a.N * a.L; r += 4 * a.nparts) {
            const float *st = a.stats + 2 * (r / a.L * a.groups + c / a.cg);
            const GnGrad t =
                gn_grad(to_f(static_cast<const T *>(a.x)[r * a.ldx + c]), st[0], st[1], w, b, a.gate != nullptr,
                        a.gate ? to_f(static_cast<const T *>(a.gate)[r * a.ldg + c]) : 0.f,
                        to_f(static_cast<const T *>(a.dy)[r * a.ldy + c]), silu);
            sw += t.dz * t.xh;
            sb += t.dz;
        }
    }
    red[0][threadIdx.x] = sw;
    red[1][threadIdx.x] = sb;
    __syncthreads();
    if (threadIdx.x < 64 && c < a.C) {
        for (int k = 1; k < 4; ++k) {
            sw += red[0][threadIdx.x + 64 * k];
            sb += red[1][threadIdx.x + 64 * k];
        }
        a.part[(2 * (int64_t)blockIdx.y) * a.C + c] = sw;
        a.part[(2 * (int64_t)blockIdx.y + 1) * a.C + c] = sb;
    }
}

__global__ __launch_bounds__(GT) void k_gn_wsum(GnArgs a)
{
    const int64_t e = (int64_t)blockIdx.x * GT + threadIdx.x;
    if (e >= 2 * (int64_t)a.C) return;
    float s = 0.f;
    for (int64_t p = 0; p < a.nparts; ++p) s += a.part[2 * p * a.C + e];
    float *to = e < a.C ? a.dw : a.db;
    if (to) to[e < a.C ? e : e - a.C] = s;
}

// Statistics of samples without rows.
__global__ void k_gn_zero(float *p, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * GT + threadIdx.x;
    if (i < n) p[i] = 0.f;
}

static int64_t wparts(const gn_shape &s)
{
    const int64_t rows = s.N * s.L;
    return rows < 1 ? 0 : (rows + 63) / 64 > 64 ? 64 : (rows + 63) / 64;
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
    if (s.N > ((int64_t(1) << 31) - 1) / s.groups) return SSD_ERR_SHAPE;
    return SSD_OK;
}

}  // namespace layer

using namespace layer;

extern "C" size_t gn_fwd_workspace_size(const gn_shape *shape)
{
    if (check_gn(shape, GN_ACT_NONE) != SSD_OK) return (size_t)-1;
    return 0;
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
    (void)workspace;
    (void)workspace_bytes;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (s.L == 0) {
        const int64_t n = 2 * s.N * s.groups;
        k_gn_zero<<<dim3((unsigned)((n + GT - 1) / GT)), dim3(GT), 0, st>>>(stats, n);
        return launch_status();
    }
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.gate = gate;
    a.y = y;
    a.stats = stats;
    a.eps = eps;
    const bool silu = act == GN_ACT_SILU;
    LAYER_DISPATCH(dtype, (k_gn_fwd<T><<<dim3((unsigned)(s.N * s.groups)), dim3(GT), 0, st>>>(a, silu)));
    return launch_status();
}

extern "C" size_t gn_bwd_workspace_size(const gn_shape *shape)
{
    if (check_gn(shape, GN_ACT_NONE) != SSD_OK) return (size_t)-1;
    return (size_t)wparts(*shape) * 2 * (size_t)shape->C * sizeof(float);
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
    const bool wanted = dweight || dbias;
    const size_t need = wanted ? gn_bwd_workspace_size(shape) : 0;
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
    a.part = static_cast<float *>(workspace);
    a.nparts = work ? wparts(s) : 0;
    const bool silu = act == GN_ACT_SILU;
    if (work && (dx || dgate))
        LAYER_DISPATCH(dtype, (k_gn_bwd<T><<<dim3((unsigned)(s.N * s.groups)), dim3(GT), 0, st>>>(a, silu)));
    if (wanted) {
        if (work)
            LAYER_DISPATCH(dtype, (k_gn_wpart<T><<<dim3((unsigned)((s.C + 63) / 64), (unsigned)a.nparts), dim3(GT), 0,
                                                  st>>>(a, silu)));
        k_gn_wsum<<<dim3((unsigned)((2 * s.C + GT - 1) / GT)), dim3(GT), 0, st>>>(a);
    }
    return launch_status();
}
