// The gated delta rule in chunks: what its kernels share.
//
//   S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  y_t = S_t^T q_t,  a_t = e^{log_decay_t}
//
// With b_t the sum of a chunk's log decays up to row t, b_L its last value, S
// the state entering the chunk, D_ij = e^{b_i - b_j} for j <= i and 0 above,
// and M = K K^T o D below the diagonal,
//   U = T diag(beta) (V - diag(e^b) K S),   T = (I + diag(beta) M)^-1
//   Y = (Q K^T o D) U + diag(e^b) Q S
//   S <- e^{b_L} S + K^T diag(e^{b_L - b}) U.
//
// T is a unit lower triangular matrix that no state enters, so all chunks'
// are formed at once beforehand (k_delta_inverse).  It is formed as a
// substitution forms it, in float32: 16 x 16 diagonal blocks row by row, and
// the rest from T_iw = -T_ii sum_j A_ij T_jw, which no power of A enters (the
// powers of a matrix of near keys reach 10^17 in a chunk of 64, its inverse
// stays at 1).
#pragma once

#include "layer_tiles.h"

namespace layer {

struct DeltaArgs : PrefillArgs {
    const float *beta;
    int64_t beta_t;
    char *inv;      // the chunks' T, [chunk][H] images
};

// Chunk number of row `begin` + `at` of sequence n, for chunks of C rows.
// Sequence n's first chunk has number begin / C + n, so that there is one for
// every chunk without a count of them; some numbers have no chunk.
__device__ __forceinline__ int chunk_number(int n, int begin, int at, int C) { return begin / C + n + at / C; }

// ---- T and P as operands: the 16 x 32 pieces on and below the diagonal, in
// the order in which lanes read them.
//
// Piece (t, s) holds rows 16 t .. and columns 32 s ..: lane l has row l % 16
// and, with g = l / 16, columns 4 g .. 4 g + 3 and 16 + 4 g .. (the order in
// which accumulators of 16 rows each give a summed axis of 32).
template <typename L, int C>
struct Pieces {
    static constexpr int TT = C / 16, N = C == 64 ? 6 : 2;
    static constexpr int PARTS = sizeof(L) == 2 ? 3 : 1;
    static constexpr int UNITS = sizeof(L) == 2 ? 1 : 2;   // 16-byte units of a lane's 8 values
    static constexpr int BYTES = N * PARTS * UNITS * 1024;
    static __device__ __forceinline__ constexpr int at(int t, int s) { return t < 2 ? t : 2 * t - 2 + s; }
    // of T^T, whose pieces lie on and above the diagonal
    static __device__ __forceinline__ constexpr int above(int t, int s)
    {
        return C == 32 ? t : t < 2 ? 2 * t + s : 2 + t;
    }
};
// The lane's 8 values of part u of piece f in an image at `p`.
template <typename L, int C>
__device__ __forceinline__ Frag<L> piece(const char *p, int f, int u, int lane)
{
    typedef Pieces<L, C> P;
    Frag<L> r;
    char *to = reinterpret_cast<char *>(&r);
#pragma unroll
    for (int i = 0; i < P::UNITS; ++i)
        *reinterpret_cast<u32x4 *>(to + 16 * i) =
            *reinterpret_cast<const u32x4 *>(p + (((f * P::PARTS + u) * P::UNITS + i) * 64 + lane) * 16);
    return r;
}

// T of every chunk and head, its columns times beta, in pieces; with BACK also
// T^T, beta left out.  A wave has 16 rows of K.
//
// About 0.9 us of dependent steps for a chunk of 64: 15 of a substitution, in
// which a row's factors come by v_readlane from the accumulators of K K^T, and
// up to nine 16 x 16 x 16 products on fp32 MFMA.  K's tile is read from memory
// once for every head of a group (from L2, after the first).
template <typename E, int KP, int C, bool VEC, bool BACK>
__global__ __launch_bounds__(4 * C) void k_delta_inverse(DeltaArgs a)
{
    typedef typename std::conditional<std::is_same<E, bf16>::value, bf16, float>::type L;
    typedef Pieces<L, C> PC;
    constexpr int TT = C / 16, PT = 4 * C, KS = KP / 32;
    constexpr int LK = KP + (sizeof(L) == 2 ? 16 : 4), LA = C + 4;
    __shared__ __align__(16) L ks[C * LK];
    __shared__ __align__(16) float A[C * LA], X[C * LA], betas[C];
    __shared__ Decays<C> d;

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int h = blockIdx.x % a.H;
    int id = blockIdx.x / a.H;
    Place p;
    if (!find(a, id, p) || p.bad || p.rows <= 0) return;
    const int g = h / (a.H / a.G);
    {
        Tile<E, C, KP, PT> tk;
        tk.template load<VEC>(static_cast<const E *>(a.k) + p.begin * a.st.k_t + g * a.st.k_g, a.st.k_t, p.rows, a.dk,
                              tid);
        const int64_t row = p.begin + lane;
        const bool on = lane < p.rows;
        const float la = on ? a.la[(a.la_t ? row * a.la_t : 0) + h] : 0.f;
        if (w == 0) make_decays(d, la, lane);
        if (w == 1 && lane < C) betas[lane] = on ? a.beta[row * a.beta_t + h] : 0.f;
        tk.template store<LK>(ks, tid);
    }
    block_sync();
    // A = diag(beta) M, a tile at a time: lane holds rows 16 i + g4 .. + 3, column 16 j + l16
    const auto tile = [&](int i, int j) {
        f32x4 x = {};
#pragma unroll
        for (int s = 0; s < KS; ++s)
            x = mma(frag8(ks + (16 * i + l16) * LK + 32 * s + 2 * g4), frag8(ks + (16 * j + l16) * LK + 32 * s + 2 * g4),
                    x);
        const f32x4 ih = *reinterpret_cast<const f32x4 *>(d.hi + 16 * i + g4);
        const f32x4 il = *reinterpret_cast<const f32x4 *>(d.lo + 16 * i + g4);
        const f32x4 bt = *reinterpret_cast<const f32x4 *>(betas + 16 * i + g4);
        const float jh = d.hi[16 * j + l16], jl = d.lo[16 * j + l16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] *= bt[e] * __expf((ih[e] - jh) + (il[e] - jl));
            if (16 * j + l16 >= 16 * i + g4 + e) x[e] = 0.f;
        }
        return x;
    };
    {
        // the wave's diagonal block: lane's column of (I + A)^-1, row by row
        const f32x4 x = tile(w, w);
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float sum = i == l16 ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j)
                sum -= __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x[i & 3]), 16 * (i >> 2) + j)) * t[j];
            t[i] = sum;
        }
        if (lane < 16)
#pragma unroll
            for (int i = 0; i < 16; ++i) X[(16 * w + i) * LA + 16 * w + l16] = t[i];
    }
    constexpr int LOW = TT * (TT - 1) / 2;
    for (int u = w; u < LOW; u += TT) {
        const int i = 1 + (u > 0) + (u > 2), j = u - i * (i - 1) / 2;
        const f32x4 x = tile(i, j);
#pragma unroll
        for (int e = 0; e < 4; ++e) A[(16 * i + g4 + e) * LA + 16 * j + l16] = x[e];
    }
    block_sync();
    {
        // column block w: T_iw = -T_ii sum_j A_ij T_jw
        f32x4 t[TT];
        const auto product = [&](const float *m, const f32x4 &b, f32x4 c) {   // m: 16 x 16 of rows LA apart
            const f32x4 f = *reinterpret_cast<const f32x4 *>(m + l16 * LA + g4);
#pragma unroll
            for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(f[e], b[e], c, 0, 0, 0);
            return c;
        };
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (i < w) continue;
            if (i == w) {
#pragma unroll
                for (int e = 0; e < 4; ++e) t[i][e] = X[(16 * w + g4 + e) * LA + 16 * w + l16];
                continue;
            }
            f32x4 sum = {};
#pragma unroll
            for (int j = 0; j < i; ++j)
                if (j >= w) sum = product(A + 16 * i * LA + 16 * j, t[j], sum);
            t[i] = product(X + 16 * i * LA + 16 * i, -sum, f32x4{});
#pragma unroll
            for (int e = 0; e < 4; ++e) X[(16 * i + g4 + e) * LA + 16 * w + l16] = t[i][e];
        }
    }
    block_sync();
    char *out = a.inv + ((int64_t)id * a.H + h) * (BACK ? 2 : 1) * PC::BYTES;
    const auto put = [&](char *to, int f, const float (&x)[8]) {
        Frag<L> parts[PC::PARTS];
        split(parts, f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
#pragma unroll
        for (int u = 0; u < PC::PARTS; ++u)
#pragma unroll
            for (int i = 0; i < PC::UNITS; ++i)
                *reinterpret_cast<u32x4 *>(to + (((f * PC::PARTS + u) * PC::UNITS + i) * 64 + lane) * 16) =
                    *reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(&parts[u]) + 16 * i);
    };
    for (int f = w; f < PC::N; f += TT) {
        const int t = f < 2 ? f : 2 + (f - 2) / 2, s = f < 2 ? 0 : (f - 2) % 2;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int col = 32 * s + (e < 4 ? 0 : 16) + g4 + (e & 3);
            // above the diagonal X was not written
            x[e] = col >= 16 * (t + 1) ? 0.f : X[(16 * t + l16) * LA + col] * betas[col];
        }
        put(out, f, x);
    }
    if constexpr (BACK) {
        for (int f = w; f < PC::N; f += TT) {
            const int t = C == 32 ? f : f < 4 ? f / 2 : f - 2, s = C == 32 ? 0 : f < 4 ? f % 2 : 1;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 32 * s + (e < 4 ? 0 : 16) + g4 + (e & 3);
                x[e] = row < 16 * t ? 0.f : X[row * LA + 16 * t + l16];
            }
            put(out + PC::BYTES, f, x);
        }
    }
}

}  // namespace layer
