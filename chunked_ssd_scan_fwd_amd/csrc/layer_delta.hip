// The gated delta rule over a packed batch and a pool of states, in chunks.
#include "layer_delta.h"

namespace layer {

// One segment of a sequence for one head and VT columns, with the state in the
// registers of VT / 16 waves, 16 columns each, which make U and Y.  Neither S
// nor U crosses waves: K S comes out of the accumulators as the operand that T
// takes, and U as the one that P and K^T take.
//
// Four more waves make what the next chunk needs, in two steps with a barrier
// between them, while the first ones work on this chunk: two have 16 rows of T
// each, two fetch and make the decays and P.
//   K S and Q S  | T's blocks joined (solve), the next A (products) | P to LDS, q and v, loads
//   U, P U, S    | inverses of the diagonal's blocks (inverse)     | P, decays, k
// k comes a step earlier than q and v where LDS holds three tiles of it, for in
// the second step A's products made T's waves the last by 1300 cycles of 5800
// (512 rows, 8 heads: 43 us so, and 39.5).
// T in a kernel of its own beforehand cost 460 us beside the large batch's 721
// (16 prompts of 8192 rows, 16 heads of 128), and 18 KB of memory a chunk and
// head; so the batch takes 909 us.  There a chunk takes a CU 6930 cycles, of
// which a SIMD has vector instructions under way in 0.56 (S in parts is anew for
// every chunk) and matrix ones in 0.40: little is left to fill.
//
// Chunks of 64 rows, whose S is split half as often, took as long (935): P and
// T have twice the products for a row then, and four waves that both fetch and
// have rows of T.  They made a prompt of 77 rows 20 us for 17.  Eight waves of 16
// columns beside four others took 721 us (64 rows, T beforehand) where four of
// 32 columns and four took 808: one wave's matrix products run beside another's
// vector instructions.
//
// For bfloat16 inputs everything that reaches the state keeps float32's
// accuracy: S, T, the residual V - diag(e^b) K S and U enter their products as
// sums of three bfloat16 numbers (six products for two such operands, the ones
// of 2^-24 and less left out).  In y the scores P, S and U enter as sums of
// two, 2^-18 of each term off, where y's own rounding is 2^-9 of their sum: 3 in
// 1000 values of y round to the neighbour.  Three parts left 2 in 10000 and took
// 6% more time (16 prompts of 8192 rows, 16 heads of 128: 970 us for 909); P as
// one part made y 0.0018 to 0.0023 from 64 bits, and its rounding alone is
// 0.00165.
constexpr int C = 32;   // rows of a chunk

template <typename E, int KP, int VT>
struct DeltaLds {
    typedef typename std::conditional<std::is_same<E, bf16>::value, bf16, float>::type L;
    typedef Pieces<L> PC;
    static constexpr int PAD = sizeof(L) == 2 ? 16 : 4;
    static constexpr int LK = KP + PAD, LV = VT + PAD;
    static constexpr int YU = PC::PARTS == 3 ? 2 : 1;   // parts of what y is made of: P, S and U
    static constexpr int PBYTES = PC::BYTES / PC::PARTS * YU;
    // k a step earlier than q and v, where a third tile of it fits
    static constexpr bool EARLY = KP <= 128 || sizeof(L) == 2;
    static constexpr int KB = EARLY ? 3 : 2;
    L q[2][C * LK], k[KB][C * LK], v[2][C * LV];
    alignas(16) char p[PBYTES], t[PC::BYTES];
    // the next chunk's diagonal blocks of T, and A's tile below, by lanes
    alignas(16) f32x4 diag[2][64], low[EARLY ? 2 : 1][64];
    Decays<C> dec[3];
    alignas(16) float beta[3][C];
};

// f b + x of 16 x 16 matrices: lanes hold rows 4 g .. of column l % 16 of f^T, b and x.
__device__ __forceinline__ f32x4 times(f32x4 f, f32x4 b, f32x4 x)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_16x16x4f32(f[e], b[e], x, 0, 0, 0);
    return x;
}

// Row N of 16 lanes in place of all four.
template <int N>
__device__ __forceinline__ float row_of_lanes(float x)
{
    // rows 0, 0, 2, 2 and 1, 1, 3, 3; then one half of them twice
    const unsigned u = __float_as_uint(x);
    const auto pairs = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const auto halves = __builtin_amdgcn_permlane32_swap(pairs[N & 1], pairs[N & 1], false, false);
    return __uint_as_float(halves[N >> 1]);
}

// Two blocks of eight waves leave a wave 128 registers; with q's, k's and v's
// tiles on their way the 64-column kernel for dk over 64 spills 18 of them.
template <typename E, int KP, int VT>
struct DeltaPerCu {
    static constexpr int n = VT == 64 && KP <= 128 && std::is_same<E, bf16>::value ? 2 : 1;
    // waves that hold S, and four more: two that fetch and two with 16 rows of T each
    static constexpr int waves = VT / 16, movers = 2;
    static constexpr int threads = 64 * (waves + 4), per_simd = n * threads / 256;
};

// OUT: y and the last state, from the state that enters the segment.  Otherwise
// the map from the state that enters it to the one that leaves it, S' = M S + B:
// B as the state that the segment makes from zero, and further blocks for the
// columns of M, which is what it makes of the identity with v = 0.
template <typename E, int KP, int VT, bool OUT, bool VEC>
__global__ __launch_bounds__((DeltaPerCu<E, KP, VT>::threads))
__attribute__((amdgpu_waves_per_eu(DeltaPerCu<E, KP, VT>::per_simd, DeltaPerCu<E, KP, VT>::per_simd))) void k_delta_chunks(DeltaArgs a)
{
    typedef DeltaLds<E, KP, VT> Lds;
    typedef typename Lds::L L;
    typedef Pieces<L> PC;
    constexpr int LK = Lds::LK, LV = Lds::LV, KB = Lds::KB;
    constexpr bool EARLY = Lds::EARLY;
    constexpr int WAVES = DeltaPerCu<E, KP, VT>::waves, MT = KP / 16, KS = KP / 32;
    constexpr int PARTS = PC::PARTS, YU = Lds::YU;
    constexpr int MOVERS = DeltaPerCu<E, KP, VT>::movers, PT = 64 * MOVERS;   // threads that fetch
    __shared__ __align__(16) Lds lds;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int tiles = OUT ? a.tiles : a.tiles + a.map_tiles;
    const int tile = blockIdx.x % tiles, h = blockIdx.x / tiles % a.H;
    int id = blockIdx.x / (tiles * a.H);
    Place p;
    if (!find(a, id, p)) return;
    if (!OUT && (p.s + 1 >= p.segs || p.bad)) return;   // nothing follows the last segment
    const bool map = !OUT && tile >= a.tiles;
    const int width = map ? a.map_cols : a.dv;
    const int g = h / (a.H / a.G), c0 = (map ? tile - a.tiles : tile) * VT, cols = min(VT, width - c0);
    E *y = static_cast<E *>(a.y) + p.begin * a.st.y_t + h * a.st.y_h + c0;
    if (OUT && p.bad) {
        for (int64_t e = threadIdx.x; e < (int64_t)p.rows * VT; e += DeltaPerCu<E, KP, VT>::threads)
            if (e % VT < cols) y[e / VT * a.st.y_t + e % VT] = from_f<E>(__builtin_nanf(""));
        return;
    }
    const int chunks = (p.rows + C - 1) / C;
    const E *q = static_cast<const E *>(a.q) + p.begin * a.st.q_t + g * a.st.q_g;
    const E *k = static_cast<const E *>(a.k) + p.begin * a.st.k_t + g * a.st.k_g;
    const E *v = static_cast<const E *>(a.v) + p.begin * a.st.v_t + h * a.st.v_h + (map ? 0 : c0);
    const float *la = a.la + (a.la_t ? p.begin * a.la_t : 0) + h;

    // half j of a lane's 8 values of part u of piece `row`
    typedef typename std::conditional<sizeof(L) == 2, bf16x4, f32x4>::type L4;
    const auto put = [&](char *to, int parts, int row, int j, int u, L4 x) {
        const int f = row * parts + u;
        *reinterpret_cast<L4 *>(to + (f * PC::UNITS * 64 + lane) * 16 + j * (PC::UNITS == 2 ? 1024 : 8)) = x;
    };

    // A tile of P, 16 x 16, on or below the diagonal.  Formed as K Q^T, so that a
    // lane holds 4 scores of one query.
    const auto scores = [&](const Decays<C> &d, const L *qs, const L *ks, int it, int jt, int lane) {
        const int l16 = lane & 15, g4 = (lane >> 4) * 4;
        f32x4 x = {};
#pragma unroll
        for (int s = 0; s < KS; ++s)
            x = mma(frag8(ks + (16 * jt + l16) * LK + 32 * s + 2 * g4), frag8(qs + (16 * it + l16) * LK + 32 * s + 2 * g4),
                    x);
        const int i = 16 * it + l16, j = 16 * jt + g4;
        const float bh = d.hi[i], bl = d.lo[i];
        const f32x4 jh = *reinterpret_cast<const f32x4 *>(d.hi + j), jl = *reinterpret_cast<const f32x4 *>(d.lo + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] *= __expf((bh - jh[e]) + (bl - jl[e]));
            if (j + e > i) x[e] = 0.f;
        }
        return x;
    };
    const auto put_scores = [&](int it, int jt, f32x4 x) {
        L4 parts[YU];
        split4(parts, x);
#pragma unroll
        for (int u = 0; u < YU; ++u) put(lds.p, YU, it, jt, u, parts[u]);
    };

    if (wave >= WAVES) {
        // ---- fetches, and T of the next chunk
        const int w = (wave - WAVES) & 1;
        const bool mover = wave < WAVES + MOVERS;
        Tile<E, C, KP, PT> tq, tk;
        Tile<E, C, VT, PT> tv;
        // Of a chunk past the last one nothing is loaded, and the zeros that it
        // leaves are not read.
        const auto load_k = [&](int c) {
            const int t0 = c * C, rows = p.rows - t0, tid = anew(threadIdx.x - 64 * WAVES);
            tk.template fetch<VEC>(k + t0 * a.st.k_t, a.st.k_t, min(C, rows), a.dk, tid);
        };
        const auto store_k = [&](int c) {
            const int tid = anew(threadIdx.x - 64 * WAVES);
            tk.template place<VEC, LK>(lds.k[c % KB], k + c * C * a.st.k_t, a.st.k_t, a.dk, tid);
        };
        const auto load = [&](int c) {
            const int t0 = c * C, rows = p.rows - t0, tid = anew(threadIdx.x - 64 * WAVES);
            if (OUT) tq.template fetch<VEC>(q + t0 * a.st.q_t, a.st.q_t, min(C, rows), a.dk, tid);
            tv.template fetch<VEC>(v + t0 * a.st.v_t, a.st.v_t, map ? 0 : min(C, rows), cols, tid);
        };
        const auto store = [&](int c) {
            const int b = c & 1, tid = anew(threadIdx.x - 64 * WAVES);
            if (OUT) tq.template place<VEC, LK>(lds.q[b], q + c * C * a.st.q_t, a.st.q_t, a.dk, tid);
            tv.template place<VEC, LV>(lds.v[b], v + c * C * a.st.v_t, a.st.v_t, cols, tid);
        };
        const float *beta = a.beta + p.begin * a.beta_t + h;
        // a row's log decay (wave 0) or beta (wave 1), and what chunk c makes of them
        const auto row_value = [&](int c) {
            const int t = c * C + lane;
            const bool on = w < 2 && lane < C && t < p.rows;
            return on ? (w == 0 ? la[t * a.la_t] : beta[t * a.beta_t]) : 0.f;
        };
        const auto row_values = [&](int c, float x) {
            if (w == 0) make_decays(lds.dec[c % 3], x, lane);
            if (w == 1 && lane < C) lds.beta[c % 3][lane] = x;
        };
        // T in three steps, a row block of 16 to a wave.  First the diagonal
        // blocks of A = diag(beta) M, and the tile left of the second.
        f32x4 m;
        const auto products = [&](int c) {
            const int lane = anew(threadIdx.x & 63), l16 = lane & 15, g4 = (lane >> 4) * 4;
            const L *ks = lds.k[c % KB];
            const Decays<C> &d = lds.dec[c % 3];
            const float *betas = lds.beta[c % 3];
            Frag<L> fk[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) fk[s] = frag8(ks + (16 * w + l16) * LK + 32 * s + 2 * g4);
            // times beta and the decays: rows of block i, columns of block j
            const auto scaled = [&](f32x4 x, int i, int j) {
                const f32x4 ih = *reinterpret_cast<const f32x4 *>(d.hi + 16 * i + g4);
                const f32x4 il = *reinterpret_cast<const f32x4 *>(d.lo + 16 * i + g4);
                const f32x4 bt = *reinterpret_cast<const f32x4 *>(betas + 16 * i + g4);
                const float jh = d.hi[16 * j + l16], jl = d.lo[16 * j + l16];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= bt[e] * __expf((ih[e] - jh) + (il[e] - jl));
                return x;
            };
            m = f32x4{};
#pragma unroll
            for (int s = 0; s < KS; ++s) m = mma(fk[s], fk[s], m);
            m = scaled(m, w, w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (l16 >= g4 + e) m[e] = 0.f;
            if (w == 0) {   // the other wave's part of `solve` is the longer
                f32x4 x = {};
#pragma unroll
                for (int s = 0; s < KS; ++s) x = mma(frag8(ks + (16 + l16) * LK + 32 * s + 2 * g4), fk[s], x);
                lds.low[EARLY ? c & 1 : 0][lane] = scaled(x, 1, 0);
            }
        };
        // Then the diagonal block's inverse X by substitution: a lane holds rows
        // 4 g .. 4 g + 3 of column l % 16, so four rows at a time, which the
        // lanes of the others then take off theirs.
        const auto inverse = [&]() {
            const int lane = anew(threadIdx.x & 63), l16 = lane & 15, g4 = (lane >> 4) * 4;
            f32x4 X;
#pragma unroll
            for (int e = 0; e < 4; ++e) X[e] = l16 == g4 + e ? 1.f : 0.f;
            const auto rows4 = [&](auto which) {
                constexpr int n = decltype(which)::value;
                const auto column = [&](int e, auto j) {   // A(g4 + e, 4 n + j)
                    constexpr int ctrl = 0x150 + 4 * n + decltype(j)::value;   // row_newbcast
                    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(m[e]), ctrl, 0xf, 0xf, true));
                };
                const ssd::IntC<0> j0;
                const ssd::IntC<1> j1;
                const ssd::IntC<2> j2;
                const ssd::IntC<3> j3;
                f32x4 y = X;
                y[1] -= column(1, j0) * y[0];
                y[2] -= column(2, j0) * y[0];
                y[3] -= column(3, j0) * y[0];
                y[2] -= column(2, j1) * y[1];
                y[3] -= column(3, j1) * y[1];
                y[3] -= column(3, j2) * y[2];
                if (g4 == 4 * n) X = y;
                if constexpr (n < 3) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = row_of_lanes<n>(y[e]);
                    f32x4 x = X;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] -= column(e, j0) * y[0];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] -= column(e, j1) * y[1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] -= column(e, j2) * y[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] -= column(e, j3) * y[3];
                    if (g4 > 4 * n) X = x;
                }
            };
            rows4(ssd::IntC<0>{});
            rows4(ssd::IntC<1>{});
            rows4(ssd::IntC<2>{});
            rows4(ssd::IntC<3>{});
            lds.diag[w][lane] = X;
        };
        // At last T_10 = -T_11 A_10 T_00.  Held transposed, so that T_11 A_10 comes
        // out of the accumulators as the next product's operand, and T's rows as
        // its pieces hold them.
        const auto put_t = [&](int row, int j, f32x4 x) {
            L4 parts[PARTS];
            split4(parts, x);
#pragma unroll
            for (int u = 0; u < PARTS; ++u) put(lds.t, PARTS, row, j, u, parts[u]);
        };
        const auto solve = [&](int c) {
            const int lane = anew(threadIdx.x & 63), l16 = lane & 15, g4 = (lane >> 4) * 4;
            const float *betas = lds.beta[c % 3];
            const float *x = reinterpret_cast<const float *>(lds.diag[w]) + 64 * (l16 >> 2) + (l16 & 3);
            f32x4 T;
#pragma unroll
            for (int e = 0; e < 4; ++e) T[e] = x[4 * (g4 + e)];
            if (w == 1) {
                const f32x4 sum = times(lds.low[EARLY ? c & 1 : 0][lane], T, f32x4{});
                put_t(1, 0, times(lds.diag[0][lane], -sum, f32x4{}) * *reinterpret_cast<const f32x4 *>(betas + g4));
            }
            put_t(w, w, T * *reinterpret_cast<const f32x4 *>(betas + 16 * w + g4));
        };
        // what a piece on the diagonal holds above it stays 0
        if (w == 0 && !mover) {
            put_scores(0, 1, f32x4{});
            put_t(0, 1, f32x4{});
        }
        if (mover) {   // the decays and P are its own too: wave 0 has P's tile (1, 0), wave 1 those on the diagonal
            f32x4 P0 = {}, P1 = {};
            const auto make_scores = [&](int c) {
                if (!OUT) return;
                const int lane = anew(threadIdx.x & 63), b = c & 1;
                P0 = scores(lds.dec[c % 3], lds.q[b], lds.k[c % KB], 1, w, lane);
                if (w == 1) P1 = scores(lds.dec[c % 3], lds.q[b], lds.k[c % KB], 0, 0, lane);
            };
            const auto write_scores = [&]() {
                if (!OUT) return;
                put_scores(1, w, P0);
                if (w == 1) put_scores(0, 0, P1);
            };
            row_values(0, row_value(0));
            float next = row_value(1);
            load_k(0);
            load(0);
            store_k(0);
            store(0);
            load_k(1);
            load(1);
            block_sync();
            make_scores(0);
            row_values(1, next);
            if (EARLY) {
                store_k(1);
                load_k(2);
            }
            block_sync();
            for (int c = 0; c < chunks; ++c) {
                next = row_value(c + 2);
                write_scores();
                if (!EARLY) {
                    store_k(c + 1);
                    load_k(c + 2);
                }
                store(c + 1);
                load(c + 2);
                block_sync();
                make_scores(c + 1);
                row_values(c + 2, next);
                if (EARLY) {
                    store_k(c + 2);
                    load_k(c + 3);
                }
                block_sync();
            }
        } else {
            block_sync();
            products(0);
            inverse();
            block_sync();
            for (int c = 0; c < chunks; ++c) {
                solve(c);
                if (EARLY) products(c + 1);
                block_sync();
                if (!EARLY) products(c + 1);
                inverse();
                block_sync();
            }
        }
        return;
    }

    // ---- states and outputs
    const int64_t state = (int64_t)a.dk * width;
    float *pool = p.slot < 0 ? nullptr : a.states + ((int64_t)p.slot * a.H + h) * state;
    float *ends = (map ? a.maps : a.ends) + ((int64_t)id * a.H + h) * state;
    const int w0 = 16 * wave;   // this wave's columns of the tile

    // S: value i of accumulator m is row 32 (m / 2) + 2 g4 + 4 (m % 2) + i, column
    // w0 + l16.  The registers hold S / scale: the chunks' decays gather in `scale`,
    // until it leaves 2^-16 .. 2^16.
    f32x4 S[MT];
    float scale = 1.f;
    const auto state_at = [&](int m, int i, int lane) {
        const int col = w0 + (lane & 15);
        const uint32_t base = col < cols ? (uint32_t)((lane >> 4) * 8 * width + c0 + col) * 4u : kOOB;
        return base + (uint32_t)(32 * (m / 2) + 4 * (m % 2) + i) * (uint32_t)width * 4u;
    };
    {
        const float *from = !OUT ? nullptr : p.segs > 1 ? ends : p.carry ? pool : nullptr;
        const rsrc_t r = make_rsrc(from, from ? state * 4 : 0);   // zeros where nothing enters
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                S[m][i] = OUT ? ssd::gload1(r, state_at(m, i, lane)) : 0.f;
                if (map && 32 * (m / 2) + 2 * g4 + 4 * (m % 2) + i == c0 + w0 + l16) S[m][i] = 1.f;
            }
    }
    block_sync();
    block_sync();
    for (int c = 0; c < chunks; ++c) {
        const int b = c & 1, rows = min(C, p.rows - c * C);
        const Decays<C> &d = lds.dec[c % 3];
        const L *qs = lds.q[b], *ks = lds.k[c % KB], *vs = lds.v[b];
        // X = K S (rows: the chunk's, columns: of v), Y^T = S^T Q^T
        f32x4 X[2], Y[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) X[t] = Y[t] = f32x4{};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            Frag<L> fs[PARTS];
            split(fs, S[2 * s], S[2 * s + 1]);
            Frag<L> f[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) f[t] = frag8(ks + (16 * t + l16) * LK + 32 * s + 2 * g4);
#pragma unroll
            for (int u = PARTS - 1; u >= 0; --u)
#pragma unroll
                for (int t = 0; t < 2; ++t) X[t] = mma(f[t], fs[u], X[t]);
            if (!OUT) continue;
#pragma unroll
            for (int t = 0; t < 2; ++t) f[t] = frag8(qs + (16 * t + l16) * LK + 32 * s + 2 * g4);
#pragma unroll
            for (int u = YU - 1; u >= 0; --u)
#pragma unroll
                for (int t = 0; t < 2; ++t) Y[t] = mma(fs[u], f[t], Y[t]);
        }
        block_sync();   // P and T are there
        // U = (T diag(beta)) (V - diag(e^b) K S)
        f32x4 U[2];
        {
            Frag<L> fg[PARTS];
            const f32x4 ea = *reinterpret_cast<const f32x4 *>(d.in + g4) * scale;
            const f32x4 eb = *reinterpret_cast<const f32x4 *>(d.in + 16 + g4) * scale;
            const Frag<L> fv = frag_col<LV, false>(vs, w0, lane);
            f32x4 ga, gb;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ga[i] = (float)fv.x[i] - ea[i] * X[0][i];
                gb[i] = (float)fv.x[4 + i] - eb[i] * X[1][i];
            }
            split(fg, ga, gb);
            U[0] = U[1] = f32x4{};
#pragma unroll
            for (int u = PARTS - 1; u >= 0; --u) {
                Frag<L> ft[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) ft[t] = piece<L>(lds.t, t, u, lane);
#pragma unroll
                for (int o = PARTS - 1 - u; o >= 0; --o)
#pragma unroll
                    for (int t = 0; t < 2; ++t) U[t] = mma(ft[t], fg[o], U[t]);
            }
        }
        // An infinity or a NaN in k, v, beta, a decay or the state shows in U.
        float zero = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) zero = __builtin_fmaf(U[t][i], 0.f, zero);
        const bool odd = __ballot(!(zero == 0.f)) != 0;
        E *yc = OUT ? y + c * C * a.st.y_t : nullptr;
        if (__builtin_expect(odd, 0)) {
            // The products above would carry it to rows before its own, where T
            // and P are 0: the recurrence itself, row by row.
#pragma unroll
            for (int m = 0; m < MT; ++m) S[m] *= scale;
            scale = 1.f;
            const int ln = anew(lane), l16 = ln & 15, g4 = (ln >> 4) * 4;
#pragma unroll 1
            for (int j = 0; j < rows; ++j) {
                const float dec = __expf(clamp_decay(la[(c * C + j) * a.la_t]));
                const float beta = a.beta[(int64_t)(p.begin + c * C + j) * a.beta_t + h];
                float dot = 0.f, out = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const Frag<L> fk = frag8(ks + j * LK + 32 * s + 2 * g4);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float &x = reinterpret_cast<float *>(&S[2 * s + i / 4])[i % 4];
                        x *= dec;
                        dot += (float)fk.x[i] * x;
                    }
                }
                dot += __shfl_xor(dot, 16);
                dot += __shfl_xor(dot, 32);
                dot = beta * (to_f(vs[j * LV + w0 + l16]) - dot);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const Frag<L> fk = frag8(ks + j * LK + 32 * s + 2 * g4), fq = frag8(qs + j * LK + 32 * s + 2 * g4);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float &x = reinterpret_cast<float *>(&S[2 * s + i / 4])[i % 4];
                        x += (float)fk.x[i] * dot;
                        out += (float)fq.x[i] * x;
                    }
                }
                out += __shfl_xor(out, 16);
                out += __shfl_xor(out, 32);
                if (OUT && ln < 16 && w0 + l16 < cols) yc[j * a.st.y_t + w0 + l16] = from_f<E>(out);
            }
            block_sync();
            continue;
        }
        const float entered = scale;
        scale = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(scale * d.all)));
        if (!(scale > 0x1p-16f && scale < 0x1p16f)) {   // and where it is NaN
#pragma unroll
            for (int m = 0; m < MT; ++m) S[m] *= scale;
            scale = 1.f;
        }
        const float unscale = 1.f / scale;
#pragma unroll
        for (int t = 0; t < 2; ++t) Y[t] *= d.in[16 * t + l16] * entered;
        if constexpr (OUT) {
            Frag<L> fu[YU], fp[2][YU];
            split(fu, U[0], U[1]);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int u = 0; u < YU; ++u) fp[t][u] = piece<L, YU>(lds.p, t, u, lane);
#pragma unroll
            for (int o = YU - 1; o >= 0; --o)   // the small products first
#pragma unroll
                for (int u = 0; u <= o; ++u)
#pragma unroll
                    for (int t = 0; t < 2; ++t) Y[t] = mma(fu[u], fp[t][o - u], Y[t]);
        }
        Frag<L> fw[PARTS];
        split(fw, U[0] * (*reinterpret_cast<const f32x4 *>(d.out + g4) * unscale),
              U[1] * (*reinterpret_cast<const f32x4 *>(d.out + 16 + g4) * unscale));
        // four accumulators' rows at a time: as many products that do not wait for each other
#pragma unroll
        for (int m0 = 0; m0 < MT; m0 += 4) {
            Frag<L> fk[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) fk[m] = frag_col<LK, true>(ks, 32 * ((m0 + m) / 2) + 4 * (m % 2), lane);
#pragma unroll
            for (int u = PARTS - 1; u >= 0; --u)
#pragma unroll
                for (int m = 0; m < 4; ++m) S[m0 + m] = mma(fk[m], fw[u], S[m0 + m]);
        }
        if constexpr (OUT) {
            const rsrc_t r = make_rsrc(yc, ((rows - 1) * a.st.y_t + cols) * (int64_t)sizeof(E));
            const int col = w0 + g4;   // 4 columns from here on
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int row = 16 * t + l16;
                const uint32_t off = (uint32_t)(row * (int)a.st.y_t + col) * (uint32_t)sizeof(E);
                E out[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) out[e] = from_f<E>(Y[t][e]);
#pragma unroll
                for (int e = 0; e < 4; e += VEC ? 4 : 1) {
                    const uint32_t o = row < rows && col + e < cols ? off + e * (uint32_t)sizeof(E) : kOOB;
                    if constexpr (VEC && sizeof(E) == 4) {
                        ssd::v4u x;
                        __builtin_memcpy(&x, out + e, 16);
                        __builtin_amdgcn_raw_buffer_store_b128(x, r, o, 0, 0);
                    } else if constexpr (VEC) {
                        ssd::v2u x;
                        __builtin_memcpy(&x, out + e, 8);
                        __builtin_amdgcn_raw_buffer_store_b64(x, r, o, 0, 0);
                    } else if constexpr (sizeof(E) == 2) {
                        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, out[e]), r, o, 0, 0);
                    } else {
                        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, out[e]), r, o, 0, 0);
                    }
                }
            }
        }
        block_sync();
    }

    float *to = OUT ? (p.s + 1 == p.segs ? pool : nullptr) : ends;
    const rsrc_t r = make_rsrc(to, to ? state * 4 : 0);
    const int at = anew(lane);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) ssd::gstore1(r, state_at(m, i, at), S[m][i] * scale);
}

// The states that enter the segments of a sequence that was cut, in place of
// the states that the segments make from zero: S_{s+1} = M_s S_s + B_s, in
// float32.  A block has 16 columns of one head's states; a wave has 16 rows of
// M (twice where dk is over 128) and the next segments' on their way, and the
// state goes round the waves through LDS, transposed.  2.3 us a segment at dk
// 128, of which its fp32 MFMA (32 of 32 cycles for each of two waves on a SIMD)
// is 1; with the loads of M 4 bytes at a time and none ahead it took 7.
template <int KP>
struct CarryWaves {
    static constexpr int n = KP / 16 < 8 ? KP / 16 : 8, ahead = KP == 256 ? 1 : 3;
};
template <int KP>
__global__ __launch_bounds__(64 * CarryWaves<KP>::n) void k_delta_carry(DeltaArgs a)
{
    constexpr int WAVES = CarryWaves<KP>::n, NR = KP / 16 / WAVES, KS = KP / 16, LS = KP + 4;
    constexpr int AHEAD = CarryWaves<KP>::ahead;
    __shared__ __align__(16) float St[2][16 * LS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int h = blockIdx.x % a.H, col = blockIdx.y * 16 + l16;
    Place p;
    int begin, end;
    about(a, blockIdx.x / a.H, p, begin, end);
    if (p.segs <= 1 || p.bad) return;
    const int64_t id0 = begin / a.seg + p.n, state = (int64_t)a.dk * a.dv, map = (int64_t)a.dk * a.map_cols;
    float *ends = a.ends + (id0 * a.H + h) * state;
    const float *maps = a.maps + (id0 * a.H + h) * map;
    // rows 16 (n WAVES + w) + g4 + i of column col; M's rows 16 (n WAVES + w) + l16, columns 16 s + g4 ..
    const auto at = [&](int n, int i) {
        const int row = 16 * (n * WAVES + w) + g4 + i;
        return col < a.dv && row < a.dk ? (uint32_t)(row * a.dv + col) * 4u : kOOB;
    };
    struct Step {
        f32x4 M[NR][KS], B[NR];
    };
    const auto load = [&](Step &x, int s) {
        const rsrc_t rm = make_rsrc(maps + s * (a.H * map), map * 4), rb = make_rsrc(ends + s * (a.H * state), state * 4);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x.B[n][i] = ssd::gload1(rb, at(n, i));
            const int row = 16 * (n * WAVES + w) + l16;   // past dk: past the end
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int c = 16 * k + g4;
                const uint32_t o = c < a.map_cols ? (uint32_t)(row * a.map_cols + c) * 4u : kOOB;
                x.M[n][k] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rm, o, 0, 0));
            }
        }
    };
    f32x4 S[NR];
    {
        const float *from = p.carry ? a.states + ((int64_t)p.slot * a.H + h) * state : nullptr;
        const rsrc_t r = make_rsrc(from, from ? state * 4 : 0);
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[n][i] = ssd::gload1(r, at(n, i));
    }
    // leaves S in place of B; false where that was the last
    const auto enter = [&](int s) {
        float *st = St[s & 1];
        const rsrc_t r = make_rsrc(ends + s * (a.H * state), state * 4);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            *reinterpret_cast<f32x4 *>(st + l16 * LS + 16 * (n * WAVES + w) + g4) = S[n];
#pragma unroll
            for (int i = 0; i < 4; ++i) ssd::gstore1(r, at(n, i), S[n][i]);
        }
        return s + 1 < p.segs;
    };
    const auto join = [&](const Step &x, int s) {
        const float *st = St[s & 1];
        f32x4 sum[NR][4];   // chains that do not wait for each other
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            sum[n][0] = x.B[n];
            sum[n][1] = sum[n][2] = sum[n][3] = f32x4{};
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const f32x4 f = *reinterpret_cast<const f32x4 *>(st + l16 * LS + 16 * k + g4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    sum[n][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.M[n][k][e], f[e], sum[n][e], 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) S[n] = (sum[n][0] + sum[n][1]) + (sum[n][2] + sum[n][3]);
    };
    // the maps of AHEAD segments in flight; the last segment made none, and the
    // loads past it are of the one before
    const int last = p.segs - 2;
    Step x[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(x[u], min(u, last));
    for (int s0 = 0;; s0 += AHEAD)
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (!enter(s0 + u)) return;
            block_sync();
            join(x[u], s0 + u);
            load(x[u], min(s0 + u + AHEAD, last));
        }
}

// ---- host side

// Columns of a block: 64 where that leaves a block a CU of its own, whose chain
// of chunks is then shorter (512 rows, 8 heads of 128: bfloat16 40 us where 128
// columns take 54; float32 108 and 158), and with bfloat16's and dk <= 64's few
// registers and LDS, where two of them share one (8 prompts of 8192 rows, 16
// heads of 64 x 128: 510 and 604).  Else 128, for T and P are then made half as
// often (16 x 8192 rows, 16 heads of 128: 909 and 1060; float32, 2 x 8192: 746
// and 964).  Long sequences count as the pieces that they can be cut into.
static int col_tile(const lin_shape &s, int dtype, int cus)
{
    if (s.dk > 128 || s.dv <= 64) return 64;
    const int64_t pieces = s.T / 256 > s.N ? s.T / 256 : s.N;
    if (pieces * s.H * ((s.dv + 63) / 64) <= cus) return 64;
    return s.dk <= 64 && dtype == LAYER_BF16 ? 64 : 128;
}

struct DeltaPlan {
    int seg = 0, ids = 0, map_cols = 0, map_tiles = 0;
    size_t ends = 0, maps = 0, total = 0;
};

// Sequences are cut where that is faster by an estimate: into segments of a
// length that makes about one block for each place on a CU out of the batch's
// rows, at least 256.  Whole, the longest one's chain of chunks counts, or all
// rows over the places; cut, the output pass's rows and, for 0.7 of its time
// each, those of the blocks for B and M, with 1.2 us for each segment that the
// carry pass joins and 15 us for two launches more.  (One prompt of 32768 rows,
// 8 heads of 128: 2965 us whole; cut into 32, 355, of which the maps take 195,
// the carry pass 74 and the outputs 118.  20 prompts, 3000 rows the longest, 24
// heads of 128 x 64: 210 us whole, 166 cut.  8 prompts of 8192, 32 heads of 64:
// 470 whole, 900 cut.)
static DeltaPlan plan_delta(const lin_shape &s, int dtype, int64_t max_seqlen, int cus)
{
    DeltaPlan P;
    const int64_t longest = max_seqlen > 0 && max_seqlen < s.T ? max_seqlen : s.T;
    const int64_t vt = col_tile(s, dtype, cus), tiles = (s.dv + vt - 1) / vt, map_tiles = (s.dk + vt - 1) / vt;
    const int64_t places = (vt == 64 && s.dk <= 128 && dtype == LAYER_BF16 ? 2 : 1) * (int64_t)cus;
    P.ids = (int)s.N;
    P.map_cols = (int)((s.dk + 3) / 4 * 4);
    P.map_tiles = (int)map_tiles;
    int64_t seg = ((s.T * s.H * tiles + places - 1) / places + 63) / 64 * 64;
    if (seg < 256) seg = 256;
    const double row = dtype == LAYER_BF16 ? 0.1 : 0.2;   // us
    const double all = (double)s.T * (double)(s.H * tiles) / (double)places;
    const double whole = row * (all > (double)longest ? all : (double)longest);
    const double cut = row * ((double)seg + 0.7 * (double)seg * (double)(tiles + map_tiles) / (double)tiles) +
                       1.2 * (double)longest / (double)seg + 15.0;
    if (longest <= seg || whole <= cut) return P;
    // and no more of them than a launch has blocks for
    const int64_t most = max_blocks(1024) / (s.H * (tiles + map_tiles)) - s.N;
    if (most < 1) return P;
    if (s.T / seg > most) seg = (s.T / most + 64) / 64 * 64;
    if (longest <= seg || seg >= (int64_t(1) << 30)) return P;
    P.seg = (int)seg;
    P.ids = (int)(s.T / seg + s.N);
    P.ends = 0;
    P.maps = ((size_t)(P.ids * s.H * s.dk * s.dv) * sizeof(float) + 255) / 256 * 256;
    P.total = P.maps + (size_t)(P.ids * s.H * s.dk * P.map_cols) * sizeof(float);
    return P;
}

// The workspace for any element type.
static size_t delta_workspace(const lin_shape &s, int64_t max_seqlen, int cus)
{
    const size_t a = plan_delta(s, LAYER_BF16, max_seqlen, cus).total, b = plan_delta(s, LAYER_F32, max_seqlen, cus).total;
    return a > b ? a : b;
}

template <typename E, int KP, int VT, bool VEC>
static int run_delta(DeltaArgs &a, hipStream_t st)
{
    constexpr int threads = DeltaPerCu<E, KP, VT>::threads;
    if (a.seg > 0) {
        const int64_t grid = (int64_t)a.ids * a.H * (a.tiles + a.map_tiles);
        k_delta_chunks<E, KP, VT, false, VEC><<<dim3((unsigned)grid), dim3(threads), 0, st>>>(a);
        const dim3 carry((unsigned)(a.N * a.H), (unsigned)((a.dv + 15) / 16));
        k_delta_carry<KP><<<carry, dim3(64 * CarryWaves<KP>::n), 0, st>>>(a);
    }
    const int64_t grid = (int64_t)a.ids * a.H * a.tiles;
    k_delta_chunks<E, KP, VT, true, VEC><<<dim3((unsigned)grid), dim3(threads), 0, st>>>(a);
    return launch_status();
}

template <typename E, bool VEC>
static int dispatch_delta(DeltaArgs &a, bool wide, hipStream_t st)
{
    if (a.dk > 128) return run_delta<E, 256, 64, VEC>(a, st);
    if (a.dk > 64) return wide ? run_delta<E, 128, 128, VEC>(a, st) : run_delta<E, 128, 64, VEC>(a, st);
    return wide ? run_delta<E, 64, 128, VEC>(a, st) : run_delta<E, 64, 64, VEC>(a, st);
}

}  // namespace layer

using namespace layer;

extern "C" size_t delta_prefill_workspace_size(const lin_shape *shape, int64_t max_seqlen)
{
    if (check_delta(shape, false) != SSD_OK || max_seqlen < 0) return (size_t)-1;
    return delta_workspace(*shape, max_seqlen, ssd::device_cus());
}

extern "C" int delta_prefill(const lin_shape *shape, int dtype, const lin_strides *strides, const void *q,
                             const void *k, const void *v, const float *log_decay, int64_t decay_stride,
                             const float *beta, int64_t beta_stride, const int32_t *cu_seqlens, const int32_t *slots,
                             const int32_t *carry, int64_t max_seqlen, float *states, void *y, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    int rc = check_delta(shape, false);
    if (rc == SSD_OK) rc = check_dtype(dtype);
    if (rc != SSD_OK) return rc;
    const lin_shape &s = *shape;
    DeltaArgs a;
    rc = resolve_strides(shape, strides, &a.st, s.T);
    if (rc != SSD_OK) return rc;
    if (decay_stride < 0 || decay_stride >= kMaxCount || beta_stride < 0 || beta_stride >= kMaxCount || max_seqlen < 0)
        return SSD_ERR_SHAPE;
    if (!slots && s.N > s.slots) return SSD_ERR_SHAPE;
    if (s.N == 0) return SSD_OK;
    if (!cu_seqlens || (s.slots > 0 && !states)) return SSD_ERR_NULL;
    if (s.T > 0 && (!q || !k || !v || !log_decay || !beta || !y)) return SSD_ERR_NULL;
    const unsigned e = dtype_size(dtype);
    if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(y, e) || misaligned(log_decay, 4) ||
        misaligned(beta, 4) || misaligned(slots, 4) || misaligned(states, 4) || misaligned(cu_seqlens, 4) ||
        misaligned(carry, 4))
        return SSD_ERR_ALIGN;
    const int cus = ssd::device_cus();
    const DeltaPlan P = plan_delta(s, dtype, max_seqlen, cus);
    const size_t need = delta_workspace(s, max_seqlen, cus);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (need > 0 && !workspace) return SSD_ERR_NULL;
    if (need > 0 && misaligned(workspace, 16)) return SSD_ERR_ALIGN;
    a.q = q;
    a.k = k;
    a.v = v;
    a.la = log_decay;
    a.la_t = decay_stride;
    a.beta = beta;
    a.beta_t = beta_stride;
    a.cu = cu_seqlens;
    a.slots = slots;
    a.carry = carry;
    a.states = states;
    a.y = y;
    a.ends = reinterpret_cast<float *>(static_cast<char *>(workspace) + P.ends);
    a.maps = reinterpret_cast<float *>(static_cast<char *>(workspace) + P.maps);
    a.segdec = nullptr;
    a.map_cols = P.map_cols;
    a.map_tiles = P.map_tiles;
    a.T = (int)s.T;
    a.N = (int)s.N;
    a.G = (int)s.G;
    a.H = (int)s.H;
    a.dk = (int)s.dk;
    a.dv = (int)s.dv;
    a.nslots = (int)s.slots;
    const int vt = col_tile(s, dtype, cus);
    a.tiles = (a.dv + vt - 1) / vt;
    a.seg = P.seg;
    a.ids = P.ids;
    a.shift = -1;
    const auto rows16 = [&](const void *ptr, int64_t row, int64_t head, int64_t d) {
        return !misaligned(ptr, 16) && row * e % 16 == 0 && head * e % 16 == 0 && d * e % 16 == 0 && row >= d;
    };
    const bool vec = rows16(q, a.st.q_t, a.st.q_g, s.dk) && rows16(k, a.st.k_t, a.st.k_g, s.dk) &&
                     rows16(v, a.st.v_t, a.st.v_h, s.dv) && rows16(y, a.st.y_t, a.st.y_h, s.dv);
    const bool wide = vt == 128;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LAYER_BF16) return vec ? dispatch_delta<bf16, true>(a, wide, st) : dispatch_delta<bf16, false>(a, wide, st);
    if (dtype == LAYER_F16) return vec ? dispatch_delta<f16, true>(a, wide, st) : dispatch_delta<f16, false>(a, wide, st);
    return vec ? dispatch_delta<float, true>(a, wide, st) : dispatch_delta<float, false>(a, wide, st);
}
