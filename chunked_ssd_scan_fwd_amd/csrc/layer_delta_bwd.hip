// Gradients of the gated delta rule over a packed batch.
//
// With M, D, b as in layer_delta.h, Z = (I + M diag(beta))^-1 (V - diag(e^b) K S)
// and U = diag(beta) Z, T = (I + diag(beta) M)^-1, P = Q K^T o D, A the
// gradient of the state that leaves a chunk and S the state that enters it:
//   dU = P^T dY + diag(e^{b_L-b}) K A,  dG = T^T dU,  dV = dR = diag(beta) dG
//   dS = e^{b_L} A + Q^T diag(e^b) dY - K^T diag(e^b) dR
//   dbeta_i = dG_i . Z_i
//   dP = dY U^T o D,  dM = -dR U^T o D (below the diagonal)
//   dQ = diag(e^b) dY S^T + dP K
//   dK = diag(e^{b_L-b}) U A^T - diag(e^b) dR S^T + dP^T Q + (dM + dM^T) K
//   dlog_decay_r = sum_{i>=r} f_i + sum_{j<r<=i} N_ij + sum_{j<r} e_j + e^{b_L} <S, A>
//     f_i = q_i . (e^b dY S^T)_i - k_i . (e^b dR S^T)_i,  e_j = k_j . (e^{b_L-b} U A^T)_j
//     N = dP o Q K^T + dM o K K^T
// (each decay factor differentiated by itself: no terms that cancel).
//
// Z and dG belong to rows, however the rows are cut into chunks.  So three
// kernels: what no state enters, for chunks of 32 rows (k_delta_back_inverse);
// the states from the left and their gradients from the right, by chunks of
// 32, both in one launch, which leave Z, dG and every CB-th row's state
// (k_delta_walk); and the products inside all chunks of CB rows at once
// (k_delta_grads).  4 x 2048 rows, 16 heads of 128, bfloat16: 36, 194 and 243
// us.  The states written and read, 536 MB, are most of what moves.
#include "layer_delta.h"

namespace layer {

constexpr int CW = 32;   // rows of a chunk of the walks

struct DeltaBackArgs : DeltaArgs {
    const void *dy;
    char *inv;                     // the walk chunks' T~, T^T and P^T, [chunk][H]
    const float *dlast;            // gradients of the last states, or null
    float *zrec, *grec;            // [walk chunk][H][CW][dvp]
    float *srec, *arec;            // [chunk of CB][H][dk][dvp]
    float *dq_head, *dk_head;      // [T][H][dk], where heads share q and k
    void *dq, *dk_out, *dv_out;
    float *dla, *dla_rows, *dbeta, *dfirst;
    int dvp, cb;
    bool clear;                    // zeros for the gradients of rows of no sequence
};

// ---- T~ = (I + M diag(beta))^-1, T^T and P^T of a chunk of 32 rows, in pieces
template <typename E, int KP, bool VEC>
__global__ __launch_bounds__(256) void k_delta_back_inverse(DeltaBackArgs a)
{
    typedef typename std::conditional<std::is_same<E, bf16>::value, bf16, float>::type L;
    typedef Pieces<L> PC;
    constexpr int PT = 256, KS = KP / 32;
    constexpr int LK = KP + (sizeof(L) == 2 ? 16 : 4), LA = CW + 4;
    __shared__ __align__(16) L ks[CW * LK], qs[CW * LK];
    __shared__ __align__(16) float A[2][16 * LA], X[2][CW * LA], betas[CW];
    __shared__ Decays<CW> d;

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int h = blockIdx.x % a.H;
    int id = blockIdx.x / a.H;
    Place p;
    if (!find(a, id, p) || p.rows <= 0) return;
    const int g = h / (a.H / a.G);
    {
        Tile<E, CW, KP, PT> tk, tq;
        const E *k = static_cast<const E *>(a.k) + p.begin * a.st.k_t + g * a.st.k_g;
        const E *q = static_cast<const E *>(a.q) + p.begin * a.st.q_t + g * a.st.q_g;
        tk.template fetch<VEC>(k, a.st.k_t, p.rows, a.dk, tid);
        tq.template fetch<VEC>(q, a.st.q_t, p.rows, a.dk, tid);
        const int64_t row = p.begin + lane;
        const bool on = lane < p.rows;
        const float la = on ? a.la[(a.la_t ? row * a.la_t : 0) + h] : 0.f;
        if (w == 0) make_decays(d, la, lane);
        if (w == 1 && lane < CW) betas[lane] = on ? a.beta[row * a.beta_t + h] : 0.f;
        tk.template place<VEC, LK>(ks, k, a.st.k_t, a.dk, tid);
        tq.template place<VEC, LK>(qs, q, a.st.q_t, a.dk, tid);
    }
    block_sync();
    const auto product = [&](const L *rows, int i, int j) {   // rows_i k_j^T
        f32x4 x = {};
#pragma unroll
        for (int s = 0; s < KS; ++s)
            x = mma(frag8(rows + (16 * i + l16) * LK + 32 * s + 2 * g4), frag8(ks + (16 * j + l16) * LK + 32 * s + 2 * g4),
                    x);
        return x;
    };
    // times D; STRICT: below the diagonal only
    const auto masked = [&](f32x4 x, int i, int j, bool strict) {
        const f32x4 ih = *reinterpret_cast<const f32x4 *>(d.hi + 16 * i + g4);
        const f32x4 il = *reinterpret_cast<const f32x4 *>(d.lo + 16 * i + g4);
        const float jh = d.hi[16 * j + l16], jl = d.lo[16 * j + l16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] *= __expf((ih[e] - jh) + (il[e] - jl));
            if (16 * j + l16 + (strict ? 0 : -1) >= 16 * i + g4 + e) x[e] = 0.f;
        }
        return x;
    };
    // waves 0, 1: diag(beta) M; waves 2, 3: M diag(beta); a diagonal block each
    const int which = w >> 1, blk = w & 1;
    const auto scaled = [&](f32x4 x, int i, int j) {
        const f32x4 bi = *reinterpret_cast<const f32x4 *>(betas + 16 * i + g4);
        const float bj = betas[16 * j + l16];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= which == 0 ? bi[e] : bj;
        return x;
    };
    {
        const f32x4 x = scaled(masked(product(ks, blk, blk), blk, blk, true), blk, blk);
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
            for (int i = 0; i < 16; ++i) X[which][(16 * blk + i) * LA + 16 * blk + l16] = t[i];
        if (blk == 1) {
            const f32x4 y = scaled(masked(product(ks, 1, 0), 1, 0, true), 1, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) A[which][(g4 + e) * LA + l16] = y[e];
        }
    }
    char *out = a.inv + ((int64_t)id * a.H + h) * 3 * PC::BYTES;
    const auto put = [&](char *to, int f, f32x4 x, f32x4 y) {
        Frag<L> parts[PC::PARTS];
        split(parts, x, y);
#pragma unroll
        for (int u = 0; u < PC::PARTS; ++u)
#pragma unroll
            for (int i = 0; i < PC::UNITS; ++i)
                *reinterpret_cast<u32x4 *>(to + (((f * PC::PARTS + u) * PC::UNITS + i) * 64 + lane) * 16) =
                    *reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(&parts[u]) + 16 * i);
    };
    block_sync();
    if (blk == 0) {   // T_10 = -T_11 A_10 T_00
        const auto times = [&](const float *m, const f32x4 &b) {   // m: 16 x 16 of rows LA apart
            const f32x4 f = *reinterpret_cast<const f32x4 *>(m + l16 * LA + g4);
            f32x4 c = {};
#pragma unroll
            for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(f[e], b[e], c, 0, 0, 0);
            return c;
        };
        f32x4 t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = X[which][(g4 + e) * LA + l16];
        t = times(X[which] + 16 * LA + 16, -times(A[which], t));
#pragma unroll
        for (int e = 0; e < 4; ++e) X[which][(16 + g4 + e) * LA + l16] = t[e];
    } else {
        // P^T: waves 1 and 3, piece 0 and 1
        const int t = which;
        const f32x4 lo = t == 0 ? masked(product(qs, 0, 0), 0, 0, false) : f32x4{};
        const f32x4 hi = t == 0 ? masked(product(qs, 1, 0), 1, 0, false) : masked(product(qs, 1, 1), 1, 1, false);
        put(out + 2 * PC::BYTES, t, lo, hi);
    }
    block_sync();
    // wave w: piece w & 1 of T~ (waves 2, 3, from X[1]) or of T^T (waves 0, 1, from X[0])
    {
        const int t = blk;
        f32x4 x, y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (which == 1) {
                x[e] = X[1][(16 * t + l16) * LA + g4 + e];
                y[e] = t == 0 ? 0.f : X[1][(16 + l16) * LA + 16 + g4 + e];
            } else {
                x[e] = t == 0 ? X[0][(g4 + e) * LA + l16] : 0.f;
                y[e] = X[0][(16 + g4 + e) * LA + 16 * t + l16];
            }
        }
        put(out + (which == 1 ? 0 : PC::BYTES), t, x, y);
    }
}

// ---- the states, and their gradients
template <typename E, int KP>
struct WalkLds {
    typedef typename std::conditional<std::is_same<E, bf16>::value, bf16, float>::type L;
    static constexpr int PAD = sizeof(L) == 2 ? 16 : 4, VT = 64;
    static constexpr int LK = KP + PAD, LV = VT + PAD;
    L q[2][CW * LK], k[2][CW * LK], v[2][CW * LV];
    Decays<CW> dec[3];
    alignas(16) float beta[3][CW];
};

// One sequence for one head and 64 columns, with the state (or its gradient)
// in the registers of four waves, 16 columns each, while four others fetch the
// next chunk.  BACK: from the last chunk to the first.  Its chain of dependent
// steps bounds it, about 3 us a chunk: a SIMD has matrix instructions under way
// in 0.2 of that and vector ones in 0.3.  Sequences are not cut, so one of 32768
// rows with 8 heads of 128 takes 2.9 ms on 32 CUs.  For dk over 128 it spills 39
// to 63 registers.
template <typename E, int KP, bool VEC, bool BACK>
__device__ __forceinline__ void walk(const DeltaBackArgs &a, WalkLds<E, KP> &lds, int n, int h, int tile)
{
    typedef WalkLds<E, KP> Lds;
    typedef typename Lds::L L;
    typedef Pieces<L> PC;
    constexpr int LK = Lds::LK, LV = Lds::LV, VT = Lds::VT, C = CW;
    constexpr int MT = KP / 16, KS = KP / 32, PARTS = PC::PARTS, PT = 256;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    int begin, end;
    rows_of(a, n, begin, end);
    const int rows = end - begin, chunks = (rows + C - 1) / C;
    const int g = h / (a.H / a.G), c0 = tile * VT, cols = min(VT, a.dv - c0);
    const int64_t id0 = chunk_number(n, begin, 0, C);
    const auto chunk = [&](int c) { return BACK ? chunks - 1 - c : c; };   // the c-th that is visited

    if (wave >= 4) {
        const int tid = threadIdx.x - 256, w = wave - 4;
        const E *q = static_cast<const E *>(a.q) + begin * a.st.q_t + g * a.st.q_g;
        const E *k = static_cast<const E *>(a.k) + begin * a.st.k_t + g * a.st.k_g;
        const int64_t v_t = BACK ? a.st.y_t : a.st.v_t;
        const E *v = BACK ? static_cast<const E *>(a.dy) + begin * a.st.y_t + h * a.st.y_h + c0
                          : static_cast<const E *>(a.v) + begin * a.st.v_t + h * a.st.v_h + c0;
        const float *la = a.la + (a.la_t ? begin * a.la_t : 0) + h;
        const float *beta = a.beta + begin * a.beta_t + h;
        Tile<E, C, KP, PT> tq, tk;
        Tile<E, C, VT, PT> tv;
        const auto load = [&](int c) {
            // past the last one: nothing
            const int64_t t0 = (int64_t)chunk(c) * C;
            const int left = c < chunks ? min(C, (int)(rows - t0)) : 0;
            const int64_t at = c < chunks ? t0 : 0;
            if (BACK) tq.template fetch<VEC>(q + at * a.st.q_t, a.st.q_t, left, a.dk, tid);
            tk.template fetch<VEC>(k + at * a.st.k_t, a.st.k_t, left, a.dk, tid);
            tv.template fetch<VEC>(v + at * v_t, v_t, left, cols, tid);
        };
        const auto decays = [&](int c) {   // two waves: the log decays, and beta
            const int t = chunk(c) * C + lane;
            const bool on = c < chunks && lane < C && t < rows;
            if (w == 3) make_decays(lds.dec[c % 3], on ? la[t * a.la_t] : 0.f, lane);
            if (w == 2 && lane < C) lds.beta[c % 3][lane] = on ? beta[t * a.beta_t] : 0.f;
        };
        const auto store = [&](int c) {
            const int b = c & 1;
            const int64_t at = c < chunks ? (int64_t)chunk(c) * C : 0;
            if (BACK) tq.template place<VEC, LK>(lds.q[b], q + at * a.st.q_t, a.st.q_t, a.dk, tid);
            tk.template place<VEC, LK>(lds.k[b], k + at * a.st.k_t, a.st.k_t, a.dk, tid);
            tv.template place<VEC, LV>(lds.v[b], v + at * v_t, v_t, cols, tid);
        };
        load(0);
        decays(0);
        store(0);
        load(1);
        block_sync();
        for (int c = 0; c < chunks; ++c) {
            decays(c + 1);
            store(c + 1);
            load(c + 2);
            block_sync();
        }
        return;
    }

    __builtin_amdgcn_s_setprio(1);
    const int64_t state = (int64_t)a.dk * a.dv, rec = (int64_t)a.dk * a.dvp;
    const int w0 = 16 * wave, col = c0 + w0 + l16;
    // S: value i of accumulator m is row 32 (m / 2) + 2 g4 + 4 (m % 2) + i, column w0 + l16
    f32x4 S[MT];
    // its byte offset in states whose rows are `width` long; a row past dk lies past the end
    const auto state_at = [&](int m, int i, int width) {
        const uint32_t row = 2 * g4 + 32 * (m / 2) + 4 * (m % 2) + i;
        return col < width ? (row * (uint32_t)width + (uint32_t)col) * 4u : kOOB;
    };
    {
        const float *all = BACK ? a.dlast : a.states;
        const float *from = all ? all + ((int64_t)n * a.H + h) * state : nullptr;
        const rsrc_t r = make_rsrc(from, from ? state * 4 : 0);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[m][i] = ssd::gload1(r, state_at(m, i, a.dv));
    }
    // the pieces of T~, or of T^T and P^T: a chunk's are on their way while the
    // chunk before it ends
    Frag<L> ft[2][PARTS], fp[2][PARTS];
    const auto load_pieces = [&](int c) {
        const char *image = a.inv + ((id0 + chunk(min(c, chunks - 1))) * a.H + h) * 3 * PC::BYTES;
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int u = 0; u < PARTS; ++u) {
                if (BACK) fp[f][u] = piece<L>(image + 2 * PC::BYTES, f, u, lane);
                ft[f][u] = piece<L>(image + (BACK ? PC::BYTES : 0), f, u, lane);
            }
    };
    if (chunks > 0) load_pieces(0);
    block_sync();
    for (int c = 0; c < chunks; ++c) {
        const int b = c & 1, cc = chunk(c);
        const Decays<C> &d = lds.dec[c % 3];
        const float *betas = lds.beta[c % 3];
        const L *qs = lds.q[b], *ks = lds.k[b], *vs = lds.v[b];
        const int64_t id = (id0 + cc) * a.H + h;
        // the state that enters the chunk of cb rows, or the gradient of the one that leaves it
        if (BACK ? (cc + 1) % (a.cb / C) == 0 || cc + 1 == chunks : cc % (a.cb / C) == 0) {
            float *to = (BACK ? a.arec : a.srec) + ((int64_t)chunk_number(n, begin, cc * C, a.cb) * a.H + h) * rec;
            const rsrc_t r = make_rsrc(to, rec * 4);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) ssd::gstore1(r, state_at(m, i, a.dvp), S[m][i]);
        }
        f32x4 X[2], part[2][PARTS] = {};   // chains that do not wait for each other
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            Frag<L> fs[PARTS];
            split(fs, S[2 * s], S[2 * s + 1]);
            const Frag<L> fk0 = frag8(ks + l16 * LK + 32 * s + 2 * g4), fk1 = frag8(ks + (16 + l16) * LK + 32 * s + 2 * g4);
#pragma unroll
            for (int u = PARTS - 1; u >= 0; --u) {
                part[0][u] = mma(fk0, fs[u], part[0][u]);
                part[1][u] = mma(fk1, fs[u], part[1][u]);
            }
        }
        const auto summed = [&](int t) {
            f32x4 x = part[t][PARTS - 1];
#pragma unroll
            for (int u = PARTS - 2; u >= 0; --u) x += part[t][u];
            return x;
        };
        X[0] = summed(0);
        X[1] = summed(1);
        const f32x4 ea = *reinterpret_cast<const f32x4 *>(d.in + g4), eb = *reinterpret_cast<const f32x4 *>(d.in + 16 + g4);
        const f32x4 wa = *reinterpret_cast<const f32x4 *>(d.out + g4), wb = *reinterpret_cast<const f32x4 *>(d.out + 16 + g4);
        const f32x4 ba = *reinterpret_cast<const f32x4 *>(betas + g4), bb = *reinterpret_cast<const f32x4 *>(betas + 16 + g4);
        const Frag<L> fv = frag_col<LV, false>(vs, w0, lane);
        f32x4 va, vb;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            va[i] = (float)fv.x[i];
            vb[i] = (float)fv.x[4 + i];
        }
        Frag<L> fx[PARTS];
        if (BACK) {
            X[0] *= wa;
            X[1] *= wb;
#pragma unroll
            for (int u = PARTS - 1; u >= 0; --u)
#pragma unroll
                for (int t = 0; t < 2; ++t) part[t][u] = mma(fp[t][u], fv, f32x4{});
            split(fx, X[0] + summed(0), X[1] + summed(1));
        } else {
            split(fx, va - ea * X[0], vb - eb * X[1]);
        }
        f32x4 R[2];   // Z, or dG
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < PARTS; ++u) part[t][u] = f32x4{};
#pragma unroll
        for (int o = PARTS - 1; o >= 0; --o)
#pragma unroll
            for (int u = 0; u <= o; ++u)
#pragma unroll
                for (int t = 0; t < 2; ++t) part[t][o] = mma(ft[t][u], fx[o - u], part[t][o]);
        R[0] = summed(0);
        R[1] = summed(1);
        load_pieces(c + 1);
        {
            float *to = (BACK ? a.grec : a.zrec) + id * C * a.dvp;
            const rsrc_t r = make_rsrc(to, (int64_t)C * a.dvp * 4);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ssd::gstore1(r, col < a.dvp ? (uint32_t)((16 * t + g4 + i) * a.dvp + col) * 4u : kOOB, R[t][i]);
        }
        Frag<L> fy[PARTS];
        if (BACK) {
            split(fy, va * ea, vb * eb);
            split(fx, -(R[0] * ba * ea), -(R[1] * bb * eb));
        } else {
            split(fx, R[0] * ba * wa, R[1] * bb * wb);
        }
        const float all = d.all;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            S[m] *= all;
            const Frag<L> fk = frag_col<LK, true>(ks, 32 * (m / 2) + 4 * (m % 2), lane);
#pragma unroll
            for (int u = PARTS - 1; u >= 0; --u) S[m] = mma(fk, fx[u], S[m]);
            if (BACK) {
                const Frag<L> fq = frag_col<LK, true>(qs, 32 * (m / 2) + 4 * (m % 2), lane);
#pragma unroll
                for (int u = PARTS - 1; u >= 0; --u) S[m] = mma(fq, fy[u], S[m]);
            }
        }
        block_sync();
    }
    if (BACK && a.dfirst) {
        float *to = a.dfirst + ((int64_t)n * a.H + h) * state;
        const rsrc_t r = make_rsrc(to, state * 4);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) ssd::gstore1(r, state_at(m, i, a.dv), S[m][i]);
    }
}

template <typename E, int KP, bool VEC>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_delta_walk(DeltaBackArgs a)
{
    __shared__ __align__(16) WalkLds<E, KP> lds;
    if (a.clear) {
        int b0, b1, e0, e1;
        rows_of(a, 0, b0, e0);
        rows_of(a, a.N - 1, b1, e1);
        for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
            if (t >= b0 && t < e1) {
                t += (e1 - 1 - t) / gridDim.x * gridDim.x;   // the last of these that is a sequence's
                continue;
            }
            const int qk = a.G * a.dk, hv = a.H * a.dv;
            for (int i = threadIdx.x; i < qk; i += 512) {
                static_cast<E *>(a.dq)[t * qk + i] = (E)0.f;
                static_cast<E *>(a.dk_out)[t * qk + i] = (E)0.f;
            }
            for (int i = threadIdx.x; i < hv; i += 512) static_cast<E *>(a.dv_out)[t * hv + i] = (E)0.f;
            for (int i = threadIdx.x; i < a.H; i += 512) {
                a.dbeta[t * a.H + i] = 0.f;
                a.dla_rows[t * a.H + i] = 0.f;
            }
        }
    }
    const int tile = blockIdx.x % a.tiles, h = blockIdx.x / a.tiles % a.H;
    const int n = blockIdx.x / (a.tiles * a.H) % a.N;
    if (blockIdx.x / (a.tiles * a.H) < (unsigned)a.N)
        walk<E, KP, VEC, true>(a, lds, n, h, tile);
    else
        walk<E, KP, VEC, false>(a, lds, n, h, tile);
}

// The sum over 16 lanes that follow one another, in all of them.
__device__ __forceinline__ float sum16(float x)
{
    x = ssd::dpp_add<ssd::kRowRor + 8>(x);
    x = ssd::dpp_add<ssd::kRowRor + 4>(x);
    x = ssd::dpp_add<ssd::kRowRor + 2>(x);
    return ssd::dpp_add<ssd::kRowRor + 1>(x);
}

// ---- the products inside a chunk of CB rows
//
// All on fp32 MFMA.  A wave has 16 columns of dQ and dK (two times 16 where dk
// is over 128); the sums over dv go by slices of 32 columns through LDS.  (The
// bfloat16 training case took 365 us so, and takes 243 in the kernel below.)
template <int KP>
struct GradsLds {
    static constexpr int CB = KP == 256 ? 32 : 64, WAVES = KP == 64 ? 4 : 8, SL = 32;
    static constexpr int TT = CB / 16, TILES = TT * (TT + 1) / 2;
    static constexpr int LK = KP + 4, LS = SL + 4, LP = CB + 4;
    alignas(16) float q[CB * LK], k[CB * LK];
    union {
        struct {
            alignas(16) float dy[CB * LS], u[CB * LS], dr[CB * LS], s[KP * LS], a[KP * LS];
        } in;
        struct {
            alignas(16) float dp[CB * LP], dm[CB * LP];
        } pair;
    };
    Decays<CB> dec;
    alignas(16) float beta[CB];
    float sums[3][WAVES][CB], rowsum[2 * TILES][16], colsum[2 * TILES][16], dot[WAVES];
};

template <typename E, int KP, bool VEC>
__global__ __launch_bounds__(64 * GradsLds<KP>::WAVES) void k_delta_grads(DeltaBackArgs a)
{
    typedef GradsLds<KP> Lds;
    constexpr int CB = Lds::CB, WAVES = Lds::WAVES, SL = Lds::SL, TT = Lds::TT, TILES = Lds::TILES;
    constexpr int LK = Lds::LK, LS = Lds::LS, LP = Lds::LP, PT = 64 * WAVES, NS = KP / 16 / WAVES, KS = KP / 32;
    constexpr int TS = CB / 32, PAIRS = (2 * TILES + WAVES - 1) / WAVES;
    constexpr int RP = CB * SL / 4, RPER = (RP + PT - 1) / PT, SP = KP * SL / 4, SPER = SP / PT;   // 16-byte pieces
    __shared__ Lds lds;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int h = blockIdx.x % a.H;
    int id = blockIdx.x / a.H;
    Place p;
    if (!find(a, id, p) || p.rows <= 0) return;
    const int g = h / (a.H / a.G);
    const int first = p.begin - p.s * CB;
    const int64_t row0 = p.begin, idw = chunk_number(p.n, first, p.s * CB, CW);
    const float *srec = a.srec + ((int64_t)id * a.H + h) * a.dk * a.dvp;
    const float *arec = a.arec + ((int64_t)id * a.H + h) * a.dk * a.dvp;
    const int64_t rec_step = (int64_t)a.H * CW * a.dvp;
    const float *zrec = a.zrec + (idw * a.H + h) * CW * a.dvp, *grec = a.grec + (idw * a.H + h) * CW * a.dvp;
    const E *dy = static_cast<const E *>(a.dy) + row0 * a.st.y_t + h * a.st.y_h;

    Tile<E, CB, SL, PT> ty;
    f32x4 tz[RPER], tg[RPER], ts[SPER], ta[SPER];
    const auto load = [&](int c0) {
        ty.template fetch<VEC>(dy + c0, a.st.y_t, c0 < a.dv ? p.rows : 0, min(SL, a.dv - c0), tid);
#pragma unroll
        for (int u = 0; u < RPER; ++u) {
            const int e = u * PT + tid, row = e / 8, col = c0 + e % 8 * 4;
            const bool on = (RP % PT == 0 || e < RP) && row < p.rows && col < a.dvp;
            const int64_t at = row / CW * rec_step + (int64_t)(row % CW) * a.dvp + col;
            tz[u] = on ? *reinterpret_cast<const f32x4 *>(zrec + at) : f32x4{};
            tg[u] = on ? *reinterpret_cast<const f32x4 *>(grec + at) : f32x4{};
        }
#pragma unroll
        for (int u = 0; u < SPER; ++u) {
            const int e = u * PT + tid, row = e / 8, col = c0 + e % 8 * 4;
            const bool on = row < a.dk && col < a.dvp;
            ts[u] = on ? *reinterpret_cast<const f32x4 *>(srec + (int64_t)row * a.dvp + col) : f32x4{};
            ta[u] = on ? *reinterpret_cast<const f32x4 *>(arec + (int64_t)row * a.dvp + col) : f32x4{};
        }
    };
    load(0);
    {
        Tile<E, CB, KP, PT> t;
        const E *k = static_cast<const E *>(a.k) + row0 * a.st.k_t + g * a.st.k_g;
        const E *q = static_cast<const E *>(a.q) + row0 * a.st.q_t + g * a.st.q_g;
        t.template fetch<VEC>(k, a.st.k_t, p.rows, a.dk, tid);
        t.template place<VEC, LK>(lds.k, k, a.st.k_t, a.dk, tid);
        t.template fetch<VEC>(q, a.st.q_t, p.rows, a.dk, tid);
        t.template place<VEC, LK>(lds.q, q, a.st.q_t, a.dk, tid);
        const bool on = lane < p.rows && lane < CB;
        if (w == 0) make_decays(lds.dec, on ? a.la[(a.la_t ? (row0 + lane) * a.la_t : 0) + h] : 0.f, lane);
        if (w == 1 && lane < CB) lds.beta[lane] = on ? a.beta[(row0 + lane) * a.beta_t + h] : 0.f;
    }
    block_sync();
    f32x4 dyS[NS][TT] = {}, dRS[NS][TT] = {}, UA[NS][TT] = {}, pair[PAIRS] = {};
    float dbeta[RPER] = {}, dot = 0.f;
    for (int c0 = 0; c0 < a.dv; c0 += SL) {
        ty.template place<VEC, LS>(lds.in.dy, dy + c0, a.st.y_t, min(SL, a.dv - c0), tid);
#pragma unroll
        for (int u = 0; u < RPER; ++u) {
            const int e = u * PT + tid, row = e / 8, col = e % 8 * 4;
            if (RP % PT != 0 && e >= RP) continue;
            const float bt = lds.beta[row];
            const f32x4 dr = tg[u] * bt;
#pragma unroll
            for (int i = 0; i < 4; ++i) dbeta[u] += tg[u][i] * tz[u][i];
            *reinterpret_cast<f32x4 *>(lds.in.u + row * LS + col) = tz[u] * bt;
            *reinterpret_cast<f32x4 *>(lds.in.dr + row * LS + col) = dr;
            if (row < p.rows) {
                E *to = static_cast<E *>(a.dv_out) + ((row0 + row) * a.H + h) * a.dv + c0 + col;
                if (VEC && c0 + col < a.dv) {
                    Vec<E, 4> x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) x.v[i] = from_f<E>(dr[i]);
                    *reinterpret_cast<Vec<E, 4> *>(to) = x;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c0 + col + i < a.dv) to[i] = from_f<E>(dr[i]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < SPER; ++u) {
            const int e = u * PT + tid, row = e / 8, col = e % 8 * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) dot += ts[u][i] * ta[u][i];
            *reinterpret_cast<f32x4 *>(lds.in.s + row * LS + col) = ts[u];
            *reinterpret_cast<f32x4 *>(lds.in.a + row * LS + col) = ta[u];
        }
        block_sync();
        load(c0 + SL);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int r = 16 * (n * WAVES + w) + l16;
            const Frag<float> fs = frag8(lds.in.s + r * LS + 2 * g4), fa = frag8(lds.in.a + r * LS + 2 * g4);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int at = (16 * t + l16) * LS + 2 * g4;
                dyS[n][t] = mma(frag8(lds.in.dy + at), fs, dyS[n][t]);
                dRS[n][t] = mma(frag8(lds.in.dr + at), fs, dRS[n][t]);
                UA[n][t] = mma(frag8(lds.in.u + at), fa, UA[n][t]);
            }
        }
#pragma unroll
        for (int x = 0; x < PAIRS; ++x) {
            const int u = x * WAVES + w, f = u < TILES ? u : u - TILES;
            if (u >= 2 * TILES) continue;
            const int it = (f > 0) + (f > 2) + (f > 5), jt = f - it * (it + 1) / 2;
            const float *rows = u < TILES ? lds.in.dy : lds.in.dr;
            pair[x] = mma(frag8(rows + (16 * it + l16) * LS + 2 * g4), frag8(lds.in.u + (16 * jt + l16) * LS + 2 * g4),
                          pair[x]);
        }
        block_sync();
    }
    const Decays<CB> &d = lds.dec;
    // dP and dM + dM^T, whole, and N's sums by rows and columns
#pragma unroll
    for (int x = 0; x < PAIRS; ++x) {
        const int u = x * WAVES + w, f = u < TILES ? u : u - TILES;
        if (u >= 2 * TILES) continue;
        const bool isP = u < TILES;
        const int it = (f > 0) + (f > 2) + (f > 5), jt = f - it * (it + 1) / 2;
        const float *rows = isP ? lds.q : lds.k;
        f32x4 s = {};
#pragma unroll
        for (int m = 0; m < KS; ++m)
            s = mma(frag8(rows + (16 * it + l16) * LK + 32 * m + 2 * g4), frag8(lds.k + (16 * jt + l16) * LK + 32 * m + 2 * g4),
                    s);
        const f32x4 ih = *reinterpret_cast<const f32x4 *>(d.hi + 16 * it + g4);
        const f32x4 il = *reinterpret_cast<const f32x4 *>(d.lo + 16 * it + g4);
        const int j = 16 * jt + l16;
        const float jh = d.hi[j], jl = d.lo[j];
        float by_col = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * it + g4 + e;
            float v = pair[x][e] * __expf((ih[e] - jh) + (il[e] - jl));
            if (isP ? j > i : j >= i) v = 0.f;
            if (!isP) v = -v;
            float n = j < i ? v * s[e] : 0.f;   // the diagonal depends on no decay
            by_col += n;
            n = sum16(n);
            if (l16 == 0) lds.rowsum[u][g4 + e] = n;
            if (isP) {
                lds.pair.dp[i * LP + j] = v;
                if (it != jt) lds.pair.dp[j * LP + i] = 0.f;
            } else if (j <= i) {
                lds.pair.dm[i * LP + j] = v;
                lds.pair.dm[j * LP + i] = v;
            }
        }
        by_col += __shfl_xor(by_col, 16);
        by_col += __shfl_xor(by_col, 32);
        if (lane < 16) lds.colsum[u][lane] = by_col;
    }
    block_sync();
    float sums[3][TT][4] = {};   // of f's two terms and of e, over this lane's columns
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        const int c16 = 16 * (n * WAVES + w), col = c16 + l16;
        Frag<float> kc[TS], qc[TS];
#pragma unroll
        for (int s = 0; s < TS; ++s) {
            kc[s] = frag_col<LK, false>(lds.k + 32 * s * LK, c16, lane);
            qc[s] = frag_col<LK, false>(lds.q + 32 * s * LK, c16, lane);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const f32x4 eb = *reinterpret_cast<const f32x4 *>(d.in + 16 * t + g4);
            const f32x4 wb = *reinterpret_cast<const f32x4 *>(d.out + 16 * t + g4);
            f32x4 gq = dyS[n][t] * eb, gr = dRS[n][t] * eb, gu = UA[n][t] * wb;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float qv = lds.q[(16 * t + g4 + e) * LK + col], kv = lds.k[(16 * t + g4 + e) * LK + col];
                sums[0][t][e] += qv * gq[e];
                sums[1][t][e] += kv * gr[e];
                sums[2][t][e] += kv * gu[e];
            }
            f32x4 gk = gu - gr;
            const auto row_frag = [&](const float *m, int s) {
                Frag<float> f;
                const float *at = m + (16 * t + l16) * LP + 32 * s + g4;
                frag_acc(f, *reinterpret_cast<const f32x4 *>(at), *reinterpret_cast<const f32x4 *>(at + 16));
                return f;
            };
#pragma unroll
            for (int s = 0; s < TS; ++s) {
                if (s <= t / 2) gq = mma(row_frag(lds.pair.dp, s), kc[s], gq);
                if (s >= t / 2) gk = mma(frag_col<LP, false>(lds.pair.dp + 32 * s * LP, 16 * t, lane), qc[s], gk);
                gk = mma(row_frag(lds.pair.dm, s), kc[s], gk);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 16 * t + g4 + e;
                if (row >= p.rows || col >= a.dk) continue;
                if (a.G == a.H) {
                    const int64_t at = ((row0 + row) * a.G + g) * a.dk + col;
                    static_cast<E *>(a.dq)[at] = from_f<E>(gq[e]);
                    static_cast<E *>(a.dk_out)[at] = from_f<E>(gk[e]);
                } else {
                    const int64_t at = ((row0 + row) * a.H + h) * a.dk + col;
                    a.dq_head[at] = gq[e];
                    a.dk_head[at] = gk[e];
                }
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 3; ++x)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float s = sum16(sums[x][t][e]);
                if (l16 == 0) lds.sums[x][w][16 * t + g4 + e] = s;
            }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) dot += __shfl_xor(dot, o);
    if (lane == 0) lds.dot[w] = dot;
#pragma unroll
    for (int u = 0; u < RPER; ++u) {
        const int e = u * PT + tid, row = e / 8;
#pragma unroll
        for (int o = 1; o < 8; o *= 2) dbeta[u] += __shfl_xor(dbeta[u], o);
        if (e % 8 == 0 && (RP % PT == 0 || e < RP) && row < p.rows) a.dbeta[(row0 + row) * a.H + h] = dbeta[u];
    }
    block_sync();
    if (w == 0) {
        double f = 0., e = 0., all = 0.;
        if (lane < CB) {
#pragma unroll
            for (int x = 0; x < WAVES; ++x) {
                f += (double)lds.sums[0][x][lane] - (double)lds.sums[1][x][lane];
                e += (double)lds.sums[2][x][lane];
            }
            const int t = lane / 16;   // N's tiles of row block t, and of column block t
#pragma unroll
            for (int x = 0; x < TILES; ++x) {
                const int it = (x > 0) + (x > 2) + (x > 5), jt = x - it * (it + 1) / 2;
                if (it == t) e -= (double)lds.rowsum[x][lane % 16] + (double)lds.rowsum[TILES + x][lane % 16];
                if (jt == t) e += (double)lds.colsum[x][lane % 16] + (double)lds.colsum[TILES + x][lane % 16];
            }
        }
#pragma unroll
        for (int x = 0; x < WAVES; ++x) all += (double)lds.dot[x];
        // the rows before, and the rows from its own on: no sum is taken back
        const double before = __shfl_up(e, 1);
        const double pre = scan64(lane > 0 ? before : 0.), post = __shfl(scan64(__shfl(f, 63 - lane)), 63 - lane);
        const double r = post + pre + (double)d.all * all;
        if (lane < p.rows && lane < CB) a.dla_rows[(row0 + lane) * a.H + h] = (float)r;
    }
}

// The same for bfloat16 calls with dk up to 128, on bf16 MFMA: whatever enters
// dlog_decay or dbeta as a sum of three bfloat16 numbers, split once on its way
// to LDS (six products for two such operands, the ones of 2^-24 and less left
// out), dP and dM, which meet K and Q for dQ and dK alone, of two.
//
// S, A, dR, U and dY pass through LDS 32 columns at a time, S and A one after
// the other in one place, and q and k take it over after them, so that two
// blocks share a CU and fill each other's waits (one block of eight waves with
// a place for each took 272 us for the training case, this 243; its waves wait
// in 0.6 of their cycles still, for barriers and loads.  For dk over 64 it
// spills 37 registers as it is; loads further ahead spill more: 307).
template <int KP>
struct GradsBfLds {
    static constexpr int CB = 64, WAVES = 4, SL = 32, TT = 4, TILES = 10;
    static constexpr int LK = KP + 16, LS = SL + 16, LP = CB + 16, NS = KP / 16 / WAVES;
    union {
        struct {
            alignas(16) bf16 dy[CB * LS], u[3][CB * LS], dr[3][CB * LS], s[3][KP * LS];
        } in;
        struct {
            alignas(16) bf16 q[CB * LK], k[CB * LK];
            union {
                struct {
                    alignas(16) bf16 dp[2][CB * LP], dm[2][CB * LP];
                };
                float sums[3][WAVES][CB];   // after them
            };
            float rowsum[2 * TILES][16], colsum[2 * TILES][16];
        } pair;
    };
    Decays<CB> dec;
    alignas(16) float beta[CB];
    float dot[WAVES];
};

template <int KP, bool VEC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_delta_grads_bf(DeltaBackArgs a)
{
    typedef GradsBfLds<KP> Lds;
    typedef bf16 E;
    constexpr int CB = Lds::CB, WAVES = Lds::WAVES, SL = Lds::SL, TT = Lds::TT, TILES = Lds::TILES, NS = Lds::NS;
    constexpr int LK = Lds::LK, LS = Lds::LS, LP = Lds::LP, PT = 256, KS = KP / 32, RROWS = PT / 8;
    constexpr int TS = CB / 32, PAIRS = (2 * TILES + WAVES - 1) / WAVES, RPER = CB / RROWS, SPER = KP / RROWS;
    __shared__ Lds lds;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int h = blockIdx.x % a.H;
    int id = blockIdx.x / a.H;
    Place p;
    if (!find(a, id, p) || p.rows <= 0) return;
    const int g = h / (a.H / a.G);
    const int first = p.begin - p.s * CB;
    const int64_t row0 = p.begin, idw = chunk_number(p.n, first, p.s * CB, CW);
    const float *srec = a.srec + ((int64_t)id * a.H + h) * a.dk * a.dvp;
    const float *arec = a.arec + ((int64_t)id * a.H + h) * a.dk * a.dvp;
    const int64_t rec_step = (int64_t)a.H * CW * a.dvp;
    const float *zrec = a.zrec + (idw * a.H + h) * CW * a.dvp, *grec = a.grec + (idw * a.H + h) * CW * a.dvp;
    const E *dy = static_cast<const E *>(a.dy) + row0 * a.st.y_t + h * a.st.y_h;

    // a thread's four columns, of RPER rows of Z and dG and of SPER rows of S and A
    const int row = tid / 8, col8 = tid % 8 * 4;
    Tile<E, CB, SL, PT> ty;
    f32x4 tz[RPER], tg[RPER], ts[SPER], ta[SPER];
    const auto load = [&](int c0) {
        ty.template fetch<VEC>(dy + c0, a.st.y_t, c0 < a.dv ? p.rows : 0, min(SL, a.dv - c0), tid);
        const int col = c0 + col8;
#pragma unroll
        for (int u = 0; u < RPER; ++u) {
            const int r = u * RROWS + row;
            const bool on = r < p.rows && col < a.dvp;
            const int64_t at = r / CW * rec_step + (int64_t)(r % CW) * a.dvp + col;
            tz[u] = on ? *reinterpret_cast<const f32x4 *>(zrec + at) : f32x4{};
            tg[u] = on ? *reinterpret_cast<const f32x4 *>(grec + at) : f32x4{};
        }
#pragma unroll
        for (int u = 0; u < SPER; ++u) {
            const int r = u * RROWS + row;
            const bool live = r < a.dk && col < a.dvp;
            ts[u] = live ? *reinterpret_cast<const f32x4 *>(srec + (int64_t)r * a.dvp + col) : f32x4{};
            ta[u] = live ? *reinterpret_cast<const f32x4 *>(arec + (int64_t)r * a.dvp + col) : f32x4{};
        }
    };
    const auto put = [&](auto &to, int r, f32x4 x) {
        bf16x4 parts[3];
        split4(parts, x);
#pragma unroll
        for (int u = 0; u < 3; ++u) *reinterpret_cast<bf16x4 *>(to[u] + r * LS + col8) = parts[u];
    };
    load(0);
    {
        const bool on = lane < p.rows;
        if (w == 0) make_decays(lds.dec, on ? a.la[(a.la_t ? (row0 + lane) * a.la_t : 0) + h] : 0.f, lane);
        if (w == 1) lds.beta[lane] = on ? a.beta[(row0 + lane) * a.beta_t + h] : 0.f;
    }
    block_sync();
    f32x4 dyS[NS][TT] = {}, dRS[NS][TT] = {}, UA[NS][TT] = {}, pair[PAIRS] = {};
    float dbeta[RPER] = {}, dot = 0.f;
    for (int c0 = 0; c0 < a.dv; c0 += SL) {
        ty.template place<VEC, LS>(lds.in.dy, dy + c0, a.st.y_t, min(SL, a.dv - c0), tid);
#pragma unroll
        for (int u = 0; u < RPER; ++u) {
            const int r = u * RROWS + row;
            const float bt = lds.beta[r];
            const f32x4 dr = tg[u] * bt;
#pragma unroll
            for (int i = 0; i < 4; ++i) dbeta[u] += tg[u][i] * tz[u][i];
            put(lds.in.u, r, tz[u] * bt);
            put(lds.in.dr, r, dr);
            if (r < p.rows) {
                E *to = static_cast<E *>(a.dv_out) + ((row0 + r) * a.H + h) * a.dv + c0 + col8;
                if (VEC && c0 + col8 < a.dv) {
                    *reinterpret_cast<bf16x4 *>(to) = __builtin_convertvector(dr, bf16x4);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c0 + col8 + i < a.dv) to[i] = from_f<E>(dr[i]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < SPER; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dot += ts[u][i] * ta[u][i];
            put(lds.in.s, u * RROWS + row, ts[u]);
        }
        block_sync();
        {
            Frag<bf16> fs[NS][3];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int u = 0; u < 3; ++u) fs[n][u] = frag8(lds.in.s[u] + (16 * (n * WAVES + w) + l16) * LS + 2 * g4);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int at = (16 * t + l16) * LS + 2 * g4;
                const Frag<bf16> fy = frag8(lds.in.dy + at);
                Frag<bf16> fr[3];
#pragma unroll
                for (int u = 0; u < 3; ++u) fr[u] = frag8(lds.in.dr[u] + at);
#pragma unroll
                for (int o = 2; o >= 0; --o)   // the small products first
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        dyS[n][t] = mma(fy, fs[n][o], dyS[n][t]);
#pragma unroll
                        for (int u = 0; u <= o; ++u) dRS[n][t] = mma(fr[u], fs[n][o - u], dRS[n][t]);
                    }
            }
        }
        // U dY^T and U dR^T: lane holds rows j of U, column i of dY or dR
#pragma unroll
        for (int x = 0; x < PAIRS; ++x) {
            const int u = x * WAVES + w, f = u < TILES ? u : u - TILES;
            if (u >= 2 * TILES) continue;
            const int it = (f > 0) + (f > 2) + (f > 5), jt = f - it * (it + 1) / 2;
            const int ai = (16 * it + l16) * LS + 2 * g4, aj = (16 * jt + l16) * LS + 2 * g4;
            if (u < TILES) {
                const Frag<bf16> fy = frag8(lds.in.dy + ai);
#pragma unroll
                for (int o = 2; o >= 0; --o) pair[x] = mma(frag8(lds.in.u[o] + aj), fy, pair[x]);
            } else {
                Frag<bf16> fr[3], fu[3];
#pragma unroll
                for (int o = 0; o < 3; ++o) {
                    fr[o] = frag8(lds.in.dr[o] + ai);
                    fu[o] = frag8(lds.in.u[o] + aj);
                }
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int z = 0; z <= o; ++z) pair[x] = mma(fu[z], fr[o - z], pair[x]);
            }
        }
        block_sync();
#pragma unroll
        for (int u = 0; u < SPER; ++u) put(lds.in.s, u * RROWS + row, ta[u]);   // A in S's place
        block_sync();
        load(c0 + SL);
        {
            Frag<bf16> fa[NS][3];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int u = 0; u < 3; ++u) fa[n][u] = frag8(lds.in.s[u] + (16 * (n * WAVES + w) + l16) * LS + 2 * g4);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                Frag<bf16> fu[3];
#pragma unroll
                for (int u = 0; u < 3; ++u) fu[u] = frag8(lds.in.u[u] + (16 * t + l16) * LS + 2 * g4);
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int u = 0; u <= o; ++u)
#pragma unroll
                        for (int n = 0; n < NS; ++n) UA[n][t] = mma(fu[u], fa[n][o - u], UA[n][t]);
            }
        }
        block_sync();
    }
    {
        Tile<E, CB, KP, PT> tk, tq;
        const E *k = static_cast<const E *>(a.k) + row0 * a.st.k_t + g * a.st.k_g;
        const E *q = static_cast<const E *>(a.q) + row0 * a.st.q_t + g * a.st.q_g;
        tk.template fetch<VEC>(k, a.st.k_t, p.rows, a.dk, tid);
        tq.template fetch<VEC>(q, a.st.q_t, p.rows, a.dk, tid);
        tk.template place<VEC, LK>(lds.pair.k, k, a.st.k_t, a.dk, tid);
        tq.template place<VEC, LK>(lds.pair.q, q, a.st.q_t, a.dk, tid);
    }
    block_sync();
    const Decays<CB> &d = lds.dec;
    // dP and dM below the diagonal, their columns in the order in which the
    // products take them, and N's sums by rows and columns
#pragma unroll
    for (int x = 0; x < PAIRS; ++x) {
        const int u = x * WAVES + w, f = u < TILES ? u : u - TILES;
        if (u >= 2 * TILES) continue;
        const bool isP = u < TILES;
        const int it = (f > 0) + (f > 2) + (f > 5), jt = f - it * (it + 1) / 2;
        const bf16 *rows = isP ? lds.pair.q : lds.pair.k;
        f32x4 s = {};
#pragma unroll
        for (int m = 0; m < KS; ++m)
            s = mma(frag8(lds.pair.k + (16 * jt + l16) * LK + 32 * m + 2 * g4), frag8(rows + (16 * it + l16) * LK + 32 * m + 2 * g4),
                    s);
        const f32x4 jh = *reinterpret_cast<const f32x4 *>(d.hi + 16 * jt + g4);
        const f32x4 jl = *reinterpret_cast<const f32x4 *>(d.lo + 16 * jt + g4);
        const int i = 16 * it + l16;
        const float ih = d.hi[i], il = d.lo[i];
        float by_row = 0.f;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 16 * jt + g4 + e;
            v[e] = pair[x][e] * __expf((ih - jh[e]) + (il - jl[e]));
            if (isP ? j > i : j >= i) v[e] = 0.f;
            if (!isP) v[e] = -v[e];
            float n = j < i ? v[e] * s[e] : 0.f;   // the diagonal depends on no decay
            by_row += n;
            n = sum16(n);
            if (l16 == 0) lds.pair.colsum[u][g4 + e] = n;
        }
        by_row += __shfl_xor(by_row, 16);
        by_row += __shfl_xor(by_row, 32);
        if (lane < 16) lds.pair.rowsum[u][lane] = by_row;
        bf16x4 parts[2];
        split4(parts, v);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            bf16 *to = (isP ? lds.pair.dp[z] : lds.pair.dm[z]) + i * LP + 32 * (jt / 2) + 2 * g4;
            *reinterpret_cast<bf16x4 *>(to + 4 * (jt % 2)) = parts[z];
            // right of a tile on the diagonal, what the same pieces hold
            if (it == jt && it % 2 == 0) *reinterpret_cast<bf16x4 *>(to + 4) = bf16x4{};
        }
    }
    block_sync();
    float sums[3][TT][4] = {};   // of f's two terms and of e, over this lane's columns
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        const int c16 = 16 * (n * WAVES + w), col = c16 + l16;
        Frag<bf16> kc[TS], qc[TS];
#pragma unroll
        for (int s = 0; s < TS; ++s) {
            kc[s] = frag_col<LK, false>(lds.pair.k + 32 * s * LK, c16, lane);
            qc[s] = frag_col<LK, false>(lds.pair.q + 32 * s * LK, c16, lane);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const f32x4 eb = *reinterpret_cast<const f32x4 *>(d.in + 16 * t + g4);
            const f32x4 wb = *reinterpret_cast<const f32x4 *>(d.out + 16 * t + g4);
            f32x4 gq = dyS[n][t] * eb, gr = dRS[n][t] * eb, gu = UA[n][t] * wb;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = (16 * t + g4 + e) * LK + col;
                const float qv = to_f(lds.pair.q[at]), kv = to_f(lds.pair.k[at]);
                sums[0][t][e] += qv * gq[e];
                sums[1][t][e] += kv * gr[e];
                sums[2][t][e] += kv * gu[e];
            }
            f32x4 gk = gu - gr;
            // rows of dP and dM, and of their transposes
#pragma unroll
            for (int s = 0; s < TS; ++s)
#pragma unroll
                for (int z = 1; z >= 0; --z) {
                    if (s <= t / 2) {
                        const int at = (16 * t + l16) * LP + 32 * s + 2 * g4;
                        gq = mma(frag8(lds.pair.dp[z] + at), kc[s], gq);
                        gk = mma(frag8(lds.pair.dm[z] + at), kc[s], gk);
                    }
                    if (s >= t / 2) {
                        const int c = 32 * (t / 2) + 4 * (t % 2);
                        gk = mma(frag_col<LP, true>(lds.pair.dp[z] + 32 * s * LP, c, lane), qc[s], gk);
                        gk = mma(frag_col<LP, true>(lds.pair.dm[z] + 32 * s * LP, c, lane), kc[s], gk);
                    }
                }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * t + g4 + e;
                if (r >= p.rows || col >= a.dk) continue;
                if (a.G == a.H) {
                    const int64_t at = ((row0 + r) * a.G + g) * a.dk + col;
                    static_cast<E *>(a.dq)[at] = from_f<E>(gq[e]);
                    static_cast<E *>(a.dk_out)[at] = from_f<E>(gk[e]);
                } else {
                    const int64_t at = ((row0 + r) * a.H + h) * a.dk + col;
                    a.dq_head[at] = gq[e];
                    a.dk_head[at] = gk[e];
                }
            }
        }
    }
    block_sync();   // the sums take the place of dP and dM
#pragma unroll
    for (int x = 0; x < 3; ++x)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float s = sum16(sums[x][t][e]);
                if (l16 == 0) lds.pair.sums[x][w][16 * t + g4 + e] = s;
            }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) dot += __shfl_xor(dot, o);
    if (lane == 0) lds.dot[w] = dot;
#pragma unroll
    for (int u = 0; u < RPER; ++u) {
        const int r = u * RROWS + row;
#pragma unroll
        for (int o = 1; o < 8; o *= 2) dbeta[u] += __shfl_xor(dbeta[u], o);
        if (col8 == 0 && r < p.rows) a.dbeta[(row0 + r) * a.H + h] = dbeta[u];
    }
    block_sync();
    if (w == 0) {
        double f = 0., e = 0., all = 0.;
#pragma unroll
        for (int x = 0; x < WAVES; ++x) {
            f += (double)lds.pair.sums[0][x][lane] - (double)lds.pair.sums[1][x][lane];
            e += (double)lds.pair.sums[2][x][lane];
            all += (double)lds.dot[x];
        }
        const int t = lane / 16;   // N's tiles of row block t, and of column block t
#pragma unroll
        for (int x = 0; x < TILES; ++x) {
            const int it = (x > 0) + (x > 2) + (x > 5), jt = x - it * (it + 1) / 2;
            if (it == t) e -= (double)lds.pair.rowsum[x][lane % 16] + (double)lds.pair.rowsum[TILES + x][lane % 16];
            if (jt == t) e += (double)lds.pair.colsum[x][lane % 16] + (double)lds.pair.colsum[TILES + x][lane % 16];
        }
        // the rows before, and the rows from its own on: no sum is taken back
        const double before = __shfl_up(e, 1);
        const double pre = scan64(lane > 0 ? before : 0.), post = __shfl(scan64(__shfl(f, 63 - lane)), 63 - lane);
        const double r = post + pre + (double)d.all * all;
        if (lane < p.rows) a.dla_rows[(row0 + lane) * a.H + h] = (float)r;
    }
}

// dq and dk of the heads of a group added up in their order: a thread for four
// columns (V = 4) or one, of the rows that belong to a sequence.
template <typename E, int V>
__global__ __launch_bounds__(256) void k_delta_group_sum(DeltaBackArgs a)
{
    const int per = a.dk / V;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = a.T;
    if (e >= rows * a.G * per) return;
    const int64_t t = e / (a.G * per);
    const int g = (int)(e / per % a.G), c = (int)(e % per) * V, rep = a.H / a.G;
    int b0, b1, e0, e1;
    rows_of(a, 0, b0, e0);
    rows_of(a, a.N - 1, b1, e1);
    if (t < b0 || t >= e1) return;
    typedef Vec<float, V> F;
    const int64_t from = (t * a.H + (int64_t)g * rep) * a.dk + c, to = (t * a.G + g) * a.dk + c;
    F q = {}, k = {};
    for (int h = 0; h < rep; ++h) {
        const F x = *reinterpret_cast<const F *>(a.dq_head + from + (int64_t)h * a.dk);
        const F y = *reinterpret_cast<const F *>(a.dk_head + from + (int64_t)h * a.dk);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            q.v[i] += x.v[i];
            k.v[i] += y.v[i];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        static_cast<E *>(a.dq)[to + i] = from_f<E>(q.v[i]);
        static_cast<E *>(a.dk_out)[to + i] = from_f<E>(k.v[i]);
    }
}

// dlog_decay of a head: the sum over all rows, in 64 bits and a fixed order.
__global__ __launch_bounds__(1024) void k_delta_decay_sum(DeltaBackArgs a)
{
    __shared__ double part[16];
    const int h = blockIdx.x;
    int b0, b1, e0, e1;
    rows_of(a, 0, b0, e0);
    rows_of(a, a.N - 1, b1, e1);
    double s = 0.;
    for (int64_t t = b0 + (int)threadIdx.x; t < e1; t += 1024) s += (double)a.dla_rows[t * a.H + h];
#pragma unroll
    for (int o = 1; o < 64; o *= 2) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.;
        for (int i = 0; i < 16; ++i) all += part[i];
        a.dla[h] = (float)all;
    }
}

// A head's dlog_decay where no sequence has a row.
__global__ __launch_bounds__(256) void k_delta_no_rows(float *dla, int H)
{
    const int h = blockIdx.x * 256 + threadIdx.x;
    if (h < H) dla[h] = 0.f;
}

// ---- host side

struct DeltaBackPlan {
    int cb = 64, dvp = 0;
    int64_t walk_ids = 0, ids = 0;
    size_t inv = 0, zrec = 0, grec = 0, srec = 0, arec = 0, dq = 0, dk = 0, dla = 0, total = 0;
};

static DeltaBackPlan plan_back(const lin_shape &s, int dtype, bool by_row)
{
    DeltaBackPlan P;
    P.cb = s.dk > 128 ? 32 : 64;
    P.dvp = (int)((s.dv + 3) / 4 * 4);
    P.walk_ids = s.T / CW + s.N;
    P.ids = s.T / P.cb + s.N;
    size_t o = 0;
    const auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    const size_t image = dtype == LAYER_BF16 ? Pieces<bf16>::BYTES : Pieces<float>::BYTES;
    const size_t rows = (size_t)(P.walk_ids * s.H * CW * P.dvp) * 4, state = (size_t)(P.ids * s.H * s.dk * P.dvp) * 4;
    P.inv = take((size_t)(P.walk_ids * s.H) * 3 * image);
    P.zrec = take(rows);
    P.grec = take(rows);
    P.srec = take(state);
    P.arec = take(state);
    const size_t heads = s.G == s.H ? 0 : (size_t)(s.T * s.H * s.dk) * 4;
    P.dq = take(heads);
    P.dk = take(heads);
    P.dla = take(by_row ? 0 : (size_t)(s.T * s.H) * 4);
    P.total = o;
    return P;
}

// The workspace for any element type and form of the log decays.
static size_t back_workspace(const lin_shape &s)
{
    if (s.T == 0 || s.N == 0) return 0;
    const size_t a = plan_back(s, LAYER_BF16, false).total, b = plan_back(s, LAYER_F32, false).total;
    return a > b ? a : b;
}

template <typename E, int KP, bool VEC>
static int run_back(DeltaBackArgs &a, const DeltaBackPlan &P, hipStream_t st)
{
    if (a.T > 0) {
        DeltaBackArgs c = a;
        c.seg = CW;
        c.ids = (int)P.walk_ids;
        k_delta_back_inverse<E, KP, VEC><<<dim3((unsigned)(P.walk_ids * a.H)), dim3(256), 0, st>>>(c);
    }
    k_delta_walk<E, KP, VEC><<<dim3((unsigned)((int64_t)2 * a.N * a.H * a.tiles)), dim3(512), 0, st>>>(a);
    if (a.T == 0) return launch_status();
    {
        DeltaBackArgs c = a;
        c.seg = GradsLds<KP>::CB;
        c.ids = (int)P.ids;
        const dim3 grid((unsigned)(P.ids * a.H));
        if constexpr (std::is_same<E, bf16>::value && KP <= 128)
            k_delta_grads_bf<KP, VEC><<<grid, dim3(256), 0, st>>>(c);
        else
            k_delta_grads<E, KP, VEC><<<grid, dim3(64 * GradsLds<KP>::WAVES), 0, st>>>(c);
    }
    if (a.G != a.H) {
        const int v = a.dk % 4 == 0 ? 4 : 1;
        const int64_t n = (int64_t)a.T * a.G * (a.dk / v);
        const dim3 grid((unsigned)((n + 255) / 256));
        if (v == 4)
            k_delta_group_sum<E, 4><<<grid, dim3(256), 0, st>>>(a);
        else
            k_delta_group_sum<E, 1><<<grid, dim3(256), 0, st>>>(a);
    }
    if (a.dla) k_delta_decay_sum<<<dim3((unsigned)a.H), dim3(1024), 0, st>>>(a);
    return launch_status();
}

template <typename E, bool VEC>
static int dispatch_back(DeltaBackArgs &a, const DeltaBackPlan &P, hipStream_t st)
{
    if (a.dk > 128) return run_back<E, 256, VEC>(a, P, st);
    if (a.dk > 64) return run_back<E, 128, VEC>(a, P, st);
    return run_back<E, 64, VEC>(a, P, st);
}

}  // namespace layer

using namespace layer;

extern "C" size_t delta_bwd_workspace_size(const lin_shape *shape)
{
    if (check_delta_bwd(shape) != SSD_OK) return (size_t)-1;
    return back_workspace(*shape);
}

extern "C" int delta_bwd(const lin_shape *shape, int dtype, const lin_strides *strides, const void *q, const void *k,
                         const void *v, const float *log_decay, int64_t decay_stride, const float *beta,
                         int64_t beta_stride, const int32_t *cu_seqlens, const float *states, const void *dy,
                         const float *dstates_last, void *dq, void *dk, void *dv, float *dlog_decay, int decay_by_row,
                         float *dbeta, float *dstates, int clear, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    int rc = check_delta_bwd(shape);
    if (rc == SSD_OK) rc = check_dtype(dtype);
    if (rc != SSD_OK) return rc;
    const lin_shape &s = *shape;
    DeltaBackArgs a;
    rc = resolve_strides(shape, strides, &a.st, s.T, false);
    if (rc != SSD_OK) return rc;
    if (decay_stride < 0 || decay_stride >= kMaxCount || beta_stride < 0 || beta_stride >= kMaxCount)
        return SSD_ERR_SHAPE;
    if (s.N == 0 && decay_by_row) return SSD_OK;
    if (s.N > 0 && !cu_seqlens) return SSD_ERR_NULL;
    if (!dlog_decay && !(decay_by_row && s.T == 0)) return SSD_ERR_NULL;
    if (s.N > 0 && s.T > 0 && (!q || !k || !v || !log_decay || !beta || !dy || !dq || !dk || !dv || !dbeta))
        return SSD_ERR_NULL;
    const unsigned e = dtype_size(dtype);
    for (const void *x : {q, k, v, dy, (const void *)dq, (const void *)dk, (const void *)dv})
        if (misaligned(x, e)) return SSD_ERR_ALIGN;
    for (const void *x : {(const void *)log_decay, (const void *)beta, (const void *)cu_seqlens, (const void *)states,
                          (const void *)dstates_last, (const void *)dlog_decay, (const void *)dbeta,
                          (const void *)dstates})
        if (misaligned(x, 4)) return SSD_ERR_ALIGN;
    const DeltaBackPlan P = plan_back(s, dtype, decay_by_row != 0);
    const size_t need = back_workspace(s);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (need > 0 && !workspace) return SSD_ERR_NULL;
    if (need > 0 && misaligned(workspace, 16)) return SSD_ERR_ALIGN;
    char *ws = static_cast<char *>(workspace);
    const auto at = [&](size_t o) { return need > 0 ? reinterpret_cast<float *>(ws + o) : nullptr; };
    a.q = q;
    a.k = k;
    a.v = v;
    a.la = log_decay;
    a.la_t = decay_stride;
    a.beta = beta;
    a.beta_t = beta_stride;
    a.cu = cu_seqlens;
    a.slots = a.carry = nullptr;
    a.states = const_cast<float *>(states);
    a.y = nullptr;
    a.ends = a.segdec = nullptr;
    a.inv = need > 0 ? ws + P.inv : nullptr;
    a.dy = dy;
    a.dlast = dstates_last;
    a.zrec = at(P.zrec);
    a.grec = at(P.grec);
    a.srec = at(P.srec);
    a.arec = at(P.arec);
    a.dq_head = at(P.dq);
    a.dk_head = at(P.dk);
    a.dq = dq;
    a.dk_out = dk;
    a.dv_out = dv;
    a.dla = decay_by_row ? nullptr : dlog_decay;
    a.dla_rows = decay_by_row ? dlog_decay : at(P.dla);
    a.dbeta = dbeta;
    a.dfirst = dstates;
    a.dvp = P.dvp;
    a.cb = P.cb;
    a.clear = clear != 0;
    a.T = (int)s.T;
    a.N = (int)s.N;
    a.G = (int)s.G;
    a.H = (int)s.H;
    a.dk = (int)s.dk;
    a.dv = (int)s.dv;
    a.nslots = (int)s.N;
    a.tiles = (a.dv + 63) / 64;
    a.seg = 0;
    a.ids = (int)s.N;
    a.shift = -1;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (s.N == 0 || s.T == 0) {   // no sequence has a row: zeros, and the last states' gradients
        if (a.dla) k_delta_no_rows<<<dim3((unsigned)((s.H + 255) / 256)), dim3(256), 0, st>>>(a.dla, (int)s.H);
        if (s.N == 0) return launch_status();
        a.dla = nullptr;
    }
    const auto rows16 = [&](const void *ptr, int64_t row, int64_t head, int64_t d) {
        return !misaligned(ptr, 16) && row * e % 16 == 0 && head * e % 16 == 0 && d * e % 16 == 0 && row >= d;
    };
    const bool vec = rows16(q, a.st.q_t, a.st.q_g, s.dk) && rows16(k, a.st.k_t, a.st.k_g, s.dk) &&
                     rows16(v, a.st.v_t, a.st.v_h, s.dv) && rows16(dy, a.st.y_t, a.st.y_h, s.dv) &&
                     !misaligned(dv, 16);
    if (dtype == LAYER_BF16) return vec ? dispatch_back<bf16, true>(a, P, st) : dispatch_back<bf16, false>(a, P, st);
    if (dtype == LAYER_F16) return vec ? dispatch_back<f16, true>(a, P, st) : dispatch_back<f16, false>(a, P, st);
    return vec ? dispatch_back<float, true>(a, P, st) : dispatch_back<float, false>(a, P, st);
}
