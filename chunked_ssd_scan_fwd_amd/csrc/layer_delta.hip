// The gated delta rule over a packed batch and a pool of states, in chunks,
// and its one-token step.
#include "layer_delta.h"

namespace layer {

// One segment of a sequence for one head and VT columns, with the state in
// registers, as the scalar-decay scan's prefill walks it: four waves hold S,
// 16 NT columns each, and make U and Y; four fetch the next chunk and form its
// scores.  Neither S nor U crosses waves: K S comes out of the accumulators
// as the operand that T takes, and U as the one that P and K^T take.
//
// For bfloat16 inputs everything that reaches the state keeps float32's
// accuracy: S, T, the residual V - diag(e^b) K S and U enter their products as
// sums of three bfloat16 numbers (six products for two such operands, the ones
// of 2^-24 and less left out).  In y, S and the scores P enter as one, U as
// two.
template <typename E, int KP, int VT, int C>
struct DeltaLds {
    typedef typename std::conditional<std::is_same<E, bf16>::value, bf16, float>::type L;
    typedef Pieces<L, C> PC;
    static constexpr int PAD = sizeof(L) == 2 ? 16 : 4;
    static constexpr int LK = KP + PAD, LV = VT + PAD;
    static constexpr int PBYTES = PC::BYTES / PC::PARTS;
    static constexpr bool T_HERE = C == 64;   // else the waves read T from memory themselves
    L q[2][C * LK], k[2][C * LK], v[2][C * LV];
    char p[2][PBYTES], t[2][T_HERE ? PC::BYTES : 16];
    Decays<C> dec[3];
};

template <typename E, int KP, int VT>
struct DeltaPerCu {
    static constexpr int n = VT == 64 && KP <= 128 && std::is_same<E, bf16>::value ? 2 : 1;
    static constexpr int C = n == 2 || sizeof(E) == 4 || KP > 128 || !std::is_same<E, bf16>::value ? 32 : 64;
};

template <typename E, int KP, int VT, int C, bool VEC>
__global__ __launch_bounds__(512)
__attribute__((amdgpu_waves_per_eu(2 * DeltaPerCu<E, KP, VT>::n, 2 * DeltaPerCu<E, KP, VT>::n)))
void k_delta_chunks(DeltaArgs a)
{
    typedef DeltaLds<E, KP, VT, C> Lds;
    typedef typename Lds::L L;
    typedef Pieces<L, C> PC;
    constexpr int LK = Lds::LK, LV = Lds::LV;
    constexpr int NT = VT / 64, MT = KP / 16, TT = C / 16, KS = KP / 32, TS = C / 32;
    constexpr int PARTS = PC::PARTS, YU = PARTS == 3 ? 2 : 1;
    constexpr int PT = 256;   // threads that fetch
    __shared__ __align__(16) Lds lds;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int tile = blockIdx.x % a.tiles, h = blockIdx.x / a.tiles % a.H;
    int id = blockIdx.x / (a.tiles * a.H);
    Place p;
    if (!find(a, id, p)) return;
    const int g = h / (a.H / a.G), c0 = tile * VT, cols = min(VT, a.dv - c0);
    E *y = static_cast<E *>(a.y) + p.begin * a.st.y_t + h * a.st.y_h + c0;
    if (p.bad) {
        for (int64_t e = threadIdx.x; e < (int64_t)p.rows * VT; e += 512)
            if (e % VT < cols) y[e / VT * a.st.y_t + e % VT] = from_f<E>(__builtin_nanf(""));
        return;
    }
    const int chunks = (p.rows + C - 1) / C;
    const int first = p.begin - p.s * a.seg;   // of the sequence
    const char *inv = a.inv + ((int64_t)chunk_number(p.n, first, p.s * a.seg, C) * a.H + h) * PC::BYTES;
    const int64_t inv_step = (int64_t)a.H * PC::BYTES;
    const E *q = static_cast<const E *>(a.q) + p.begin * a.st.q_t + g * a.st.q_g;
    const E *k = static_cast<const E *>(a.k) + p.begin * a.st.k_t + g * a.st.k_g;
    const E *v = static_cast<const E *>(a.v) + p.begin * a.st.v_t + h * a.st.v_h + c0;
    const float *la = a.la + (a.la_t ? p.begin * a.la_t : 0) + h;

    if (wave >= 4) {
        // ---- fetches and scores
        const int tid = threadIdx.x - 256, w = wave - 4;
        constexpr int TU = PC::BYTES / 16, TPER = Lds::T_HERE ? (TU + PT - 1) / PT : 1;
        Tile<E, C, KP, PT> tq, tk;
        Tile<E, C, VT, PT> tv;
        u32x4 tt[TPER];
        const auto load = [&](int c) {
            const int t0 = c * C, rows = p.rows - t0;
            tq.template load<VEC>(q + t0 * a.st.q_t, a.st.q_t, min(C, rows), a.dk, tid);
            tk.template load<VEC>(k + t0 * a.st.k_t, a.st.k_t, min(C, rows), a.dk, tid);
            tv.template load<VEC>(v + t0 * a.st.v_t, a.st.v_t, min(C, rows), cols, tid);
            if constexpr (Lds::T_HERE) {
                const rsrc_t r = make_rsrc(inv + c * inv_step, rows > 0 ? PC::BYTES : 0);
#pragma unroll
                for (int u = 0; u < TPER; ++u)
                    tt[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (u * PT + tid) * 16, 0, 0));
            }
        };
        const auto log_decay = [&](int c) {
            const int t = c * C + lane;
            return lane < C && t < p.rows ? la[t * a.la_t] : 0.f;
        };
        const auto store = [&](int c) {
            const int b = c & 1;
            tq.template store<LK>(lds.q[b], tid);
            tk.template store<LK>(lds.k[b], tid);
            tv.template store<LV>(lds.v[b], tid);
            if constexpr (Lds::T_HERE)
#pragma unroll
                for (int u = 0; u < TPER; ++u)
                    if (TU % PT == 0 || u * PT + tid < TU) reinterpret_cast<u32x4 *>(lds.t[b])[u * PT + tid] = tt[u];
        };
        // P: the 16 x 16 tiles on and below the diagonal, dealt to the four
        // waves.  Formed as K Q^T, so that a lane holds 4 scores of one query.
        const auto scores = [&](int c) {
            const int b = c & 1;
            const L *qs = lds.q[b], *ks = lds.k[b];
            const Decays<C> &d = lds.dec[c % 3];
            constexpr int TILES = TT * (TT + 1) / 2;
            const auto product = [&](int u) {
                const int it = TT == 2 ? (u > 0) : (u > 0) + (u > 2) + (u > 5), jt = u - it * (it + 1) / 2;
                f32x4 x = {};
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    x = mma(frag8(ks + (16 * jt + l16) * LK + 32 * s + 2 * g4),
                            frag8(qs + (16 * it + l16) * LK + 32 * s + 2 * g4), x);
                return x;
            };
            const auto masked = [&](int u, f32x4 x) {
                const int it = TT == 2 ? (u > 0) : (u > 0) + (u > 2) + (u > 5), jt = u - it * (it + 1) / 2;
                const int i = 16 * it + l16, j = 16 * jt + g4;
                const float bh = d.hi[i], bl = d.lo[i];
                const f32x4 jh = *reinterpret_cast<const f32x4 *>(d.hi + j);
                const f32x4 jl = *reinterpret_cast<const f32x4 *>(d.lo + j);
                float out[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    out[e] = x[e] * __expf((bh - jh[e]) + (bl - jl[e]));
                    if (j + e > i) out[e] = 0.f;
                }
                // half jt % 2 of the lane's 8 values
                store4(reinterpret_cast<L *>(lds.p[b] + (PC::at(it, jt / 2) * PC::UNITS * 64 + lane) * 16 +
                                             (jt % 2) * (PC::UNITS == 2 ? 1024 : 8)), out);
            };
            if constexpr (TILES == 10) {
                const f32x4 x0 = product(w), x1 = product(w + 4);
                f32x4 x2 = {};
                if (w < 2) x2 = product(w + 8);
                masked(w, x0);
                masked(w + 4, x1);
                if (w < 2) masked(w + 8, x2);
            } else {
                f32x4 x = {};
                if (w < TILES) x = product(w);
                if (w < TILES) masked(w, x);
            }
        };
        // the scores above the diagonal that a piece on it holds stay 0
        if (w < TT && w % 2 == 0) {
            const float zero[4] = {};
#pragma unroll
            for (int b = 0; b < 2; ++b)
                store4(reinterpret_cast<L *>(lds.p[b] + (PC::at(w, w / 2) * PC::UNITS * 64 + lane) * 16 +
                                             (PC::UNITS == 2 ? 1024 : 8)), zero);
        }
        // Without conditions: a chunk past the last one loads nothing and
        // leaves zeros in a buffer that is not read.
        load(0);
        if (w == 3) make_decays(lds.dec[0], log_decay(0), lane);
        store(0);
        load(1);
        block_sync();
        scores(0);
        if (w == 3) make_decays(lds.dec[1], log_decay(1), lane);
        block_sync();
        for (int c = 0; c < chunks; ++c) {
            const float la2 = log_decay(c + 2);
            store(c + 1);
            load(c + 2);
            block_sync();
            scores(c + 1);
            if (w == 3) make_decays(lds.dec[(c + 2) % 3], la2, lane);
            block_sync();
        }
        return;
    }

    // ---- states and outputs
    __builtin_amdgcn_s_setprio(1);
    const int64_t state = (int64_t)a.dk * a.dv;
    float *pool = p.slot < 0 ? nullptr : a.states + ((int64_t)p.slot * a.H + h) * state;
    const int w0 = 16 * NT * wave;   // this wave's columns of the tile

    // S: value i of accumulator m, n is row 32 (m / 2) + 2 g4 + 4 (m % 2) + i,
    // column w0 + l16 or, of two column tiles, w0 + 8 (l16 / 4) + 4 n + l16 % 4:
    // then a lane's values of Y are 8 columns that follow one another.
    // The registers hold S / scale: the chunks' decays gather in `scale`,
    // until it leaves 2^-16 .. 2^16.
    f32x4 S[MT][NT];
    float scale = 1.f;
    const auto column = [&](int n) { return w0 + (NT == 2 ? 8 * (l16 >> 2) + 4 * n + (l16 & 3) : l16); };
    const auto state_at = [&](int m, int n, int i) {
        const int col = column(n);
        const uint32_t base = col < cols ? (uint32_t)(2 * g4 * a.dv + c0 + col) * 4u : kOOB;
        return base + (uint32_t)(32 * (m / 2) + 4 * (m % 2) + i) * (uint32_t)a.dv * 4u;
    };
    {
        const float *from = p.carry ? pool : nullptr;
        const rsrc_t r = make_rsrc(from, from ? state * 4 : 0);   // zeros where nothing enters
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[m][n][i] = ssd::gload1(r, state_at(m, n, i));
    }
    block_sync();
    block_sync();
    for (int c = 0; c < chunks; ++c) {
        const int b = c & 1, rows = min(C, p.rows - c * C);
        const Decays<C> &d = lds.dec[c % 3];
        const L *qs = lds.q[b], *ks = lds.k[b], *vs = lds.v[b];
        const char *ts = Lds::T_HERE ? lds.t[b] : inv + c * inv_step;
        Frag<L> own_t[Lds::T_HERE ? 1 : PC::N][PARTS];
        if constexpr (!Lds::T_HERE)
#pragma unroll
            for (int f = 0; f < PC::N; ++f)
#pragma unroll
                for (int u = 0; u < PARTS; ++u) own_t[f][u] = piece<L, C>(ts, f, u, lane);
        // X = K S (rows: the chunk's, columns: of v), Y^T = S^T Q^T
        f32x4 X[NT][TT], Y[NT][TT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < TT; ++t) X[n][t] = Y[n][t] = f32x4{};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            Frag<L> fs[NT][PARTS];
#pragma unroll
            for (int n = 0; n < NT; ++n) split(fs[n], S[2 * s][n], S[2 * s + 1][n]);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const Frag<L> fk = frag8(ks + (16 * t + l16) * LK + 32 * s + 2 * g4);
                const Frag<L> fq = frag8(qs + (16 * t + l16) * LK + 32 * s + 2 * g4);
#pragma unroll
                for (int u = PARTS - 1; u >= 0; --u)
#pragma unroll
                    for (int n = 0; n < NT; ++n) X[n][t] = mma(fk, fs[n][u], X[n][t]);
#pragma unroll
                for (int n = 0; n < NT; ++n) Y[n][t] = mma(fs[n][0], fq, Y[n][t]);
            }
        }
        // U = (T diag(beta)) (V - diag(e^b) K S)
        f32x4 U[NT][TT];
        {
            Frag<L> fg[TS][NT][PARTS];
#pragma unroll
            for (int s = 0; s < TS; ++s) {
                const f32x4 ea = *reinterpret_cast<const f32x4 *>(d.in + 32 * s + g4) * scale;
                const f32x4 eb = *reinterpret_cast<const f32x4 *>(d.in + 32 * s + 16 + g4) * scale;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const Frag<L> fv = frag_col<LV, NT == 2>(vs + 32 * s * LV, w0 + 4 * n, lane);
                    f32x4 ga, gb;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ga[i] = (float)fv.x[i] - ea[i] * X[n][2 * s][i];
                        gb[i] = (float)fv.x[4 + i] - eb[i] * X[n][2 * s + 1][i];
                    }
                    split(fg[s][n], ga, gb);
                }
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
#pragma unroll
                for (int n = 0; n < NT; ++n) U[n][t] = f32x4{};
#pragma unroll
                for (int s = 0; s <= t / 2; ++s) {
                    Frag<L> ft[PARTS];
#pragma unroll
                    for (int u = 0; u < PARTS; ++u) {
                        if constexpr (Lds::T_HERE)
                            ft[u] = piece<L, C>(ts, PC::at(t, s), u, lane);
                        else
                            ft[u] = own_t[PC::at(t, s)][u];
                    }
#pragma unroll
                    for (int o = PARTS - 1; o >= 0; --o)   // the small products first
#pragma unroll
                        for (int u = 0; u <= o; ++u)
#pragma unroll
                            for (int n = 0; n < NT; ++n) U[n][t] = mma(ft[u], fg[s][n][o - u], U[n][t]);
                }
            }
        }
        // An infinity or a NaN in k, v, beta, a decay or the state shows in U.
        float zero = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) zero = __builtin_fmaf(U[n][t][i], 0.f, zero);
        const bool odd = __ballot(!(zero == 0.f)) != 0;
        // the other waves' barrier between their tiles and their scores
        block_sync();
        E *yc = y + c * C * a.st.y_t;
        if (__builtin_expect(odd, 0)) {
            // The products above would carry it to rows before its own, where T
            // and P are 0: the recurrence itself, row by row.
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) S[m][n] *= scale;
            scale = 1.f;
#pragma unroll 1
            for (int j = 0; j < rows; ++j) {
                const float dec = __expf(clamp_decay(la[(c * C + j) * a.la_t]));
                const float beta = a.beta[(int64_t)(p.begin + c * C + j) * a.beta_t + h];
                float dot[NT], out[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) dot[n] = out[n] = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const Frag<L> fk = frag8(ks + j * LK + 32 * s + 2 * g4);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float &x = reinterpret_cast<float *>(&S[2 * s + i / 4][n])[i % 4];
                            x *= dec;
                            dot[n] += (float)fk.x[i] * x;
                        }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    dot[n] += __shfl_xor(dot[n], 16);
                    dot[n] += __shfl_xor(dot[n], 32);
                    dot[n] = beta * (to_f(vs[j * LV + column(n)]) - dot[n]);
                }
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const Frag<L> fk = frag8(ks + j * LK + 32 * s + 2 * g4), fq = frag8(qs + j * LK + 32 * s + 2 * g4);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float &x = reinterpret_cast<float *>(&S[2 * s + i / 4][n])[i % 4];
                            x += (float)fk.x[i] * dot[n];
                            out[n] += (float)fq.x[i] * x;
                        }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    out[n] += __shfl_xor(out[n], 16);
                    out[n] += __shfl_xor(out[n], 32);
                    if (lane < 16 && column(n) < cols) yc[j * a.st.y_t + column(n)] = from_f<E>(out[n]);
                }
            }
            block_sync();
            continue;
        }
        const float entered = scale;
        scale = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(scale * d.all)));
        if (!(scale > 0x1p-16f && scale < 0x1p16f)) {   // and where it is NaN
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) S[m][n] *= scale;
            scale = 1.f;
        }
        const float unscale = 1.f / scale;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float e = d.in[16 * t + l16] * entered;
#pragma unroll
            for (int n = 0; n < NT; ++n) Y[n][t] *= e;
        }
#pragma unroll
        for (int s = 0; s < TS; ++s) {
            Frag<L> fu[NT][YU], fw[NT][PARTS];
            const f32x4 wa = *reinterpret_cast<const f32x4 *>(d.out + 32 * s + g4) * unscale;
            const f32x4 wb = *reinterpret_cast<const f32x4 *>(d.out + 32 * s + 16 + g4) * unscale;
#pragma unroll
            for (int n = 0; n < NT; ++n) split(fu[n], U[n][2 * s], U[n][2 * s + 1]);
#pragma unroll
            for (int t = 2 * s; t < TT; ++t) {
                Frag<L> fp;
                char *to = reinterpret_cast<char *>(&fp);
#pragma unroll
                for (int i = 0; i < PC::UNITS; ++i)
                    *reinterpret_cast<u32x4 *>(to + 16 * i) = *reinterpret_cast<const u32x4 *>(
                        lds.p[b] + ((PC::at(t, s) * PC::UNITS + i) * 64 + lane) * 16);
#pragma unroll
                for (int u = YU - 1; u >= 0; --u)
#pragma unroll
                    for (int n = 0; n < NT; ++n) Y[n][t] = mma(fu[n][u], fp, Y[n][t]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) split(fw[n], U[n][2 * s] * wa, U[n][2 * s + 1] * wb);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const Frag<L> fk = frag_col<LK, true>(ks + 32 * s * LK, 32 * (m / 2) + 4 * (m % 2), lane);
#pragma unroll
                for (int u = PARTS - 1; u >= 0; --u)
#pragma unroll
                    for (int n = 0; n < NT; ++n) S[m][n] = mma(fk, fw[n][u], S[m][n]);
            }
        }
        {
            const rsrc_t r = make_rsrc(yc, ((rows - 1) * a.st.y_t + cols) * (int64_t)sizeof(E));
            const int col = w0 + NT * g4;   // 4 NT columns from here on
            constexpr int W = 4 * NT, PIECE = 16 / (int)sizeof(E) < W ? 16 / (int)sizeof(E) : W;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int row = 16 * t + l16;
                const uint32_t off = (uint32_t)(row * (int)a.st.y_t + col) * (uint32_t)sizeof(E);
                E out[W];
#pragma unroll
                for (int e = 0; e < W; ++e) out[e] = from_f<E>(Y[e / 4][t][e % 4]);
#pragma unroll
                for (int e = 0; e < W; e += VEC ? PIECE : 1) {
                    const uint32_t o = row < rows && col + e < cols ? off + e * (uint32_t)sizeof(E) : kOOB;
                    if constexpr (VEC && PIECE * sizeof(E) == 16) {
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

    const rsrc_t r = make_rsrc(pool, pool ? state * 4 : 0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) ssd::gstore1(r, state_at(m, n, i), S[m][n][i] * scale);
}

// ---- host side

static int col_tile(int64_t dk, int64_t dv) { return dk > 128 || dv <= 64 ? 64 : 128; }

// Rows of a chunk (DeltaPerCu).
static int chunk_rows(int dtype, int64_t dk, int64_t dv)
{
    return dtype == LAYER_BF16 && dk <= 128 && col_tile(dk, dv) == 128 ? 64 : 32;
}

struct DeltaPlan {
    int64_t ids = 0;     // chunk numbers
    size_t total = 0;    // bytes of the workspace
};

static DeltaPlan plan_delta(const lin_shape &s, int dtype)
{
    DeltaPlan P;
    const int C = chunk_rows(dtype, s.dk, s.dv);
    P.ids = s.T / C + s.N;
    const int64_t image = dtype == LAYER_BF16 ? (C == 64 ? Pieces<bf16, 64>::BYTES : Pieces<bf16, 32>::BYTES)
                                              : Pieces<float, 32>::BYTES;
    P.total = (size_t)(P.ids * s.H) * (size_t)image;
    return P;
}

// The workspace for any element type.
static size_t delta_workspace(const lin_shape &s)
{
    const size_t a = plan_delta(s, LAYER_BF16).total, b = plan_delta(s, LAYER_F32).total;
    return a > b ? a : b;
}

template <typename E, int KP, int VT, bool VEC>
static int run_delta(DeltaArgs &a, int64_t ids, hipStream_t st)
{
    constexpr int C = DeltaPerCu<E, KP, VT>::C;
    if (ids > 0 && a.T > 0) {
        DeltaArgs c = a;
        c.seg = C;
        c.ids = (int)ids;
        k_delta_inverse<E, KP, C, VEC, false><<<dim3((unsigned)(ids * a.H)), dim3(4 * C), 0, st>>>(c);
    }
    const int64_t grid = (int64_t)a.ids * a.H * a.tiles;
    k_delta_chunks<E, KP, VT, C, VEC><<<dim3((unsigned)grid), dim3(512), 0, st>>>(a);
    return launch_status();
}

template <typename E, bool VEC>
static int dispatch_delta(DeltaArgs &a, int64_t ids, hipStream_t st)
{
    const bool wide = col_tile(a.dk, a.dv) == 128;
    if (a.dk > 128) return run_delta<E, 256, 64, VEC>(a, ids, st);
    if (a.dk > 64) return wide ? run_delta<E, 128, 128, VEC>(a, ids, st) : run_delta<E, 128, 64, VEC>(a, ids, st);
    return wide ? run_delta<E, 64, 128, VEC>(a, ids, st) : run_delta<E, 64, 64, VEC>(a, ids, st);
}

}  // namespace layer

using namespace layer;

extern "C" size_t delta_prefill_workspace_size(const lin_shape *shape, int64_t max_seqlen)
{
    if (check_delta(shape, false) != SSD_OK || max_seqlen < 0) return (size_t)-1;
    return delta_workspace(*shape);
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
    const size_t need = delta_workspace(s);
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
    a.ends = a.segdec = nullptr;
    a.inv = static_cast<char *>(workspace);
    a.T = (int)s.T;
    a.N = (int)s.N;
    a.G = (int)s.G;
    a.H = (int)s.H;
    a.dk = (int)s.dk;
    a.dv = (int)s.dv;
    a.nslots = (int)s.slots;
    const int vt = col_tile(s.dk, s.dv);
    a.tiles = (a.dv + vt - 1) / vt;
    a.seg = 0;
    a.ids = (int)s.N;
    a.shift = -1;
    const int64_t ids = plan_delta(s, dtype).ids;
    const auto rows16 = [&](const void *ptr, int64_t row, int64_t head, int64_t d) {
        return !misaligned(ptr, 16) && row * e % 16 == 0 && head * e % 16 == 0 && d * e % 16 == 0 && row >= d;
    };
    const bool vec = rows16(q, a.st.q_t, a.st.q_g, s.dk) && rows16(k, a.st.k_t, a.st.k_g, s.dk) &&
                     rows16(v, a.st.v_t, a.st.v_h, s.dv) && rows16(y, a.st.y_t, a.st.y_h, s.dv);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LAYER_BF16) return vec ? dispatch_delta<bf16, true>(a, ids, st) : dispatch_delta<bf16, false>(a, ids, st);
    if (dtype == LAYER_F16) return vec ? dispatch_delta<f16, true>(a, ids, st) : dispatch_delta<f16, false>(a, ids, st);
    return vec ? dispatch_delta<float, true>(a, ids, st) : dispatch_delta<float, false>(a, ids, st);
}
