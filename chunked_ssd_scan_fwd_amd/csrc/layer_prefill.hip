// The scalar-decay scan of a packed batch over a pool of states, in chunks.
//
// With b_t the sum of a chunk's log decays up to row t, b_L its last value and
// S the state entering the chunk,
//   Y  = (Q K^T o D) V + diag(e^b) Q S,   D_ij = e^{b_i - b_j} for j <= i, else 0
//   S <- e^{b_L} S + K^T diag(e^{b_L - b}) V.
//
// A block walks the chunks of one segment of a sequence for one head and VT
// columns of v, with S in its registers: q, k, v are read once and y is
// written once, and no chunk's state goes to memory.  Each of the waves that
// hold S owns 16 or 32 columns of S, of Y and of V and all dk rows of S, so S
// never crosses waves; only the masked scores P = Q K^T o D do, through LDS.
//
// Sequences longer than the plan's segment are cut: one pass leaves the state
// each segment makes from zero, a second pass joins them into the states that
// enter the segments, a third walks the segments from those.
//
// bfloat16 inputs run on bf16 MFMA, float32 and float16 ones on fp32 MFMA (a
// float16 P or S would overflow or vanish where float32 does not).  For bf16
// two operands are rounded to it: P, and the copy of S that meets Q, each by
// half a step of its own values.  That is what the matrix unit's rate costs:
// y is 0.0023 from 64 bits where its own rounding makes 0.0017 (up to 0.0036
// in a row of one term, whose P is not averaged with others).  S itself, its
// update and all sums stay float32, so nothing of it adds up over a sequence.
// q, k and v handed in as float32 are rounded nowhere.
#include "layer_tiles.h"

namespace layer {

constexpr int CT = 256;   // threads of a block of the carry pass

// One segment for one head and VT columns.  KP: dk rounded up; C: rows of a
// chunk.  OUT: y and the last state, from the state that enters the segment.
// Otherwise: the state that the segment makes from zero, and its decay.
//
// The block's first four waves hold S and make Y, 16 NT columns each; the
// other four fetch the next chunks, write them to LDS and form the next
// chunk's scores, so that neither waits for the other's loads.  Vector
// instructions ran beside matrix ones for a sixth of the matrix time only, so
// what counts for the first four is instructions: Q, K and P, which every one
// of them reads, are read once for NT column tiles.
//
// Every operand is read from LDS 16 bytes at a time, or transposed; pairs of
// 8-byte reads ran at a quarter of that rate.  So that S can meet Q as it
// comes out of its accumulators, a lane's 8 rows of S (two accumulators) are
// 8 rows of S that follow one another, and P is stored in the order in which
// the transposed reads of V give its rows.  Rows of 2-byte values are padded
// by 32 bytes: 16-byte reads of 16 rows then moved 252 bytes a clock, and 128
// with 16 bytes.
template <typename E, int KP, int VT, int C, bool OUT>
struct ChunkLds {
    typedef typename std::conditional<std::is_same<E, bf16>::value, bf16, float>::type L;
    static constexpr int PAD = sizeof(L) == 2 ? 16 : 4;
    static constexpr int LK = KP + PAD, LV = VT + PAD, LP = C + PAD;
    L q[2][OUT ? C * LK : 8], k[2][C * LK], v[2][C * LV], p[2][OUT ? C * LP : 8];
    Decays<C> dec[3];
    alignas(16) float odd[2][256];   // by fetching thread: 0, or NaN where its part of v has an infinity or a NaN
};

// Blocks that share a CU.  With 64 columns and 32-row chunks two of them fit
// its LDS and registers, and fill each other's waits: 20 mixed prompts of 24
// heads of 128 x 64 took 44 us so, 49 with one and 64-row chunks, 20 of 500
// rows 33 and 46, one of 32768 155 and 216; 8 of 2048 took 73 and 69.  Heads
// of 128 columns are faster as one block of them with 64-row chunks than as
// two blocks of 64 with 32-row ones (171 against 210 us for 65536 rows of 8
// heads, 428 against 523 for 16 prompts of 8192 and 16 heads).
template <typename E, int KP, int VT>
struct PerCu {
    static constexpr int n = VT == 64 && KP <= 128 && std::is_same<E, bf16>::value ? 2 : 1;
    static constexpr int C = n == 2 || sizeof(E) == 4 || KP > 128 || !std::is_same<E, bf16>::value ? 32 : 64;
};

template <typename E, int KP, int VT, int C, bool OUT, bool VEC>
__global__ __launch_bounds__(512)
__attribute__((amdgpu_waves_per_eu(2 * PerCu<E, KP, VT>::n, 2 * PerCu<E, KP, VT>::n))) void k_lin_chunks(PrefillArgs a)
{
    typedef ChunkLds<E, KP, VT, C, OUT> Lds;
    typedef typename Lds::L L;
    constexpr int LK = Lds::LK, LV = Lds::LV, LP = Lds::LP;
    constexpr int NT = VT / 64, MT = KP / 16, TT = C / 16, KS = KP / 32, TS = C / 32;
    constexpr int PT = 256;   // threads that fetch
    __shared__ __align__(16) Lds lds;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int tile = blockIdx.x % a.tiles, h = blockIdx.x / a.tiles % a.H;
    int id = blockIdx.x / (a.tiles * a.H);
    Place p;
    if (!find(a, id, p)) return;
    if (!OUT && p.s + 1 >= p.segs) return;   // nothing follows the last segment
    const int g = h / (a.H / a.G), c0 = tile * VT, cols = min(VT, a.dv - c0);
    E *y = static_cast<E *>(a.y) + p.begin * a.st.y_t + h * a.st.y_h + c0;
    if (p.bad) {
        if (OUT)
            for (int64_t e = threadIdx.x; e < (int64_t)p.rows * VT; e += 512)
                if (e % VT < cols) y[e / VT * a.st.y_t + e % VT] = from_f<E>(__builtin_nanf(""));
        return;
    }
    const int chunks = (p.rows + C - 1) / C;

    if (wave >= 4) {
        // ---- fetches and scores
        const int tid = threadIdx.x - 256, w = wave - 4;
        const E *q = static_cast<const E *>(a.q) + p.begin * a.st.q_t + g * a.st.q_g;
        const E *k = static_cast<const E *>(a.k) + p.begin * a.st.k_t + g * a.st.k_g;
        const E *v = static_cast<const E *>(a.v) + p.begin * a.st.v_t + h * a.st.v_h + c0;
        const float *la = a.la + (a.la_t ? p.begin * a.la_t : 0) + h;
        Tile<E, C, KP, PT> tq, tk;
        Tile<E, C, VT, PT> tv;
        // The tiles of chunk c, after those of the chunk before it went to LDS.
        // Whether v's had infinities or NaN is looked at with the loads of q
        // and k on their way, and told in the place that was stored last.
        const auto load = [&](int c) {
            const int t0 = c * C, rows = p.rows - t0;
            if (OUT) tq.template load<VEC>(q + t0 * a.st.q_t, a.st.q_t, min(C, rows), a.dk, tid);
            tk.template load<VEC>(k + t0 * a.st.k_t, a.st.k_t, min(C, rows), a.dk, tid);
            if (c > 0) lds.odd[(c - 1) & 1][tid] = tv.zero_times();
            tv.template load<VEC>(v + t0 * a.st.v_t, a.st.v_t, min(C, rows), cols, tid);
        };
        const auto log_decay = [&](int c) {
            const int t = c * C + lane;
            return lane < C && t < p.rows ? la[t * a.la_t] : 0.f;
        };
        const auto store = [&](int c) {
            const int b = c & 1;
            if (OUT) tq.template store<LK>(lds.q[b], tid);
            tk.template store<LK>(lds.k[b], tid);
            tv.template store<LV>(lds.v[b], tid);
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
                store4(lds.p[b] + i * LP + 32 * (jt / 2) + 2 * g4 + 4 * (jt % 2), out);
            };
            // a wave's tiles together, so that one's reads run beside the
            // others' products
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
        // the scores above the diagonal that a 32-wide step over them reads stay 0
        if (OUT && w < TT && w % 2 == 0)
            for (int e = lane; e < 512; e += 64)
                lds.p[e / 256][(16 * w + e / 16 % 16) * LP + 16 * w + 8 * (e / 4 % 4) + 4 + e % 4] = (L)0.f;
        // Without conditions: a chunk past the last one loads nothing and
        // leaves zeros in a buffer that is not read.  (With them the compiler
        // copied the tiles' registers and waited for the loads to do so.)
        load(0);
        if (w == 3) make_decays(lds.dec[0], log_decay(0), lane);
        store(0);
        load(1);
        block_sync();
        if (OUT) scores(0);
        if (w == 3) make_decays(lds.dec[1], log_decay(1), lane);
        if (OUT) block_sync();
        for (int c = 0; c < chunks; ++c) {
            const float la2 = log_decay(c + 2);
            store(c + 1);
            load(c + 2);
            if (OUT) {
                block_sync();
                scores(c + 1);
            }
            if (w == 3) make_decays(lds.dec[(c + 2) % 3], la2, lane);
            block_sync();
        }
        return;
    }

    // ---- states and outputs
    //
    // Ahead of the others where both have something to issue: 204 us for 65536
    // rows of 16 heads of 64, 206 without; other shapes within the noise.
    __builtin_amdgcn_s_setprio(1);
    const int64_t state = (int64_t)a.dk * a.dv;
    float *pool = p.slot < 0 ? nullptr : a.states + ((int64_t)p.slot * a.H + h) * state;
    float *ends = p.segs > 1 ? a.ends + ((int64_t)id * a.H + h) * state : nullptr;
    const int w0 = 16 * NT * wave;   // this wave's columns of the tile

    // S: value i of accumulator m, n is row 32 (m / 2) + 2 g4 + 4 (m % 2) + i,
    // column w0 + l16 or, of two column tiles, w0 + 8 (l16 / 4) + 4 n + l16 % 4:
    // then a lane's values of Y are 8 columns that follow one another.
    // Offsets step by constants from one lane's base; a row past dk lies past
    // the resource's end, and a column past the tile's is sent there.
    //
    // The registers hold S / scale: the chunks' decays gather in `scale`, which
    // costs a factor of Y's instead of a multiplication of all of S, until it
    // leaves 2^-16 .. 2^16.
    f32x4 S[MT][NT];
    float scale = 1.f;
    const auto state_at = [&](int m, int n, int i) {
        const int col = w0 + (NT == 2 ? 8 * (l16 >> 2) + 4 * n + (l16 & 3) : l16);
        const uint32_t base = col < cols ? (uint32_t)(2 * g4 * a.dv + c0 + col) * 4u : kOOB;
        return base + (uint32_t)(32 * (m / 2) + 4 * (m % 2) + i) * (uint32_t)a.dv * 4u;
    };
    {
        const float *from = !OUT ? nullptr : p.segs > 1 ? ends : p.carry ? pool : nullptr;
        const rsrc_t r = make_rsrc(from, from ? state * 4 : 0);   // zeros where nothing enters
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[m][n][i] = OUT ? ssd::gload1(r, state_at(m, n, i)) : 0.f;
    }
    double total = 0.0;
    block_sync();
    if (OUT) block_sync();
    for (int c = 0; c < chunks; ++c) {
        const int b = c & 1;
        const Decays<C> &d = lds.dec[c % 3];
        const L *qs = lds.q[b], *ks = lds.k[b], *vs = lds.v[b], *ps = lds.p[b];
        const f32x4 o = *reinterpret_cast<const f32x4 *>(lds.odd[b] + 4 * lane);
        const bool odd = __ballot(!((o[0] + o[1]) + (o[2] + o[3]) == 0.f)) != 0;
        f32x4 Y[NT][TT];
        if (OUT) {
            // Y^T = diag(e^b) S^T Q^T, rows: columns of v, columns: queries
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int t = 0; t < TT; ++t) Y[n][t] = f32x4{};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                Frag<L> fs[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) frag_acc(fs[n], S[2 * s][n], S[2 * s + 1][n]);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const Frag<L> fq = frag8(qs + (16 * t + l16) * LK + 32 * s + 2 * g4);
#pragma unroll
                    for (int n = 0; n < NT; ++n) Y[n][t] = mma(fs[n], fq, Y[n][t]);
                }
            }
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
        // The terms of v's infinities and NaN, which are 0 in the tile from then
        // on: at the scores above the diagonal, where P is 0, they would reach
        // earlier rows, and the parts of a product with an infinity do not add
        // up to it.  No other wave reads this one's columns.  (Y is scaled by
        // e^b after them, which leaves an infinity one or makes it NaN.)
        const auto odd_terms = [&]() {
            const auto finite = [](float x) { return __builtin_fabsf(x) < __builtin_inff(); };
#pragma unroll 1
            for (int j = 0; j < min(C, p.rows - c * C); ++j) {
                L *vj = lds.v[b] + j * LV + w0;
                const L *pj = ps + 32 * (j / 32) + 8 * (j % 16 / 4) + 4 * (j / 16 % 2) + j % 4;
                if (OUT) {
                    float score[TT], x[4 * NT];
#pragma unroll
                    for (int t = 0; t < TT; ++t) score[t] = to_f(pj[(16 * t + l16) * LP]);
#pragma unroll
                    for (int e = 0; e < 4 * NT; ++e) x[e] = to_f(vj[NT * g4 + e]);
#pragma unroll
                    for (int e = 0; e < 4 * NT; ++e)
#pragma unroll
                        for (int t = 0; t < TT; ++t)
                            Y[e / 4][t][e % 4] += finite(x[e]) || j > 16 * t + l16 ? 0.f : score[t] * x[e];
                }
                __builtin_amdgcn_wave_barrier();   // the lanes have read the row's values that others take out
                const float out = d.out[j];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    L *at = vj + (NT == 2 ? 8 * (l16 >> 2) + 4 * n + (l16 & 3) : l16);
                    const float x = to_f(*at);
                    if (finite(x)) continue;
                    *at = (L)0.f;
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        const Frag<L> fk = frag8(ks + j * LK + 32 * s + 2 * g4);
#pragma unroll
                        for (int i = 0; i < 8; ++i) S[2 * s + i / 4][n][i % 4] += to_f(fk.x[i]) * (x * out);
                    }
                }
            }
            __builtin_amdgcn_wave_barrier();
        };
        if (__builtin_expect(odd, 0)) odd_terms();
        if (OUT) {
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float e = d.in[16 * t + l16] * entered;
#pragma unroll
                for (int n = 0; n < NT; ++n) Y[n][t] *= e;
            }
        }
        const float unscale = 1.f / scale;
        const auto rows32 = [&](auto step) {   // 32 rows of the chunk
            constexpr int s = decltype(step)::value, PARTS = sizeof(L) == 4 ? 1 : 3;
            Frag<L> fv[NT], fw[NT][3];
            const f32x4 wa = *reinterpret_cast<const f32x4 *>(d.out + 32 * s + g4) * unscale;
            const f32x4 wb = *reinterpret_cast<const f32x4 *>(d.out + 32 * s + 16 + g4) * unscale;
#pragma unroll
            for (int n = 0; n < NT; ++n) fv[n] = frag_col<LV, NT == 2>(vs + 32 * s * LV, w0 + 4 * n, lane);
            if (OUT) {
#pragma unroll
                for (int t = 2 * s; t < TT; ++t) {
                    const Frag<L> fp = frag8(ps + (16 * t + l16) * LP + 32 * s + 2 * g4);
#pragma unroll
                    for (int n = 0; n < NT; ++n) Y[n][t] = mma(fv[n], fp, Y[n][t]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) weigh<PARTS>(fw[n], fv[n], wa, wb);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const Frag<L> fk = frag_col<LK, true>(ks + 32 * s * LK, 32 * (m / 2) + 4 * (m % 2), lane);
#pragma unroll
                for (int u = PARTS - 1; u >= 0; --u)
#pragma unroll
                    for (int n = 0; n < NT; ++n) S[m][n] = mma(fk, fw[n][u], S[m][n]);
            }
        };
        // the other waves' barrier between their tiles and their scores: needed
        // nowhere here, it stands about where they get to theirs
        if (TS == 1 && OUT) block_sync();
        rows32(ssd::IntC<0>{});
        if (TS == 2 && OUT) block_sync();
        if constexpr (TS == 2) rows32(ssd::IntC<1>{});
        if (OUT) {
            const int t0 = c * C, rows = min(C, p.rows - t0);
            const rsrc_t r = make_rsrc(y + t0 * a.st.y_t, ((rows - 1) * a.st.y_t + cols) * (int64_t)sizeof(E));
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
        total += d.sum;
        block_sync();
    }

    float *to = OUT ? (p.s + 1 == p.segs ? pool : nullptr) : ends;
    const rsrc_t r = make_rsrc(to, to ? state * 4 : 0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) ssd::gstore1(r, state_at(m, n, i), S[m][n][i] * scale);
    if (!OUT && tile == 0 && threadIdx.x == 0) a.segdec[(int64_t)id * a.H + h] = expf((float)total);
}

// The state entering each segment of a sequence that was cut, in place of the
// states that the segments make from zero: V values of a state in a thread.
// The loads of U segments are in flight together.
template <int V>
__global__ __launch_bounds__(CT) void k_lin_carry(PrefillArgs a)
{
    typedef Vec<float, V> X;
    constexpr int U = 16;
    const int h = blockIdx.x % a.H;
    Place p;
    int begin, end;
    about(a, blockIdx.x / a.H, p, begin, end);
    const int64_t state = (int64_t)a.dk * a.dv;
    const int64_t e = ((int64_t)blockIdx.y * CT + threadIdx.x) * V;
    if (p.segs <= 1 || p.bad || e >= state) return;
    X cur = {};
    if (p.carry) cur = *reinterpret_cast<const X *>(a.states + ((int64_t)p.slot * a.H + h) * state + e);
    const int64_t id0 = begin / a.seg + p.n;
    float *x = a.ends + (id0 * a.H + h) * state + e;
    const float *dec = a.segdec + id0 * a.H + h;
    const int64_t step = a.H * state;
    for (int s0 = 0; s0 < p.segs; s0 += U) {
        X made[U];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = min(s0 + u, p.segs - 2);   // the last segment made none
            made[u] = *reinterpret_cast<const X *>(x + s * step);
            f[u] = dec[(int64_t)s * a.H];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u < p.segs) {
                *reinterpret_cast<X *>(x + (s0 + u) * step) = cur;
#pragma unroll
                for (int i = 0; i < V; ++i) cur.v[i] = f[u] * cur.v[i] + made[u].v[i];
            }
    }
}

// ---- host side

struct PrefillPlan {
    int seg = 0, ids = 0;
    size_t ends = 0, segdec = 0, total = 0;
};

static int col_tile(int64_t dk, int64_t dv) { return dk > 128 || dv <= 64 ? 64 : 128; }

// Sequences are cut where that is faster by an estimate: into segments of a
// length that makes about one block for each place on a CU out of the batch's
// rows, at least 128 rows.  Whole, the longest one's chain of chunks counts.
// Cut, a segment's two passes count for twice its rows, with 7 us for the two
// launches more and the time to write, carry and read the segments' states.
// A row takes 37 ns in bf16, 30 and 1 more for 128 values of a state on fp32
// MFMA; that is measured at heads of 128 and 128 x 64 with rows on 16 bytes.
// Rows that are not take about twice as long, which the estimate leaves out.
// Measured whole and cut, in us: one prompt of 384 rows 20 and 24, of 768 34
// and 24, of 65536 2374 and 167 (8 heads of 128); mixed prompts, 30 of up to
// 1004 rows 49 and 71 (the same heads), 8 of up to 4526 177 and 132, 8 of 8192
// 320 and 338 (16 heads).
static PrefillPlan plan_prefill(const lin_shape &s, int dtype, int64_t max_seqlen, int cus)
{
    PrefillPlan P;
    const int64_t longest = max_seqlen > 0 && max_seqlen < s.T ? max_seqlen : s.T;
    const int64_t vt = col_tile(s.dk, s.dv), tiles = (s.dv + vt - 1) / vt;
    const int64_t per_cu = vt == 64 && s.dk <= 128 && dtype == LAYER_BF16 ? 2 : 1;   // PerCu
    const int64_t work = s.T * s.H * tiles;
    const int64_t places = per_cu * cus;
    int64_t seg = ((work + places - 1) / places + 63) / 64 * 64;
    if (seg < 128) seg = 128;
    P.ids = (int)s.N;
    const double state = (double)s.H * (double)(s.dk * s.dv);
    const double row = dtype == LAYER_BF16 ? 37.0 : 30.0 + (double)(s.dk * (s.dv < vt ? s.dv : vt)) / 128.0;
    const double cut = 2.0 * row * (double)seg + 7000.0 + (double)(s.T / seg + s.N) * state * 16.0 / 4500.0;
    if (longest <= seg || row * (double)longest <= cut) return P;
    // and no more of them than a launch has blocks for
    const int64_t most = max_blocks(512) / (s.H * tiles) - s.N;
    if (most < 1) return P;
    if (s.T / seg > most) seg = (s.T / most + 64) / 64 * 64;
    if (longest <= seg || seg >= (int64_t(1) << 30)) return P;
    P.seg = (int)seg;
    P.ids = (int)(s.T / seg + s.N);
    size_t o = 0;
    P.ends = o;
    o += (size_t)P.ids * s.H * s.dk * s.dv * sizeof(float);
    o = (o + 255) / 256 * 256;
    P.segdec = o;
    o += (size_t)P.ids * s.H * sizeof(float);
    P.total = (o + 255) / 256 * 256;
    return P;
}

// Segments start in the order of falling lengths, so that the long ones have
// company that ends early and none is left to the end.  Mixed prompts in us,
// so and as they came: 40 of up to 1248 rows and 24 heads of 128 x 64 81 and
// 105, 60 of up to 1262 and 8 heads of 128 74 and 87, 16 of up to 6180 and such
// heads, cut, 132 and 151.  Finding its place in the order costs a block about
// a microsecond, so it is not done where each block has a CU for itself, nor
// for prompts that are short (64 of up to 259 rows and 24 heads: 45 and 43) or
// equal by the bound of their lengths, nor for more of them than a wave has
// lanes (an order of 100 of up to 512 rows and 8 heads: 73 and 70).
static int order_shift(const lin_shape &s, const PrefillPlan &P, int64_t max_seqlen, int64_t blocks, int cus)
{
    const int64_t longest = max_seqlen > 0 && max_seqlen < s.T ? max_seqlen : s.T;
    if (s.N < 2 || s.N > SORTED || blocks <= cus || longest < 512 ||
        longest * s.N < s.T + s.T / 2)
        return -1;
    const int64_t most = P.seg > 0 ? P.seg : longest;
    int shift = 0;
    while (most >> shift >= 1 << KEY) ++shift;
    return shift;
}

// The workspace for any element type.
static size_t prefill_workspace(const lin_shape &s, int64_t max_seqlen, int cus)
{
    const size_t a = plan_prefill(s, LAYER_BF16, max_seqlen, cus).total;
    const size_t b = plan_prefill(s, LAYER_F32, max_seqlen, cus).total;
    return a > b ? a : b;
}

template <typename E, int KP, int VT, bool VEC>
static int run_prefill(PrefillArgs &a, hipStream_t st)
{
    // chunks of 64 rows; of 32 for float tiles, which are twice as wide, for
    // rows of 256, and where two blocks share a CU
    constexpr int C = PerCu<E, KP, VT>::C;
    const int64_t grid = (int64_t)a.ids * a.H * a.tiles;
    if (a.seg > 0) {
        k_lin_chunks<E, KP, VT, C, false, VEC><<<dim3((unsigned)grid), dim3(512), 0, st>>>(a);
        const int v = a.dk * a.dv % 4 == 0 && !misaligned(a.states, 16) ? 4 : 1;
        const int chunks = (a.dk * a.dv + CT * v - 1) / (CT * v);
        const dim3 g((unsigned)(a.N * a.H), (unsigned)chunks);
        if (v == 4)
            k_lin_carry<4><<<g, dim3(CT), 0, st>>>(a);
        else
            k_lin_carry<1><<<g, dim3(CT), 0, st>>>(a);
    }
    k_lin_chunks<E, KP, VT, C, true, VEC><<<dim3((unsigned)grid), dim3(512), 0, st>>>(a);
    return launch_status();
}

template <typename E, bool VEC>
static int dispatch_prefill(PrefillArgs &a, hipStream_t st)
{
    const bool wide = col_tile(a.dk, a.dv) == 128;
    if (a.dk > 128) return run_prefill<E, 256, 64, VEC>(a, st);
    if (a.dk > 64) return wide ? run_prefill<E, 128, 128, VEC>(a, st) : run_prefill<E, 128, 64, VEC>(a, st);
    return wide ? run_prefill<E, 64, 128, VEC>(a, st) : run_prefill<E, 64, 64, VEC>(a, st);
}

}  // namespace layer

using namespace layer;

extern "C" size_t lin_prefill_workspace_size(const lin_shape *shape, int64_t max_seqlen)
{
    if (check_lin(shape, false) != SSD_OK || max_seqlen < 0) return (size_t)-1;
    return prefill_workspace(*shape, max_seqlen, ssd::device_cus());
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
    const int cus = ssd::device_cus();
    const PrefillPlan P = plan_prefill(s, dtype, max_seqlen, cus);
    const size_t need = prefill_workspace(s, max_seqlen, cus);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (need > 0 && !workspace) return SSD_ERR_NULL;
    if (need > 0 && misaligned(workspace, 16)) return SSD_ERR_ALIGN;
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
    a.ends = reinterpret_cast<float *>(static_cast<char *>(workspace) + P.ends);
    a.segdec = reinterpret_cast<float *>(static_cast<char *>(workspace) + P.segdec);
    a.T = (int)s.T;
    a.N = (int)s.N;
    a.G = (int)s.G;
    a.H = (int)s.H;
    a.dk = (int)s.dk;
    a.dv = (int)s.dv;
    a.nslots = (int)s.slots;
    const int vt = col_tile(s.dk, s.dv);
    a.tiles = (a.dv + vt - 1) / vt;
    a.seg = P.seg;
    a.ids = P.ids;
    a.shift = order_shift(s, P, max_seqlen, (int64_t)a.ids * a.H * a.tiles, cus);
    // 16 bytes at a time where every row of every head begins on 16 bytes and
    // holds a whole number of them
    const auto rows16 = [&](const void *ptr, int64_t row, int64_t head, int64_t d) {
        return !misaligned(ptr, 16) && row * e % 16 == 0 && head * e % 16 == 0 && d * e % 16 == 0 && row >= d;
    };
    const bool vec = rows16(q, a.st.q_t, a.st.q_g, s.dk) && rows16(k, a.st.k_t, a.st.k_g, s.dk) &&
                     rows16(v, a.st.v_t, a.st.v_h, s.dv) && rows16(y, a.st.y_t, a.st.y_h, s.dv);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LAYER_BF16) return vec ? dispatch_prefill<bf16, true>(a, st) : dispatch_prefill<bf16, false>(a, st);
    if (dtype == LAYER_F16) return vec ? dispatch_prefill<f16, true>(a, st) : dispatch_prefill<f16, false>(a, st);
    return vec ? dispatch_prefill<float, true>(a, st) : dispatch_prefill<float, false>(a, st);
}
