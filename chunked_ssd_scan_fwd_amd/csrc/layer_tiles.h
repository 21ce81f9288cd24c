// What the chunked kernels over a packed batch share (layer_prefill.hip,
// layer_delta*.hip): operands of the matrix products in registers and LDS,
// tiles of q, k and v, the decays of a chunk, and where a block works.
#pragma once

#include <type_traits>

#include "layer_device.h"
#include "ssd_device.h"

namespace layer {

using ssd::block_sync;
using ssd::kOOB;
using ssd::rsrc_t;
using ssd::make_rsrc;
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int SORTED = 64, KEY = 8;   // most sequences that are put in order, by as many bits of their lengths

struct PrefillArgs {
    const void *q, *k, *v;
    const float *la;
    const int32_t *cu, *slots, *carry;
    float *states, *ends, *segdec;   // ends [id][H][dk][dv], segdec [id][H]
    void *y;
    int64_t la_t;
    lin_strides st;
    int T, N, G, H, dk, dv, nslots, tiles;
    int seg;       // rows of a segment; 0: sequences are not cut
    int ids;       // blocks' segment numbers, T / seg + N
    int shift;     // lengths >> shift order the segments; -1: as they come
};

// x, as a value that the compiler does not know: what is computed from it is
// computed where it stands, not ahead of a loop and kept in registers that the
// loop does not have.
__device__ __forceinline__ int anew(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// ---- fragments of the matrix products
//
// A fragment is the 8 values a lane holds of a 16 x 32 operand: its row (or
// column) is lane % 16, and the 8 values lie along the summed axis.  Which 8
// is free as long as both operands agree.

template <typename L>
struct Frag;
template <>
struct Frag<bf16> {
    bf16x8 x;
};
template <>
struct Frag<float> {
    float x[8];
};

__device__ __forceinline__ f32x4 mma(const Frag<bf16> &a, const Frag<bf16> &b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.x, b.x, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float> &a, const Frag<float> &b, f32x4 c)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x[j], b.x[j], c, 0, 0, 0);
    return c;
}

// 8 values in a row.
__device__ __forceinline__ Frag<bf16> frag8(const bf16 *p) { return {*reinterpret_cast<const bf16x8 *>(p)}; }
__device__ __forceinline__ Frag<float> frag8(const float *p)
{
    Frag<float> r;
    *reinterpret_cast<f32x4 *>(r.x) = *reinterpret_cast<const f32x4 *>(p);
    *reinterpret_cast<f32x4 *>(r.x + 4) = *reinterpret_cast<const f32x4 *>(p + 4);
    return r;
}
// One column of a tile in LDS whose rows are LD apart, at rows 4g .. 4g+3 and
// 16+4g .. 16+4g+3 (g = lane / 16).  Lane i = lane % 16 takes column `col` + i,
// or with SPLIT column `col` + 8 (i / 4) + i % 4.
template <int LD, bool SPLIT>
__device__ __forceinline__ Frag<bf16> frag_col(const bf16 *p, int col, int lane)
{
    // ds_read_b64_tr_b16: the 16 lanes of a group name the 8-byte pieces of a
    // 4 x 16 tile in order, and lane i of them receives its column i
    const int i = lane & 15, g = lane >> 4;
    typedef __attribute__((address_space(3))) s16x4 *lds_t;
    const bf16 *a = p + (4 * g + (i >> 2)) * LD + col + (i & 3) * (SPLIT ? 8 : 4);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(a));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(a + 16 * LD));
    return {__builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7))};
}
template <int LD, bool SPLIT>
__device__ __forceinline__ Frag<float> frag_col(const float *p, int col, int lane)
{
    Frag<float> r;
    const int i = lane & 15;
    const float *a = p + (lane >> 4) * 4 * LD + col + (SPLIT ? 8 * (i >> 2) + (i & 3) : i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.x[j] = a[j * LD];
        r.x[4 + j] = a[(16 + j) * LD];
    }
    return r;
}
// Two accumulators as an operand.
__device__ __forceinline__ void frag_acc(Frag<bf16> &r, f32x4 a, f32x4 b)
{
    r.x = __builtin_shufflevector(__builtin_convertvector(a, bf16x4), __builtin_convertvector(b, bf16x4), 0, 1, 2, 3, 4,
                                  5, 6, 7);
}
__device__ __forceinline__ void frag_acc(Frag<float> &r, f32x4 a, f32x4 b)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.x[j] = a[j];
        r.x[4 + j] = b[j];
    }
}

// V's rows times e^{b_L - b} (wa, wb: the fragment's first and last four
// rows), in PARTS summands.  float32 takes one.  Three bf16 numbers hold what
// a float32 product does: states came out within 2e-7 of 64 bits, as float32
// sums do.  Two leave 2e-6, and a slow decay carries that to the end of the
// sequence, so the first pass over one that is cut takes three as well.
// Two bf16 numbers by their bits, in a register: as an inline constant of the
// dot product this compiler passed (-1, 0) the wrong way round.
__device__ __forceinline__ bf16x2 pair_of(unsigned bits)
{
    asm("" : "+s"(bits));
    return __builtin_bit_cast(bf16x2, bits);
}
template <int PARTS>
__device__ __forceinline__ void weigh(Frag<bf16> (&fw)[3], const Frag<bf16> &fv, f32x4 wa, f32x4 wb)
{
    // Pairs: two values are rounded by one instruction, and what is left of
    // each is taken by one too, a dot product of the rounded pair with (-1, 0)
    // or (0, -1).
    const bf16x2 first = pair_of(0x0000bf80u), second = pair_of(0xbf800000u);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        f32x2 x = {(float)fv.x[e], (float)fv.x[e + 1]};
        x[0] *= e < 4 ? wa[e & 3] : wb[e & 3];
        x[1] *= e < 4 ? wa[(e & 3) + 1] : wb[(e & 3) + 1];
#pragma unroll
        for (int u = 0; u < PARTS; ++u) {
            const bf16x2 r = __builtin_convertvector(x, bf16x2);
            fw[u].x[e] = r[0];
            fw[u].x[e + 1] = r[1];
            if (u + 1 < PARTS) {
                x[0] = __builtin_amdgcn_fdot2_f32_bf16(r, first, x[0], false);
                x[1] = __builtin_amdgcn_fdot2_f32_bf16(r, second, x[1], false);
            }
        }
    }
}
template <int PARTS>
__device__ __forceinline__ void weigh(Frag<float> (&fw)[3], const Frag<float> &fv, f32x4 wa, f32x4 wb)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) fw[0].x[e] = fv.x[e] * (e < 4 ? wa[e & 3] : wb[e & 3]);
}

// Two accumulators as an operand in PARTS summands, the same way.
template <int PARTS>
__device__ __forceinline__ void split(Frag<bf16> (&f)[PARTS], f32x4 a, f32x4 b)
{
    const bf16x2 first = pair_of(0x0000bf80u), second = pair_of(0xbf800000u);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        f32x2 x = {e < 4 ? a[e & 3] : b[e & 3], e < 4 ? a[(e & 3) + 1] : b[(e & 3) + 1]};
#pragma unroll
        for (int u = 0; u < PARTS; ++u) {
            const bf16x2 r = __builtin_convertvector(x, bf16x2);
            f[u].x[e] = r[0];
            f[u].x[e + 1] = r[1];
            if (u + 1 < PARTS) {
                x[0] = __builtin_amdgcn_fdot2_f32_bf16(r, first, x[0], false);
                x[1] = __builtin_amdgcn_fdot2_f32_bf16(r, second, x[1], false);
            }
        }
    }
}
template <int PARTS>
__device__ __forceinline__ void split(Frag<float> (&f)[PARTS], f32x4 a, f32x4 b)
{
    frag_acc(f[0], a, b);
}

// Four values in PARTS summands of type L.
template <int PARTS>
__device__ __forceinline__ void split4(bf16x4 (&f)[PARTS], f32x4 x)
{
    const bf16x2 first = pair_of(0x0000bf80u), second = pair_of(0xbf800000u);
#pragma unroll
    for (int e = 0; e < 4; e += 2)
#pragma unroll
        for (int u = 0; u < PARTS; ++u) {
            const bf16x2 r = __builtin_convertvector((f32x2{x[e], x[e + 1]}), bf16x2);
            f[u][e] = r[0];
            f[u][e + 1] = r[1];
            if (u + 1 < PARTS) {
                x[e] = __builtin_amdgcn_fdot2_f32_bf16(r, first, x[e], false);
                x[e + 1] = __builtin_amdgcn_fdot2_f32_bf16(r, second, x[e + 1], false);
            }
        }
}
template <int PARTS>
__device__ __forceinline__ void split4(f32x4 (&f)[PARTS], f32x4 x)
{
    f[0] = x;
}

__device__ __forceinline__ void store4(bf16 *p, const float (&x)[4])
{
    *reinterpret_cast<bf16x4 *>(p) = __builtin_convertvector((f32x4{x[0], x[1], x[2], x[3]}), bf16x4);
}
__device__ __forceinline__ void store4(float *p, const float (&x)[4])
{
    *reinterpret_cast<f32x4 *>(p) = f32x4{x[0], x[1], x[2], x[3]};
}

// ---- tiles of q, k and v: global memory to registers to LDS

// sum + 0 x of the elements x in a register.
template <typename E>
__device__ __forceinline__ float add_zero_times(unsigned bits, float sum)
{
    if constexpr (std::is_same<E, bf16>::value)
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, bits), pair_of(0), sum, false);
    else if constexpr (std::is_same<E, f16>::value)
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, bits), f16x2{}, sum, false);
    else
        return __builtin_fmaf(__uint_as_float(bits), 0.f, sum);
}

// A ROWS x COLS tile of elements E, PER pieces of 16 bytes to each of PT threads.
template <typename E, int ROWS, int COLS, int PT>
struct Tile {
    static constexpr int VE = 16 / (int)sizeof(E), PIECES = ROWS * COLS / VE, PER = (PIECES + PT - 1) / PT;
    // Rows that one resource covers, so that its offsets stay below 2^31 and
    // kOOB past its end: 64 of 2-byte elements, 32 of 4-byte ones.
    static constexpr int SPAN = 128 / (int)sizeof(E);
    static_assert((int64_t)(SPAN - 1) * (kMaxCount - 1) * sizeof(E) + COLS * sizeof(E) <= kOOB, "offsets below 2^31");
    // rows between a thread's pieces
    static constexpr int STEP = PT * VE / COLS;
    u32x4 buf[PER];

    // Whether piece u of a thread exists.
    static __device__ __forceinline__ bool has(int u, int tid) { return PIECES % PT == 0 || u * PT + tid < PIECES; }

    // Rows 0 .. rows-1 and columns 0 .. cols-1 of the matrix at `base`, whose
    // rows are `ld` elements apart (less than 2^24); 0 elsewhere.
    // VEC (ld >= cols, and all on 16 bytes): rows past the last lie past the
    // resource's end, so the offsets are the same for every tile.
    template <bool VEC>
    __device__ __forceinline__ void load(const E *base, int64_t ld, int rows, int cols, int tid)
    {
        if constexpr (ROWS > SPAN) return load_spans<VEC>(base, ld, rows, cols, tid);
        const int64_t bytes = rows > 0 ? ((rows - 1) * ld + cols) * (int64_t)sizeof(E) : 0;
        if constexpr (VEC) {
            const rsrc_t r = make_rsrc(base, bytes);
            // pieces of a thread lie PT VE / COLS rows apart
            static_assert(PT * VE % COLS == 0, "whole rows between a thread's pieces");
            const int row = tid * VE / COLS, col = tid * VE % COLS;
            const uint32_t step = (uint32_t)(PT * VE / COLS * (int)ld) * (uint32_t)sizeof(E);
            uint32_t off = col < cols ? (uint32_t)(row * (int)ld + col) * (uint32_t)sizeof(E) : kOOB;
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                buf[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, has(u, tid) ? off : kOOB, 0, 0));
                off += step;
            }
        } else {
            const rsrc_t r = make_rsrc(base, bytes);
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int e = (u * PT + tid) * VE, row = e / COLS, col = e % COLS;
                const uint32_t off = (uint32_t)(row * (int)ld + col) * (uint32_t)sizeof(E);
                E x[VE];
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const uint32_t o =
                        has(u, tid) && row < rows && col + i < cols ? off + i * (uint32_t)sizeof(E) : kOOB;
                    if constexpr (sizeof(E) == 2)
                        x[i] = __builtin_bit_cast(E, (short)__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0));
                    else
                        x[i] = __builtin_bit_cast(E, __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0));
                }
                __builtin_memcpy(&buf[u], x, 16);
            }
        }
    }

    // The same for more rows than one resource covers.
    template <bool VEC>
    __device__ __forceinline__ void load_spans(const E *base, int64_t ld, int rows, int cols, int tid)
    {
        static_assert(sizeof(E) == 4 && 64 * VE <= SPAN * COLS && (STEP % SPAN == 0 || SPAN % STEP == 0),
                      "a wave's pieces in one span");
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int row = u * STEP + tid * VE / COLS, col = tid * VE % COLS;
            const int span = STEP <= SPAN ? u * STEP / SPAN : __builtin_amdgcn_readfirstlane(row / SPAN);
            const int at = row - span * SPAN, left = min(rows - span * SPAN, SPAN);
            const rsrc_t r = make_rsrc(base + span * SPAN * ld, left > 0 ? ((left - 1) * ld + cols) * (int64_t)sizeof(E) : 0);
            const uint32_t off = (uint32_t)(at * (int)ld + col) * (uint32_t)sizeof(E);
            const bool on = has(u, tid) && at < left;
            if constexpr (VEC) {
                buf[u] = __builtin_bit_cast(u32x4,
                                            __builtin_amdgcn_raw_buffer_load_b128(r, on && col < cols ? off : kOOB, 0, 0));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    buf[u][i] = __builtin_amdgcn_raw_buffer_load_b32(r, on && col + i < cols ? off + i * 4u : kOOB, 0, 0);
            }
        }
    }

    // The same tile for rows on any alignment, kept as the words that hold it
    // until `place` writes it: an element of 2 bytes may begin in the middle of
    // one, so a piece is five words.  The first and the last of a tile may hold
    // two bytes that are not its own, and no element of any.  (Loads of 2 bytes
    // into halves of registers, eight to a piece, came out of this compiler
    // with halves lost where it ran out of registers.)
    unsigned fifth[PER];
    template <bool VEC>
    __device__ __forceinline__ void fetch(const E *base, int64_t ld, int rows, int cols, int tid)
    {
        if constexpr (VEC || sizeof(E) != 2) {
            load<VEC>(base, ld, rows, cols, tid);
        } else {
            static_assert(ROWS <= SPAN, "one resource");
            const uintptr_t at = reinterpret_cast<uintptr_t>(base);
            const uint32_t skip = (uint32_t)(at & 2);
            const int64_t bytes = rows > 0 ? (((rows - 1) * ld + cols) * 2 + skip + 3) / 4 * 4 : 0;
            const rsrc_t r = make_rsrc(reinterpret_cast<const void *>(at - skip), bytes);
            const int row0 = tid * VE / COLS, col = tid * VE % COLS;
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int row = row0 + u * (PT * VE / COLS);
                const uint32_t first = ((uint32_t)(row * (int)ld + col) * 2u + skip) & ~3u;
                const uint32_t off = has(u, tid) && row < rows && col < cols ? first : kOOB;
#pragma unroll
                for (int i = 0; i < 4; ++i) buf[u][i] = __builtin_amdgcn_raw_buffer_load_b32(r, off + 4 * i, 0, 0);
                fifth[u] = __builtin_amdgcn_raw_buffer_load_b32(r, off + 16, 0, 0);
            }
        }
    }
    // What `fetch` with the same base, ld, cols and tid got, to LDS.
    template <bool VEC, int LD, typename L>
    __device__ __forceinline__ void place(L *lds, const E *base, int64_t ld, int cols, int tid)
    {
        if constexpr (!VEC && sizeof(E) == 2) {
            const uint32_t skip = (uint32_t)(reinterpret_cast<uintptr_t>(base) >> 1);
            const int row0 = tid * VE / COLS, col = tid * VE % COLS;
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const uint32_t odd = (skip + (uint32_t)((row0 + u * (PT * VE / COLS)) * (int)ld + col)) & 1u;
                unsigned w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned next = i < 3 ? buf[u][i + 1 < 4 ? i + 1 : 3] : fifth[u];
                    w[i] = __builtin_amdgcn_alignbit(next, buf[u][i], odd * 16);
                    w[i] = col + 2 * i + 1 < cols ? w[i] : col + 2 * i < cols ? w[i] & 0xffffu : 0u;
                }
                buf[u] = u32x4{w[0], w[1], w[2], w[3]};
            }
        }
        store<LD>(lds, tid);
    }

    // 0, or NaN where one of the thread's elements is an infinity or a NaN: the
    // sum of 0 times each, in four chains that do not wait for each other.
    __device__ __forceinline__ float zero_times() const
    {
        float sum[4] = {};
#pragma unroll
        for (int u = 0; u < PER; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = add_zero_times<E>(buf[u][i], sum[i]);
        return (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }

    template <int LD, typename L>
    __device__ __forceinline__ void store(L *lds, int tid) const
    {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            if (!has(u, tid)) continue;
            const int e = (u * PT + tid) * VE, row = e / COLS, col = e % COLS;
            L *to = lds + row * LD + col;
            if constexpr (std::is_same<E, L>::value) {
                *reinterpret_cast<u32x4 *>(to) = buf[u];
            } else {
                E x[VE];
                __builtin_memcpy(x, &buf[u], 16);
#pragma unroll
                for (int i = 0; i < VE; i += 4)
                    *reinterpret_cast<f32x4 *>(to + i) =
                        f32x4{to_f(x[i]), to_f(x[i + 1]), to_f(x[i + 2]), to_f(x[i + 3])};
            }
        }
    }
};

// ---- decays of a chunk

// Sums of log decays grow over a chunk while their differences matter, so
// they are formed in 64 bits and kept as a float and its remainder.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add64(double x)
{
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(u & 0xffffffffu), CTRL, ROWS, 0xf, true);
    const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xf, true);
    return x + __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
__device__ __forceinline__ double scan64(double x)
{
    x = dpp_add64<ssd::kRowShr + 1, 0xf>(x);
    x = dpp_add64<ssd::kRowShr + 2, 0xf>(x);
    x = dpp_add64<ssd::kRowShr + 4, 0xf>(x);
    x = dpp_add64<ssd::kRowShr + 8, 0xf>(x);
    x = dpp_add64<ssd::kRowBcast15, 0xa>(x);
    return dpp_add64<ssd::kRowBcast31, 0xc>(x);
}

template <int C>
struct Decays {
    float hi[C], lo[C];   // b_t
    float in[C];          // e^{b_t}
    float out[C];         // e^{b_L - b_t}
    float all;            // e^{b_L}
    double sum;           // b_L
};

// One wave: the decays of a chunk whose log decay at row `lane` is la (0 past
// the last row).
template <int C>
__device__ __forceinline__ void make_decays(Decays<C> &d, float la, int lane)
{
    const double b = scan64((double)clamp_decay(la));
    const unsigned long long u = __builtin_bit_cast(unsigned long long, b);
    const unsigned lo = __builtin_amdgcn_readlane((int)(u & 0xffffffffu), 63);
    const unsigned hi = __builtin_amdgcn_readlane((int)(u >> 32), 63);
    const double last = __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
    if (lane < C) {
        const float h = (float)b;
        d.hi[lane] = h;
        d.lo[lane] = (float)(b - (double)h);
        d.in[lane] = __expf((float)b);
        d.out[lane] = __expf((float)(last - b));
    }
    if (lane == 0) {
        d.all = __expf((float)last);
        d.sum = last;
    }
}

// ---- where a block works

struct Place {
    int n, begin, rows;   // sequence, first row and number of rows of the segment
    int segs, s;          // segments of the sequence, and which one this is
    int slot;             // -1: no state is kept
    bool carry;           // the sequence starts from its slot's state
    bool bad;             // the slot does not exist, or an earlier sequence has it
};

// Sequence n's rows, clamped to the batch.
__device__ __forceinline__ void rows_of(const PrefillArgs &a, int n, int &begin, int &end)
{
    begin = min(max(a.cu[n], 0), a.T);
    end = min(max(a.cu[n + 1], begin), a.T);
}

// Whether an earlier sequence has sequence n's slot.
__device__ __forceinline__ bool taken(const PrefillArgs &a, int n, int slot)
{
    bool found = false;
#pragma unroll 4
    for (int j0 = 0; j0 < n; j0 += 64) {
        const int j = j0 + (int)(threadIdx.x & 63);
        found = found || (j < n && a.slots[j < n ? j : 0] == slot);
    }
    return __ballot(found) != 0;
}

// What there is to know about sequence n; everything is loaded at once.
__device__ __forceinline__ void about(const PrefillArgs &a, int n, Place &p, int &begin, int &end)
{
    p.n = n;
    const int b = a.cu[n], e = a.cu[n + 1], slot = index_of(a.slots, n), carry = a.carry ? a.carry[n] : 1;
    begin = min(max(b, 0), a.T);
    end = min(max(e, begin), a.T);
    p.slot = slot < 0 ? -1 : slot;
    p.bad = slot >= a.nslots;
    p.carry = slot >= 0 && carry != 0;
    if (a.slots && slot >= 0 && !p.bad) p.bad = taken(a, n, slot);
    p.segs = a.seg == 0 ? 1 : max(1, (end - begin + a.seg - 1) / a.seg);
}

// Segment number r in the order of falling lengths, for every wave by itself,
// a sequence to a lane: the whole ones (of a.seg rows) by their sequence, then
// each sequence's rest, or the sequence where none is cut, by KEY bits of its
// length from `shift` on, equal ones as they come.  An empty sequence counts
// as a rest.  False: there are no more.
__device__ __forceinline__ bool by_length(const PrefillArgs &a, int r, int &n, int &s)
{
    const int lane = threadIdx.x & 63;
    const bool on = lane < a.N;
    int b, e;
    rows_of(a, min(lane, a.N - 1), b, e);
    const int len = on ? e - b : 0, whole = a.seg > 0 ? len / a.seg : 0, rest = len - whole * a.seg;
    if (a.seg > 0) {
        int sum = whole;   // of the lanes up to this one
        for (int d = 1; d < 64; d *= 2) {
            const int x = __shfl_up(sum, d);
            if (lane >= d) sum += x;
        }
        const unsigned long long m = __ballot(sum > r);
        if (m != 0) {
            n = __ffsll(m) - 1;
            s = r - __builtin_amdgcn_readlane(sum - whole, n);
            return true;
        }
        r -= __builtin_amdgcn_readlane(sum, 63);
    }
    // bit by bit, the lanes that have the r-th largest key
    const int key = min(rest >> a.shift, (1 << KEY) - 1);
    unsigned long long left = __ballot(on && (rest > 0 || len == 0));
#pragma unroll
    for (int bit = KEY - 1; bit >= 0; --bit) {
        const unsigned long long set = __ballot(key >> bit & 1) & left;
        const int c = __popcll(set);
        left = r < c ? set : left & ~set;
        r -= r < c ? 0 : c;
    }
    const int before = __builtin_amdgcn_mbcnt_hi((unsigned)(left >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)left, 0));
    const unsigned long long hit = __ballot(before == r) & left;
    n = __ffsll(hit) - 1;
    s = -1;   // the last
    return hit != 0;
}

// Where block number `id` works, and the number of its segment in its place.
// Sequence n's segments have the numbers from begin / seg + n on; there are at
// least as many up to the next sequence's first as it has segments, and the
// ones left over have none.  All 64 lanes look at sequences, so a batch of 64
// takes one load's latency.
__device__ __forceinline__ bool find(const PrefillArgs &a, int &id, Place &p)
{
    int n = id, s = 0;
    if (a.shift >= 0) {
        if (!by_length(a, id, n, s)) return false;
    } else if (a.seg > 0) {
        n = -1;
        for (int j0 = 0; j0 < a.N; j0 += 64) {
            const int j = j0 + (int)(threadIdx.x & 63);
            int b = 0, e = 0;
            if (j < a.N) rows_of(a, j, b, e);
            const int t = id - (b / a.seg + j);
            const unsigned long long m = __ballot(j < a.N && t >= 0 && (t == 0 || t * (int64_t)a.seg < e - b));
            if (m != 0 && n < 0) n = j0 + __ffsll(m) - 1;
        }
        if (n < 0) return false;
    }
    int begin, end;
    about(a, n, p, begin, end);
    p.s = 0;
    p.begin = begin;
    p.rows = end - begin;
    if (a.seg > 0) {
        const int first = begin / a.seg + n;
        p.s = a.shift < 0 ? id - first : s < 0 ? p.segs - 1 : s;
        id = first + p.s;
        p.begin += p.s * a.seg;
        p.rows = min(a.seg, end - p.begin);
    }
    return true;
}


}  // namespace layer
