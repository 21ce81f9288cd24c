// Beam search over a pool of states: the best continuations of each request's
// beams, and the states of the beams that go on.
#include "layer_device.h"
#include "ssd_device.h"

namespace layer {

constexpr int BT = 256, BW = BT / 64;   // threads and waves of a block
constexpr int PER = 32;                 // a lane's logits of a tile
constexpr int TILE = 64 * PER;          // logits of a wave's tile

// ---- the best 64 of many, one to a lane
//
// A key orders candidates: the greater is the better, and no two are equal.

// The value of lane `lane ^ J`: within 16 lanes by DPP, which costs no trip
// through LDS.
template <int J>
__device__ __forceinline__ int across(int x)
{
    constexpr int ror8 = ssd::kRowRor + 8, half_mirror = 0x141;
    if constexpr (J == 1) return __builtin_amdgcn_update_dpp(0, x, 0xb1, 0xf, 0xf, true);
    if constexpr (J == 2) return __builtin_amdgcn_update_dpp(0, x, 0x4e, 0xf, 0xf, true);
    if constexpr (J == 4) {   // 7 - i after 3 - i
        const int y = __builtin_amdgcn_update_dpp(0, x, 0x1b, 0xf, 0xf, true);
        return __builtin_amdgcn_update_dpp(0, y, half_mirror, 0xf, 0xf, true);
    }
    if constexpr (J == 8) return __builtin_amdgcn_update_dpp(0, x, ror8, 0xf, 0xf, true);
    if constexpr (J == 16) return __builtin_amdgcn_ds_swizzle(x, 0x10 << 10 | 0x1f);
    return __shfl_xor(x, 32);
}
// The value of the lane before (lane 0: its own place is never asked).
__device__ __forceinline__ int lane_before(int x)
{
    return __builtin_amdgcn_update_dpp(0, x, ssd::kWaveShr1, 0xf, 0xf, true);
}

// A logit and its place: its bits in an order, then the lower place first.
struct LogitKey {
    unsigned v, p;   // p: ~place
    __device__ __forceinline__ bool operator>(const LogitKey &o) const { return v > o.v || (v == o.v && p > o.p); }
    __device__ __forceinline__ LogitKey at(int lane) const   // the same lane for all
    {
        return {(unsigned)__builtin_amdgcn_readlane((int)v, lane), (unsigned)__builtin_amdgcn_readlane((int)p, lane)};
    }
    __device__ __forceinline__ LogitKey from(int lane) const { return {(unsigned)__shfl((int)v, lane), (unsigned)__shfl((int)p, lane)}; }
    template <int J>
    __device__ __forceinline__ LogitKey other() const { return {(unsigned)across<J>((int)v), (unsigned)across<J>((int)p)}; }
    __device__ __forceinline__ LogitKey before() const { return {(unsigned)lane_before((int)v), (unsigned)lane_before((int)p)}; }
    static __device__ __forceinline__ LogitKey least() { return {0, 0}; }
};
__device__ __forceinline__ unsigned ordered(float x)
{
    const unsigned u = __float_as_uint(x + 0.f);   // -0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(unsigned v)
{
    return __uint_as_float(v & 0x80000000u ? v & 0x7fffffffu : ~v);
}

// A score in 64 bits, and its place among the request's candidates.
struct ScoreKey {
    double c;
    unsigned place;
    __device__ __forceinline__ bool operator>(const ScoreKey &o) const
    {
        return c > o.c || (c == o.c && place < o.place);
    }
    template <typename F>
    __device__ __forceinline__ ScoreKey moved(const F &f) const
    {
        const unsigned long long u = __builtin_bit_cast(unsigned long long, c);
        const unsigned lo = (unsigned)f((int)(unsigned)u), hi = (unsigned)f((int)(unsigned)(u >> 32));
        return {__builtin_bit_cast(double, (unsigned long long)hi << 32 | lo), (unsigned)f((int)place)};
    }
    __device__ __forceinline__ ScoreKey from(int lane) const
    {
        return moved([&](int x) { return __shfl(x, lane); });
    }
    __device__ __forceinline__ ScoreKey at(int lane) const { return from(lane); }
    template <int J>
    __device__ __forceinline__ ScoreKey other() const { return moved([](int x) { return across<J>(x); }); }
    __device__ __forceinline__ ScoreKey before() const { return moved([](int x) { return lane_before(x); }); }
    static __device__ __forceinline__ ScoreKey least() { return {-__builtin_inf(), 0xffffffffu}; }
};

// Falling order over the lanes.
template <int J, typename K>
__device__ __forceinline__ void keep(K &x, int lane, bool falling)
{
    const K y = x.template other<J>();
    const bool low = (lane & J) == 0;
    if ((y > x) == (low == falling)) x = y;
}
template <int J, typename K>
__device__ __forceinline__ void merge(K &x, int lane, bool falling)   // of two orders that meet
{
    keep<J>(x, lane, falling);
    if constexpr (J > 1) merge<J / 2>(x, lane, falling);
}
template <typename K>
__device__ __forceinline__ K sorted(K x, int lane)
{
    merge<1>(x, lane, (lane & 2) == 0);
    merge<2>(x, lane, (lane & 4) == 0);
    merge<4>(x, lane, (lane & 8) == 0);
    merge<8>(x, lane, (lane & 16) == 0);
    merge<16>(x, lane, (lane & 32) == 0);
    merge<32>(x, lane, true);
    return x;
}
template <typename K>
struct Best {
    K list, last;   // lane i: the i-th best so far; the n-th of them
    int n;
    __device__ __forceinline__ explicit Best(int n_) : list(K::least()), last(K::least()), n(n_) {}
    __device__ __forceinline__ void insert(K y, int lane)   // y: the same for all lanes
    {
        const int at = __popcll(__ballot(list > y));
        const K shifted = list.before();
        if (lane > at) list = shifted;
        if (lane == at) list = y;
    }
    // Candidates x of the lanes in `on`: few one by one, many sorted and merged.
    __device__ __forceinline__ void take(K x, bool on, int lane)
    {
        unsigned long long m = __ballot(on && x > last);
        if (m == 0) return;
        if (__popcll(m) > 12) return join(sorted(on ? x : K::least(), lane), lane);
        for (; m != 0; m &= m - 1) insert(x.at(__ffsll(m) - 1), lane);
        last = list.at(n - 1);
    }
    // A list in falling order.
    __device__ __forceinline__ void join(K x, int lane)
    {
        const K y = x.from(63 - lane);
        if (y > list) list = y;
        merge<32>(list, lane, true);
        last = list.at(n - 1);
    }
};

struct BeamArgs {
    const void *logits;
    const float *scores;
    const uint8_t *ended;
    int64_t ld_r, ld_k;    // elements between requests and between a request's beams
    int R, K, V, n, tiles, pieces;   // tiles of a piece, pieces of a row
    int end;
    float *stat;           // [R K][pieces][2]: the piece's largest logit m and sum of e^{x - m}
    LogitKey *top;         // [R K][pieces][n]: its best, or keys of 0
    float *out;
    int32_t *tokens, *parents;
};

__device__ __forceinline__ bool goes_on(const BeamArgs &a, int row)
{
    return !(a.ended && a.ended[row]) && a.scores[row] > -__builtin_inff();
}

// The largest logit, the sum of exponentials and the n best of a piece of a
// row, in one pass: a wave to a piece, 2048 logits at a time in registers.
//
// Vector instructions bound it: 256 rows of 131072 bfloat16 logits take 24 us,
// where 67 MB are 13.  A SIMD has them under way in 0.7 of that: 15 for 64
// logits by the counters, one of them an exponential at half the rate.
// About 11 are every tile's (conversion, largest, the exponential and its sum,
// the votes), the rest orders and candidates.  So the candidates have to cost
// little: a logit is compared with the n-th best so far.  For the first 2048
// that is the n-th largest of the lanes' own largest ones (at least n logits
// reach it); the few that reach it go into the list one by one.  With each
// lane's best offered in turn, and sorts through LDS, it took 33.
template <typename T, bool VEC>
__global__ __launch_bounds__(BT) void k_beam_rows(BeamArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t at = (int64_t)blockIdx.x * BW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (at >= (int64_t)a.R * a.K * a.pieces) return;
    const int row = (int)(at / a.pieces), piece = (int)(at % a.pieces);
    if (!goes_on(a, row)) return;
    const T *x0 = static_cast<const T *>(a.logits) + row / a.K * a.ld_r + row % a.K * a.ld_k;
    const int first = piece * a.tiles * TILE, end = min(a.V, first + a.tiles * TILE);
    constexpr int VE = VEC ? 16 / (int)sizeof(T) : 1;
    typedef Vec<T, VE> V;
    // place of a lane's value i within a tile
    const auto place = [](int lane, int i) { return (i / VE * 64 + lane) * VE + i % VE; };
    V next[PER / VE];
    const auto load = [&](int t0) {
#pragma unroll
        for (int u = 0; u < PER / VE; ++u) {
            const int p = t0 + place(lane, u * VE);
            // whole vectors: VEC rows hold a whole number of them
            if (p < end)
                next[u] = *reinterpret_cast<const V *>(x0 + p);
            else
#pragma unroll
                for (int i = 0; i < VE; ++i) next[u].v[i] = from_f<T>(-__builtin_inff());
        }
    };
    Best<LogitKey> best(a.n);
    float m = -__builtin_inff(), s = 0.f, reach = -__builtin_inff();
    load(first);
    for (int t0 = first; t0 < end; t0 += TILE) {
        float x[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = to_f(next[i / VE].v[i % VE]);
        if (t0 + TILE < end) load(t0 + TILE);
        float big = x[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) big = fmaxf(big, x[i]);
        float top = big;
        top = fmaxf(top, __int_as_float(across<1>(__float_as_int(top))));
        top = fmaxf(top, __int_as_float(across<2>(__float_as_int(top))));
        top = fmaxf(top, __int_as_float(across<4>(__float_as_int(top))));
        top = fmaxf(top, __int_as_float(across<8>(__float_as_int(top))));
        top = fmaxf(top, __int_as_float(across<16>(__float_as_int(top))));
        top = fmaxf(top, __int_as_float(across<32>(__float_as_int(top))));
        const float M = fmaxf(m, top);
        if (M > -__builtin_inff()) {
            float sum[4] = {};
#pragma unroll
            for (int i = 0; i < PER; ++i) sum[i & 3] += __expf(x[i] - M);
            s = s * __expf(m - M) + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
            m = M;
        } else {   // nothing but -infinity, or NaN
#pragma unroll
            for (int i = 0; i < PER; ++i) s += x[i] == x[i] ? 0.f : x[i];
            continue;
        }
        if (t0 == first) {
            // (a lane's largest may be -infinity or come from a NaN's place: then fewer are passed over)
            const LogitKey own = {ordered(big), (unsigned)lane};
            reach = unordered(sorted(own, lane).at(a.n - 1).v);
        }
        if (__ballot(big >= reach) == 0) continue;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            unsigned long long c = __ballot(x[i] >= reach);
            if (c == 0) continue;
            const LogitKey key = {ordered(x[i]), ~(unsigned)(t0 + place(lane, i))};
            for (c &= __ballot(key > best.last); c != 0; c &= c - 1) {
                const LogitKey y = key.at(__ffsll(c) - 1);
                if (y > best.last) {
                    best.insert(y, lane);
                    best.last = best.list.at(a.n - 1);
                }
            }
        }
        if (best.last.v != 0) reach = fmaxf(reach, unordered(best.last.v));
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if (lane == 0) {
        a.stat[at * 2] = m;
        a.stat[at * 2 + 1] = s;
    }
    if (lane < a.n) a.top[at * a.n + lane] = best.list;
}

// The n best of a request, out of its beams' pieces: a block to a request.  A
// chain of dependent loads, a logarithm and orders over lanes: 8 us for one
// request of 4 beams, 11 for 64.
__global__ __launch_bounds__(BT) void k_beam_join(BeamArgs a)
{
    __shared__ double lse[BEAM_MAX];
    __shared__ ScoreKey lists[BW][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = blockIdx.x;
    for (int k = w; k < a.K; k += BW) {
        const int row = r * a.K + k;
        const float *st = a.stat + (int64_t)row * a.pieces * 2;
        const bool live = goes_on(a, row);
        float m = -__builtin_inff();
        double s = 0.;
        if (live) {
            for (int p = lane; p < a.pieces; p += 64) m = fmaxf(m, st[2 * p]);
#pragma unroll
            for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
            for (int p = lane; p < a.pieces; p += 64)
                s += st[2 * p + 1] == 0.f ? 0. : (double)st[2 * p + 1] * exp((double)st[2 * p] - (double)m);
#pragma unroll
            for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
        }
        // not a number where the beam offers nothing
        if (lane == 0) lse[k] = live && m > -__builtin_inff() ? (double)m + log(s) : (double)__builtin_nan("");
    }
    __syncthreads();
    Best<ScoreKey> best(a.n);
    const int per = a.pieces * a.n, all = a.K * per;
    for (int e0 = w * 64; e0 < all; e0 += BT) {
        const int e = e0 + lane, k = min(e / per, a.K - 1);
        ScoreKey key = ScoreKey::least();
        bool on = e < all && lse[k] == lse[k];
        if (on) {
            const LogitKey y = a.top[((int64_t)r * a.K + k) * per + e % per];
            const double c = (double)a.scores[r * a.K + k] + ((double)unordered(y.v) - lse[k]);
            on = y.v != 0 && c > -__builtin_inf();
            key = {c, (unsigned)k * (unsigned)a.V + ~y.p};
        }
        best.take(key, on, lane);
    }
    if (w == 0) {   // beams that have ended go on as they are
        const int row = r * a.K + min(lane, a.K - 1);
        const bool on = lane < a.K && a.ended && a.ended[row] && a.scores[row] > -__builtin_inff();
        const ScoreKey key = {(double)a.scores[row], (unsigned)lane * (unsigned)a.V + (unsigned)a.end};
        best.take(key, on, lane);
    }
    lists[w][lane] = best.list;
    __syncthreads();
    if (w != 0) return;
    for (int x = 1; x < BW; ++x) best.join(lists[x][lane], lane);
    if (lane < a.n) {
        const ScoreKey key = best.list;
        const bool none = key.place == 0xffffffffu;
        const int64_t at = (int64_t)r * a.n + lane;
        a.out[at] = none ? -__builtin_inff() : (float)key.c;
        a.tokens[at] = none ? -1 : (int)(key.place % (unsigned)a.V);
        a.parents[at] = none ? -1 : (int)(key.place / (unsigned)a.V);
    }
}

// ---- reordering

struct ReorderArgs {
    const int32_t *slots, *parents;
    float *states;
    int R, K, nslots, chunks;
    int64_t state;   // values of a state
};

// States of a request's beams, the values of one place (V of them) in a
// thread for all beams: it has read all before it writes any, so the states
// can change places with no copy of the pool.  A state that stays is neither
// read nor written.  Memory bounds it: 64 requests of 4 beams, 1 MB each, of
// which 356 MB move: 74 to 78 us (4.6 to 4.8 TB/s).
template <int KM, int V>
__global__ __launch_bounds__(BT) void k_state_reorder(ReorderArgs a)
{
    typedef Vec<float, V> X;
    __shared__ int slot[KM], from[KM];   // from: the slot to read, -1 not to write, -2 for NaN
    __shared__ int shared;
    const int tid = threadIdx.x, r = blockIdx.x / a.chunks;
    if (tid == 0) shared = 0;
    if (tid < a.K) slot[tid] = index_of(a.slots, r * a.K + tid);
    __syncthreads();
    if (tid < a.K) {
        const int to = slot[tid], p = a.parents[r * a.K + tid];
        bool write = to >= 0 && to < a.nslots && p >= 0;
        for (int j = tid + 1; j < a.K; ++j) write = write && slot[j] != to;   // the last one counts
        const int s = p >= 0 && p < a.K ? slot[p] : -1;
        from[tid] = !write || s == to ? -1 : s >= 0 && s < a.nslots ? s : -2;
    }
    if (a.slots) {
        bool found = false;
        for (int64_t j0 = 0; j0 < (int64_t)r * a.K; j0 += BT) {
            const int64_t j = j0 + tid;
            const int other = j < (int64_t)r * a.K ? a.slots[j] : -1;
            for (int i = 0; i < a.K; ++i) found = found || (other >= 0 && other == slot[i]);
        }
        if (found) shared = 1;
    }
    __syncthreads();
    if (shared) return;   // an earlier request has one of the slots
    const int64_t step = (int64_t)a.chunks * BT * V;
    for (int64_t e = ((int64_t)(blockIdx.x % a.chunks) * BT + tid) * V; e < a.state; e += step) {
        X x[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            const int s = j < a.K ? __builtin_amdgcn_readfirstlane(from[j]) : -1;
            if (s >= 0) x[j] = *reinterpret_cast<const X *>(a.states + s * a.state + e);
            if (s == -2)
#pragma unroll
                for (int i = 0; i < V; ++i) x[j].v[i] = __builtin_nanf("");
        }
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            const int s = j < a.K ? __builtin_amdgcn_readfirstlane(from[j]) : -1;
            if (s != -1) *reinterpret_cast<X *>(a.states + (int64_t)slot[j] * a.state + e) = x[j];
        }
    }
}

// ---- host side

struct BeamPlan {
    int tiles = 1, pieces = 1;
    size_t top = 0, total = 0;
};

// Tiles of a wave: as many as leave 16 waves for every CU, 8 at most.  (256 rows
// of 131072 logits: 4 each 36 us, one 47, 8 35, in float32 44, 50 and 39; 4 rows
// of 32001: one each 17 us, 8 each 33, for a wave's tiles come one after the
// other.)
static BeamPlan plan_beam(const beam_shape &s, int cus)
{
    BeamPlan P;
    const int64_t rows = s.requests * s.beams, all = (s.vocabulary + TILE - 1) / TILE;
    int64_t tiles = rows * all / ((int64_t)cus * 16);
    tiles = tiles < 1 ? 1 : tiles > 8 ? 8 : tiles;
    P.tiles = (int)tiles;
    P.pieces = (int)((all + tiles - 1) / tiles);
    P.top = ((size_t)(rows * P.pieces) * 2 * sizeof(float) + 255) / 256 * 256;
    P.total = P.top + (size_t)(rows * P.pieces * s.n) * sizeof(LogitKey);
    return P;
}

}  // namespace layer

using namespace layer;

extern "C" size_t beam_select_workspace_size(const beam_shape *shape)
{
    if (check_beam(shape) != SSD_OK) return (size_t)-1;
    return shape->requests == 0 ? 0 : plan_beam(*shape, ssd::device_cus()).total;
}

extern "C" int beam_select(const beam_shape *shape, int dtype, const void *logits, int64_t ld_request, int64_t ld_beam,
                           const float *scores, const uint8_t *ended, int32_t end_token, float *out_scores,
                           int32_t *tokens, int32_t *parents, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = check_beam(shape);
    if (rc == SSD_OK) rc = check_dtype(dtype);
    if (rc != SSD_OK) return rc;
    const beam_shape &s = *shape;
    const int64_t lim = int64_t(1) << 40;
    if (ld_beam < 0 || ld_beam >= lim || ld_request < 0 || ld_request >= lim) return SSD_ERR_SHAPE;
    if (ended && (end_token < 0 || end_token >= s.vocabulary)) return SSD_ERR_SHAPE;
    if (s.requests == 0) return SSD_OK;
    if (!logits || !scores || !out_scores || !tokens || !parents) return SSD_ERR_NULL;
    const unsigned e = dtype_size(dtype);
    if (misaligned(logits, e) || misaligned(scores, 4) || misaligned(out_scores, 4) || misaligned(tokens, 4) ||
        misaligned(parents, 4))
        return SSD_ERR_ALIGN;
    const BeamPlan P = plan_beam(s, ssd::device_cus());
    if (workspace_bytes < P.total) return SSD_ERR_WORKSPACE;
    if (!workspace) return SSD_ERR_NULL;
    if (misaligned(workspace, 16)) return SSD_ERR_ALIGN;
    BeamArgs a;
    a.logits = logits;
    a.scores = scores;
    a.ended = ended;
    a.ld_r = ld_request;
    a.ld_k = ld_beam;
    a.R = (int)s.requests;
    a.K = (int)s.beams;
    a.V = (int)s.vocabulary;
    a.n = (int)s.n;
    a.tiles = P.tiles;
    a.pieces = P.pieces;
    a.end = end_token;
    a.stat = static_cast<float *>(workspace);
    a.top = reinterpret_cast<LogitKey *>(static_cast<char *>(workspace) + P.top);
    a.out = out_scores;
    a.tokens = tokens;
    a.parents = parents;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t waves = s.requests * s.beams * P.pieces;
    const dim3 grid((unsigned)((waves + BW - 1) / BW));
    const bool vec = !misaligned(logits, 16) && ld_beam * e % 16 == 0 && ld_request * e % 16 == 0 &&
                     s.vocabulary * e % 16 == 0;
    LAYER_DISPATCH(dtype, {
        if (vec)
            k_beam_rows<T, true><<<grid, dim3(BT), 0, st>>>(a);
        else
            k_beam_rows<T, false><<<grid, dim3(BT), 0, st>>>(a);
    });
    k_beam_join<<<dim3((unsigned)s.requests), dim3(BT), 0, st>>>(a);
    return launch_status();
}

template <int KM, int V>
static void launch_reorder(ReorderArgs &a, hipStream_t st)
{
    // four places to a thread, and no more blocks than there are places
    const int64_t places = (a.state / V + BT - 1) / BT;
    int64_t chunks = (places + 3) / 4;
    const int64_t most = max_blocks(BT) / a.R;
    if (chunks > most) chunks = most;
    a.chunks = (int)chunks;
    k_state_reorder<KM, V><<<dim3((unsigned)(a.R * chunks)), dim3(BT), 0, st>>>(a);
}

extern "C" int state_reorder(const state_reorder_shape *shape, const int32_t *parents, const int32_t *slots,
                             float *states, void *stream)
{
    const int rc = check_reorder(shape);
    if (rc != SSD_OK) return rc;
    const state_reorder_shape &s = *shape;
    if (!slots && s.requests * s.beams > s.slots) return SSD_ERR_SHAPE;
    if (s.requests == 0) return SSD_OK;
    if (!parents || (s.slots > 0 && !states)) return SSD_ERR_NULL;
    if (misaligned(parents, 4) || misaligned(slots, 4) || misaligned(states, 4)) return SSD_ERR_ALIGN;
    ReorderArgs a;
    a.slots = slots;
    a.parents = parents;
    a.states = states;
    a.R = (int)s.requests;
    a.K = (int)s.beams;
    a.nslots = (int)s.slots;
    a.state = s.H * s.dk * s.dv;
    hipStream_t st = static_cast<hipStream_t>(stream);
    // A place of all beams is in registers: four values of up to 16 beams, or one
    // of up to 64.  States of 1 MB that no cache holds, at random parents: 64
    // requests of 4 beams (340 MB move) 72 us, 578 with one value and room for 64;
    // 16 of 16 beams (415 MB) 98 and 178.  Room for 4 or 8 beams where that is
    // enough: 64 of 4 72 us, with 16's 73; 32 of 8 (397 MB) 88 and 97.
    const bool vec = a.state % 4 == 0 && !misaligned(states, 16);
    if (!vec) {
        if (a.K <= 8) launch_reorder<8, 1>(a, st);
        else launch_reorder<64, 1>(a, st);
    } else if (a.K <= 4) {
        launch_reorder<4, 4>(a, st);
    } else if (a.K <= 8) {
        launch_reorder<8, 4>(a, st);
    } else if (a.K <= 16) {
        launch_reorder<16, 4>(a, st);
    } else {
        launch_reorder<64, 1>(a, st);
    }
    return launch_status();
}
