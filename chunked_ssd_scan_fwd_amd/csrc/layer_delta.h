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
// T is a unit lower triangular matrix that no state enters.  It is formed as a
// substitution forms it, in float32: 16 x 16 diagonal blocks row by row, and
// the rest in products of blocks that no power of A = diag(beta) M enters (the
// powers of a matrix of near keys reach 10^17 in a chunk of 64, its inverse
// stays at 1).
#pragma once

#include "layer_tiles.h"

namespace layer {

struct DeltaArgs : PrefillArgs {
    const float *beta;
    int64_t beta_t;
    float *maps;    // segments' transitions, [id][H][dk][map_cols]
    int map_cols, map_tiles;   // dk rounded up to a multiple of 4, and blocks for as many columns
};

// Chunk number of row `begin` + `at` of sequence n, for chunks of C rows.
// Sequence n's first chunk has number begin / C + n, so that there is one for
// every chunk without a count of them; some numbers have no chunk.
__device__ __forceinline__ int chunk_number(int n, int begin, int at, int C) { return begin / C + n + at / C; }

// ---- T and P of a chunk of 32 rows as operands: two pieces of 16 x 32, in the
// order in which lanes read them.
//
// Piece t holds rows 16 t ..: lane l has row l % 16 and, with g = l / 16,
// columns 4 g .. 4 g + 3 and 16 + 4 g .. (the order in which accumulators of 16
// rows each give a summed axis of 32).
template <typename L>
struct Pieces {
    static constexpr int PARTS = sizeof(L) == 2 ? 3 : 1;
    static constexpr int UNITS = sizeof(L) == 2 ? 1 : 2;   // 16-byte units of a lane's 8 values
    static constexpr int BYTES = 2 * PARTS * UNITS * 1024;
};
// The lane's 8 values of part u of piece t in an image of PARTS parts at `p`.
template <typename L, int PARTS = Pieces<L>::PARTS>
__device__ __forceinline__ Frag<L> piece(const char *p, int t, int u, int lane)
{
    typedef Pieces<L> P;
    Frag<L> r;
    char *to = reinterpret_cast<char *>(&r);
#pragma unroll
    for (int i = 0; i < P::UNITS; ++i)
        *reinterpret_cast<u32x4 *>(to + 16 * i) =
            *reinterpret_cast<const u32x4 *>(p + (((t * PARTS + u) * P::UNITS + i) * 64 + lane) * 16);
    return r;
}

}  // namespace layer
