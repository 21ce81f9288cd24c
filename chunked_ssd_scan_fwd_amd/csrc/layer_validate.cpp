// Host-only argument checks of the linear-attention layer's calls.  This
// unit makes no HIP call.
#include "layer.h"

namespace layer {

int check_dtype(int dtype)
{
    return dtype == LAYER_F32 || dtype == LAYER_BF16 || dtype == LAYER_F16 ? SSD_OK : SSD_ERR_UNSUPPORTED;
}

int check_lin(const lin_shape *s, bool step)
{
    if (!s) return SSD_ERR_NULL;
    if (s->N < 0 || s->G < 1 || s->H < 1 || s->dk < 1 || s->dv < 1 || s->slots < 0) return SSD_ERR_SHAPE;
    if (!step && s->T < 0) return SSD_ERR_SHAPE;
    if (s->H % s->G != 0) return SSD_ERR_SHAPE;
    if (s->dk > kMaxHeadDim || s->dv > kMaxHeadDim) return SSD_ERR_UNSUPPORTED;
    if (s->N >= kMaxCount || s->slots >= kMaxCount || s->H >= 65536) return SSD_ERR_SHAPE;
    if (!step && s->T >= (int64_t(1) << 30)) return SSD_ERR_SHAPE;
    // a block for each row (or sequence), head and column tile
    const int64_t tiles = (s->dv + 31) / 32;
    if (s->N > max_blocks(512) / (s->H * tiles)) return SSD_ERR_SHAPE;
    return SSD_OK;
}

int check_delta(const lin_shape *s, bool step)
{
    const int rc = check_lin(s, step);
    if (rc != SSD_OK || step) return rc;
    // a block for each chunk (of 32 rows or more) and head
    return s->T / 32 + s->N > max_blocks(256) / s->H ? SSD_ERR_SHAPE : SSD_OK;
}

int check_delta_bwd(const lin_shape *s)
{
    const int rc = check_delta(s, false);
    if (rc != SSD_OK) return rc;
    // both walks of a sequence in one launch, and four columns of a row's q to a thread
    const int64_t tiles = (s->dv + 63) / 64;
    if (s->N > max_blocks(512) / (2 * s->H * tiles)) return SSD_ERR_SHAPE;
    // a block of 512 threads for each chunk of the products and head
    if (s->T / (s->dk > 128 ? 32 : 64) + s->N > max_blocks(512) / s->H) return SSD_ERR_SHAPE;
    return s->G != s->H && s->T > max_blocks(256) * 256 / (s->G * s->dk) ? SSD_ERR_SHAPE : SSD_OK;
}

int resolve_strides(const lin_shape *s, const lin_strides *st, lin_strides *o, int64_t rows, bool written)
{
    if (!st) {
        *o = {s->G * s->dk, s->dk, s->G * s->dk, s->dk, s->H * s->dv, s->dv, s->H * s->dv, s->dv};
    } else {
        *o = *st;
    }
    for (int64_t x : {o->q_t, o->k_t, o->v_t, o->y_t})
        if (x < 0 || x >= kMaxCount) return SSD_ERR_SHAPE;
    for (int64_t x : {o->q_g, o->k_g, o->v_h, o->y_h})
        if (x < 0 || x >= (int64_t(1) << 40)) return SSD_ERR_SHAPE;
    if (!written) return SSD_OK;
    // two values of y never share their place: heads inside rows, or rows inside heads
    const int64_t d = s->dv, H = s->H;
    const bool in_rows = (H == 1 || o->y_h >= d) && (rows <= 1 || o->y_t >= (H == 1 ? 0 : (H - 1) * o->y_h) + d);
    const bool in_heads = (rows <= 1 || o->y_t >= d) && (H == 1 || o->y_h >= (rows <= 1 ? 0 : (rows - 1) * o->y_t) + d);
    return in_rows || in_heads ? SSD_OK : SSD_ERR_SHAPE;
}

int check_gn(const gn_shape *s, int act)
{
    if (!s) return SSD_ERR_NULL;
    if (s->N < 0 || s->L < 0 || s->C < 1 || s->groups < 1 || s->C % s->groups != 0) return SSD_ERR_SHAPE;
    if (act != GN_ACT_NONE && act != GN_ACT_SILU) return SSD_ERR_UNSUPPORTED;
    const int64_t lim = int64_t(1) << 40;
    if (s->C >= kMaxCount || s->L >= (int64_t(1) << 30) || s->N > lim) return SSD_ERR_SHAPE;
    if (s->N > lim / (s->L + 1) || s->N * (s->L + 1) > lim / s->C) return SSD_ERR_SHAPE;
    return SSD_OK;
}

int check_cache(const state_cache_shape *s)
{
    if (!s) return SSD_ERR_NULL;
    if (s->n < 0 || s->slots < 0 || s->entries < 0 || s->H < 1 || s->dk < 1 || s->dv < 1) return SSD_ERR_SHAPE;
    if (s->dk > kMaxHeadDim || s->dv > kMaxHeadDim) return SSD_ERR_UNSUPPORTED;
    if (s->n >= kMaxCount || s->slots >= kMaxCount || s->entries >= kMaxCount || s->H >= 65536) return SSD_ERR_SHAPE;
    return SSD_OK;
}

// A place among a request's candidates, and the end of the 8 tiles of 2048 that
// may follow it, fit 31 bits.
constexpr int64_t kMaxCandidates = (int64_t(1) << 31) - (1 << 14) - 1;

int check_beam(const beam_shape *s)
{
    if (!s) return SSD_ERR_NULL;
    if (s->requests < 0 || s->beams < 1 || s->vocabulary < 1 || s->n < 1) return SSD_ERR_SHAPE;
    if (s->beams > BEAM_MAX || s->n > BEAM_MAX) return SSD_ERR_UNSUPPORTED;
    if (s->requests >= kMaxCount || s->vocabulary > kMaxCandidates / s->beams) return SSD_ERR_SHAPE;
    // a wave for 2048 logits or more
    const int64_t pieces = (s->vocabulary + 2047) / 2048;
    return s->requests * s->beams > max_blocks(256) / pieces ? SSD_ERR_SHAPE : SSD_OK;
}

int check_reorder(const state_reorder_shape *s)
{
    if (!s) return SSD_ERR_NULL;
    if (s->requests < 0 || s->beams < 1 || s->slots < 0 || s->H < 1 || s->dk < 1 || s->dv < 1) return SSD_ERR_SHAPE;
    if (s->beams > BEAM_MAX || s->dk > kMaxHeadDim || s->dv > kMaxHeadDim) return SSD_ERR_UNSUPPORTED;
    if (s->requests >= kMaxCount || s->slots >= kMaxCount || s->H >= 65536) return SSD_ERR_SHAPE;
    return SSD_OK;
}

}  // namespace layer
