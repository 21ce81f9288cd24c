"""Beam search's calls: refusals on the CPU, and on the GPU the selection
against a sort in 64 bits and the reordering against a copy."""
import ctypes
import math

import pytest
import torch

import chunked_ssd_scan_fwd_amd as ssd
from chunked_ssd_scan_fwd_amd.layer import BeamShapeArg, StateReorderShapeArg
from gpu_util import need_gpu, say

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = range(6)
P = 0x10000   # a pointer that is never followed
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF, NAN = math.inf, math.nan
# A sum of float32 exponentials is within 2^-21 of itself (2^-24 (1 + |x - m|) a term, whose weight falls as
# e^-|x - m|, and the partial sums' roundings), so its logarithm is within 2^-21: candidates of two beams are told
# apart where they differ by more than twice that.
TIE = 2.0 ** -20


def select(shape, dtype=1, lr=64, lk=16, end=0, ws=(P, 1 << 40), **other):
    p = dict.fromkeys(("logits", "scores", "ended", "out", "tokens", "parents"), P) | other
    return ssd.library().beam_select(ctypes.byref(shape), dtype, p["logits"], lr, lk, p["scores"], p["ended"], end,
                                     p["out"], p["tokens"], p["parents"], *ws, None)


def test_select_refuses():
    s = BeamShapeArg(2, 4, 16, 4)
    for bad, code in (((-1, 4, 16, 4), SHAPE), ((2, 0, 16, 4), SHAPE), ((2, 4, 0, 4), SHAPE), ((2, 4, 16, 0), SHAPE),
                      ((2, 65, 16, 4), UNSUPPORTED), ((2, 4, 16, 65), UNSUPPORTED), ((1 << 24, 4, 16, 4), SHAPE),
                      ((2, 4, 1 << 29, 4), SHAPE), ((1 << 23, 4, 16, 4), SHAPE)):
        assert select(BeamShapeArg(*bad)) == code, bad
    assert select(s, dtype=3) == UNSUPPORTED
    assert select(s, lr=-1) == SHAPE and select(s, lk=1 << 40) == SHAPE
    assert select(s, end=16) == SHAPE and select(s, end=-1) == SHAPE
    for name in ("logits", "scores", "out", "tokens", "parents"):
        assert select(s, **{name: None}) == NULL and select(s, **{name: P + 1}) == ALIGN, name
    need = ssd.layer.beam_select_workspace_size(2, 4, 16, 4)
    assert select(s, ws=(P, need - 1)) == WORKSPACE
    assert select(s, ws=(None, need)) == NULL and select(s, ws=(P + 8, need)) == ALIGN
    assert select(BeamShapeArg(0, 4, 16, 4), logits=None, ws=(None, 0)) == OK
    assert ssd.library().beam_select(None, 0, None, 0, 0, None, None, 0, None, None, None, None, 0, None) == NULL
    with pytest.raises(ValueError):
        ssd.layer.beam_select_workspace_size(2, 65, 16, 4)
    with pytest.raises(ValueError):
        ssd.beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2), 2)
    with pytest.raises(TypeError):
        ssd.beam_select(torch.zeros(1, 2, 8, dtype=torch.float64), torch.zeros(1, 2), 2)


def test_select_refuses_places_past_31_bits():
    """The last tiles of a row end within 31 bits too."""
    for beams in (1, 2, 64):
        most = ((1 << 31) - (1 << 14) - 1) // beams
        assert ssd.layer.beam_select_workspace_size(1, beams, most, 4) > 0
        for V in (most + 1, ((1 << 31) - 1) // beams):
            assert select(BeamShapeArg(1, beams, V, 4)) == SHAPE


def reorder(shape, parents=P, slots=P, states=P):
    return ssd.library().state_reorder(ctypes.byref(shape), parents, slots, states, None)


def test_reorder_refuses():
    s = StateReorderShapeArg(2, 4, 9, 1, 8, 8)
    for bad, code in (((-1, 4, 9, 1, 8, 8), SHAPE), ((2, 0, 9, 1, 8, 8), SHAPE), ((2, 4, -1, 1, 8, 8), SHAPE),
                      ((2, 4, 9, 0, 8, 8), SHAPE), ((2, 65, 9, 1, 8, 8), UNSUPPORTED), ((2, 4, 9, 1, 257, 8), UNSUPPORTED),
                      ((2, 4, 9, 1, 8, 257), UNSUPPORTED), ((1 << 24, 4, 9, 1, 8, 8), SHAPE), ((2, 4, 1 << 24, 1, 8, 8), SHAPE),
                      ((2, 4, 9, 1 << 16, 8, 8), SHAPE)):
        assert reorder(StateReorderShapeArg(*bad)) == code, bad
    assert reorder(s, parents=None) == NULL and reorder(s, states=None) == NULL
    for name in ("parents", "slots", "states"):
        assert reorder(s, **{name: P + 2}) == ALIGN
    assert reorder(StateReorderShapeArg(3, 4, 9, 1, 8, 8), slots=None) == SHAPE
    assert reorder(StateReorderShapeArg(0, 4, 0, 1, 8, 8), None, None, None) == OK
    assert ssd.library().state_reorder(None, None, None, None, None) == NULL
    with pytest.raises(ValueError):
        ssd.state_reorder(torch.zeros(4, 1, 2, 2), torch.zeros(1, 4, dtype=torch.int32))


# ---- on the GPU


def check_select(name, logits, scores, n, ended=None, end=0, move=lambda t: t.to("cuda")):
    R, K, V = logits.shape
    say(f"beam_select {name} {tuple(logits.shape)} {logits.dtype} n {n}")
    got = ssd.beam_select(move(logits), scores.to("cuda"), n, ended=None if ended is None else ended.to("cuda"),
                          end_token=end)
    torch.cuda.synchronize()
    gs, gt, gp = (t.cpu() for t in got)
    x = logits.double()
    c = scores.double()[..., None] + (x - torch.logsumexp(x, -1, keepdim=True))
    bad = torch.isnan(x).any(-1) | (x == INF).any(-1) | (x == -INF).all(-1) | ~(scores > -INF)
    c[bad] = -INF
    if ended is not None:
        for r, k in ended.nonzero().tolist():
            c[r, k] = -INF
            c[r, k, end] = scores[r, k].double() if scores[r, k] > -INF else -INF
    c = c.flatten(1)
    val, at = c.sort(dim=-1, descending=True, stable=True)
    for r in range(R):
        m = min(n, int((val[r] > -INF).sum()))
        assert bool((gt[r, m:] == -1).all()) and bool((gp[r, m:] == -1).all()) and bool((gs[r, m:] == -INF).all())
        flat = (gp[r, :m].long() * V + gt[r, :m].long())
        assert len(set(flat.tolist())) == m
        assert bool((gt[r, :m] >= 0).all()) and bool((gt[r, :m] < V).all())
        ours = c[r][flat]
        # half a float32 step of the score, and the logarithm's error
        assert bool(((gs[r, :m].double() - ours).abs() <= 2.0 ** -24 * ours.abs() + TIE / 2).all())
        for i in range(m):
            if int(flat[i]) != int(at[r, i]):
                # another beam's candidate, as near as the sums' errors; within a beam the order is exact
                assert int(flat[i]) // V != int(at[r, i]) // V, (r, i, flat[i], at[r, i])
                assert abs(float(ours[i] - val[r, i])) <= TIE, (r, i)
    return gs, gt, gp


def rows(R, K, V, dtype, seed, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R, K, V, generator=g) * scale).to(dtype), -8.0 * torch.rand(R, K, generator=g)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("R,K,V,n", [(1, 1, 1, 1), (1, 1, 3, 5), (2, 3, 7, 4), (3, 4, 100, 8), (1, 4, 2047, 8), (2, 2, 2048, 4),
                                     (2, 5, 2049, 10), (1, 4, 32001, 8), (2, 8, 5000, 16), (1, 64, 1003, 64), (5, 1, 70000, 64),
                                     (40, 4, 4096, 8), (7, 16, 9999, 33)])
def test_select_sizes(R, K, V, n, dtype):
    need_gpu()
    check_select("sizes", *rows(R, K, V, dtype, V + n), n)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_select_large_rows_in_several_tiles(dtype):
    need_gpu()
    check_select("many", *rows(72, 4, 70001, dtype, 5), 8)     # more than one tile to a wave
    check_select("many", *rows(72, 4, 65536, dtype, 6), 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("kind", ["equal", "zeros of both signs", "rising", "falling", "two values", "peak", "far", "large"])
@pytest.mark.parametrize("n", [1, 8, 64])
def test_select_ties_and_orders(kind, n, dtype):
    need_gpu()
    R, K, V = 2, 3, 5003
    x, s = rows(R, K, V, dtype, 3)
    if kind == "equal":
        x[:], s[:] = 1.5, -2.0
    elif kind == "zeros of both signs":
        x[:] = 0.0
        x[..., ::3] = -0.0
    elif kind == "rising":
        x = (torch.arange(V).double() / V * 20).expand(R, K, V).to(dtype)
    elif kind == "falling":
        x = (-torch.arange(V).double() / V * 20).expand(R, K, V).to(dtype)
    elif kind == "two values":
        x = (x > 1).to(dtype)
    elif kind == "peak":
        x[0, 1, 4000] = 200.0
    elif kind == "far":
        x -= 30000.0
    else:
        x *= 1000.0
    check_select(kind, x.contiguous(), s, n)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF, F16])
def test_select_masked_ended_and_dead_beams(dtype):
    need_gpu()
    R, K, V = 4, 5, 3001
    x, s = rows(R, K, V, dtype, 11)
    x[0, 0, :] = -INF                       # nothing left of a beam
    x[0, 1, 10:] = -INF
    x[1, 2, 77] = NAN
    x[1, 3, 78] = INF
    x[2, :, 5:] = -INF                      # few candidates
    x[2, 0, :] = NAN
    s[3, 1:] = -INF                         # a request that has just begun
    s[1, 4] = NAN
    ended = torch.zeros(R, K, dtype=torch.uint8)
    check_select("masked", x, s, 8, ended)
    check_select("masked", x, s, 64)
    ended[0, 0] = ended[1, 1] = ended[2, 0] = 1   # also one whose logits hold NaN: they are not read
    ended[3, :] = 1
    check_select("ended", x, s, 8, ended, 2999)
    check_select("ended", x, s, 40, ended.bool(), 0)
    ended[:] = 1
    s[0] = -INF
    check_select("all ended", x, s, 8, ended, 7)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_select_strides(dtype):
    """Slices of padded rows on every alignment, and beams that share one row."""
    need_gpu()
    x, s = rows(3, 4, 2500, dtype, 2)
    for lo, pad in ((0, 12), (1, 3), (3, 5), (8, 8)):
        big = torch.full((3, 4, lo + 2500 + pad), NAN, dtype=dtype, device="cuda")
        big[..., lo:lo + 2500] = x.to("cuda")
        check_select("slices", x, s, 8, move=lambda _, b=big, o=lo: b[..., o:o + 2500])
    one = x[:, :1].expand(3, 4, 2500)
    check_select("shared", one, s, 8, move=lambda _: x[:, :1].to("cuda").expand(3, 4, 2500))
    check_select("beams first", x, s, 8, move=lambda t: t.to("cuda").transpose(0, 1).contiguous().transpose(0, 1))


def reordered(states, parents, slots):
    """The definition, one request after the other."""
    R, K = parents.shape
    out, seen = states.clone(), set()
    for r in range(R):
        mine = slots[r * K:(r + 1) * K]
        if seen & {m for m in mine if m >= 0}:
            seen |= {m for m in mine if m >= 0}
            continue
        seen |= {m for m in mine if m >= 0}
        for j in range(K):
            p, to = int(parents[r, j]), mine[j]
            if p < 0 or not 0 <= to < len(states) or to in mine[j + 1:]:
                continue
            src = mine[p] if p < K else -1
            out[to] = states[src] if 0 <= src < len(states) else NAN
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 2, 4, 5, 8, 16, 17, 64])
@pytest.mark.parametrize("H,dk,dv", [(2, 16, 16), (1, 3, 5), (3, 33, 20)])
def test_reorder(K, H, dk, dv):
    need_gpu()
    say(f"state_reorder K {K} {H} {dk} {dv}")
    g = torch.Generator().manual_seed(K)
    R = 3
    S = torch.randn(R * K + 5, H, dk, dv, generator=g)
    for slots in (None, torch.randperm(R * K + 5, generator=g)[:R * K].int()):
        parents = torch.randint(0, K, (R, K), generator=g).int()
        parents[0, 0] = -1
        pool = S.to("cuda")
        ssd.state_reorder(pool, parents.to("cuda"), slots=None if slots is None else slots.to("cuda"))
        want = reordered(S, parents, list(range(R * K)) if slots is None else slots.tolist())
        assert torch.equal(pool.cpu(), want)


@pytest.mark.gpu
def test_reorder_of_unusable_indexes():
    need_gpu()
    S = torch.randn(12, 1, 4, 6, generator=torch.Generator().manual_seed(1))
    parents = torch.tensor([[1, 0, 7, 2], [3, 3, 0, 1], [1, 2, 3, 0], [1, 0, 3, 2]], dtype=torch.int32)
    slots = [0, 1, 2, 3, 4, -1, 5, 99, 6, 2, 8, 9, 10, 11, 10, 7]
    pool = S.to("cuda")
    ssd.state_reorder(pool, parents.to("cuda"), slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    want = reordered(S, parents, slots)
    got = pool.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[4]).all())   # parents that do not exist
    assert torch.equal(got[[6, 8, 9]], S[[6, 8, 9]])                             # a slot of an earlier request


@pytest.mark.gpu
def test_reorder_off_16_bytes():
    need_gpu()
    S = torch.randn(8, 2, 8, 8, generator=torch.Generator().manual_seed(1))
    pool = torch.empty(S.numel() + 1, device="cuda")[1:].view(S.shape).copy_(S)
    parents = torch.tensor([[3, 2, 1, 0], [0, 0, 0, 0]], dtype=torch.int32)
    ssd.state_reorder(pool, parents.to("cuda"))
    assert torch.equal(pool.cpu(), reordered(S, parents, list(range(8))))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_select_into_its_own_scores(dtype):
    """The scores of a step in the place of those of the step before."""
    need_gpu()
    R, K, V = 5, 4, 9001
    x, s = rows(R, K, V, dtype, 8)
    ended = torch.zeros(R, K, dtype=torch.uint8, device="cuda")
    ended[1, 2] = ended[3] = 1
    x, s = x.to("cuda"), s.to("cuda")
    want = ssd.beam_select(x, s, K, ended=ended, end_token=7)
    out = (s, *(torch.empty(R, K, dtype=torch.int32, device="cuda") for _ in range(2)))
    got = ssd.beam_select(x, s, K, ended=ended, end_token=7, out=out)
    assert got[0] is s and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("n", [1, 8, 64])
def test_select_of_masked_pieces(n, dtype):
    """Masks that leave nothing of a row's first pieces, little of them, or one token at its end."""
    need_gpu()
    x, s = rows(3, 2, 40007, dtype, 21)
    x[0, 0, :30000] = -INF
    x[0, 1, 5:] = -INF
    x[1, 0, :40006] = -INF
    x[1, 1, 2000:39990] = -INF
    x[2, 0, ::2] = -INF
    x[2, 1, torch.arange(40007) % 701 != 3] = -INF
    check_select("masked pieces", x, s, n)


@pytest.mark.gpu
def test_reorder_with_beams_for_the_shapes_sake():
    """Negative slots stand for no beam in any number of requests; one that does not exist counts as a slot of both."""
    need_gpu()
    S = torch.randn(8, 2, 4, 6, generator=torch.Generator().manual_seed(1))
    parents = torch.tensor([[1, 0, -1], [1, 0, -1], [1, 0, 2], [1, 0, 2]], dtype=torch.int32)
    for pad, served in ((-1, (0, 1, 2, 3)), (-7, (0, 1, 2, 3)), (8, (0,)), (1 << 30, (0,))):
        slots = [x for r in range(4) for x in (2 * r, 2 * r + 1, pad)]
        want = S.clone()
        for r in served:
            want[[2 * r, 2 * r + 1]] = S[[2 * r + 1, 2 * r]]
        assert torch.equal(reordered(S, parents, slots), want)
        pool = S.to("cuda")
        ssd.state_reorder(pool, parents.to("cuda"), slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert torch.equal(pool.cpu(), want)
