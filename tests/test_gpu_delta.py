"""The gated delta rule on the GPU, element by element against its 64-bit
form (delta_ref)."""
import numpy as np
import pytest
import torch

import chunked_ssd_scan_fwd_amd as ssd
import delta_ref as ref
from gpu_util import need_gpu, say
from layer_ref import beyond
from test_gpu_layer import dev, fused, ids, offsets

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def check_prefill(name, heads, dtype, lens, per_token=True, carry=None, slots=None, npool=None, strided=False, tail=0,
                  max_seqlen=None, change=None, seed=0, **more):
    G, H, dk, dv = heads
    say(f"delta_prefill {name} {heads} {dtype} lens {lens[:6]} tail {tail} max {max_seqlen}")
    N = len(lens)
    cu = offsets(lens)
    T = cu[-1] + tail
    q, k, v, ld, beta, S = ref.inputs(T, G, H, dk, dv, dtype, per_token, seed, npool or max(N, 1), strided, **more)
    if change is not None:
        q, k, v, ld, beta, S = change(q, k, v, ld, beta, S)
    out = torch.full((T, H, dv), 7.0, dtype=dtype, device="cuda")
    pool = dev(S)
    move = fused if strided else dev
    got = ssd.delta_prefill(move(q), move(k), move(v), dev(ld), dev(beta), ids(cu), pool,
                            slots=None if slots is None else ids(slots), carry=None if carry is None else ids(carry),
                            max_seqlen=max(lens, default=0) if max_seqlen is None else max_seqlen, out=out)
    torch.cuda.synchronize()
    y, S1, ye, Se, ym = ref.rule(q, k, v, ld, beta, cu, S, slots, carry)
    e = beyond(got[:cu[-1]], y[:cu[-1]], ref.y_bound(dtype, y, ye, ym)[:cu[-1]])
    es = beyond(pool, S1, Se + 1e-30)
    say(f"  y {e:.3f} states {es:.3f} of the bound")
    assert e <= 1 and es <= 1
    assert bool((got[cu[-1]:] == 7.0).all())
    untouched = sorted(set(range(S.shape[0])) - set(range(N) if slots is None else slots))
    assert torch.equal(pool.cpu()[untouched], S[untouched])
    return got, pool


HEADS = [(1, 1, 128, 128), (2, 4, 48, 40), (2, 8, 128, 128), (1, 6, 128, 64), (3, 3, 64, 64), (1, 2, 256, 128),
         (1, 2, 64, 256), (1, 1, 256, 256), (1, 2, 1, 1), (1, 3, 33, 97), (2, 2, 5, 200), (1, 1, 200, 3), (1, 1, 130, 129),
         (1, 2, 100, 33), (2, 2, 77, 127), (1, 3, 63, 31)]


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", HEADS)
def test_prefill_heads(heads, dtype):
    check_prefill("heads", heads, dtype, [1, 64, 130, 63, 65], per_token=heads[2] != 64, carry=[1, 0, 1, 0, 1],
                  slots=[4, 2, 0, 5, 1], npool=7, tail=3, seed=heads[2] * 7 + heads[3])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 128, 129, 200])
def test_prefill_lengths(n, dtype):
    check_prefill("length", (1, 2, 64, 128), dtype, [n], seed=n)
    check_prefill("length", (2, 2, 128, 64), dtype, [n, 3], per_token=False, seed=n)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", [(2, 4, 48, 40), (1, 3, 128, 128), (1, 2, 33, 97)])
def test_prefill_slices_of_a_projection(heads, dtype):
    check_prefill("strides", heads, dtype, [70, 0, 100], strided=True, seed=3)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens,max_seqlen", [([4500], 0), ([3000, 17, 0, 1400], 0), ([2500], 5), ([1024, 2048, 512], 0)])
def test_prefill_long(lens, max_seqlen, dtype):
    """Cut over the length: with no bound given, with the right one, and with one that is too small."""
    carry = [1] * (len(lens) - 1) + [0] if len(lens) > 1 else None
    for heads, per_token in (((1, 1, 128, 128), True), ((1, 2, 64, 48), False)):
        check_prefill("long", heads, dtype, lens, per_token=per_token, max_seqlen=max_seqlen, seed=5, carry=carry, mu=-6.0)


@pytest.mark.parametrize("heads,dtype", [((1, 1, 256, 130), BF), ((1, 2, 96, 200), F16), ((1, 1, 33, 17), F32),
                                         ((2, 2, 64, 64), BF), ((1, 1, 20, 256), BF), ((1, 1, 256, 64), F32)])
def test_prefill_cut_at_other_heads(heads, dtype):
    check_prefill("cut", heads, dtype, [1500, 1700], carry=[0, 1], slots=[2, 0], npool=3, tail=2, seed=13, mu=-6.0)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", [(2, 144, 128, 128), (1, 150, 33, 97), (4, 144, 64, 128), (1, 90, 100, 200), (2, 80, 77, 256)])
def test_prefill_many_heads(heads, dtype):
    """Blocks of 128 columns, which batches of few blocks do not get."""
    check_prefill("many heads", heads, dtype, [1, 40, 130, 65], carry=[1, 0, 1, 1], slots=[4, 2, 0, 1], npool=5, tail=3,
                  seed=heads[2], strided=heads[2] == 77)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", [(1, 8, 128, 128), (2, 8, 100, 97), (1, 8, 128, 256)])
def test_prefill_many_heads_cut(heads, dtype):
    assert ssd.layer.delta_prefill_workspace_size(5100, 3, *heads, 3) > 0
    check_prefill("many heads, cut", heads, dtype, [4500, 0, 600], carry=[1, 0, 0], seed=6, mu=-6.0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_prefill_many_heads_infinities_and_nan(bad, dtype):
    G, H, dk, dv = 1, 144, 128, 128
    q, k, v, ld, beta, S = (dev(t) for t in ref.inputs(200, G, H, dk, dv, dtype, True, 9, 2))
    clean = S.clone()
    want = ssd.delta_prefill(q, k, v, ld, beta, ids([0, 90, 200]), clean)
    v[131, 140, 70] = bad
    say(f"delta_prefill many heads v {bad} {dtype}")
    y = ssd.delta_prefill(q, k, v, ld, beta, ids([0, 90, 200]), S)
    assert torch.equal(y[:90], want[:90]) and torch.equal(y[:, :140], want[:, :140]) and torch.equal(S[0], clean[0])
    assert bool(torch.isfinite(y[:131]).all()) and not bool(torch.isfinite(y[131:, 140, 70]).any())
    y[131:, 140, 70] = want[131:, 140, 70]
    assert float((y.double() - want.double()).abs().max()) < 0.05
    assert not bool(torch.isfinite(S[1, 140, :, 70]).all())


def test_prefill_long_runs_are_cut():
    """The shapes above do run cut: they ask for a workspace."""
    for shape in ((4500, 1, 1, 1, 128, 128, 1), (4417, 4, 1, 2, 64, 48, 4), (3202, 2, 1, 1, 256, 130, 3),
                  (3202, 2, 1, 1, 33, 17, 3)):
        assert ssd.layer.delta_prefill_workspace_size(*shape) > 0, shape


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("near", [0.5, 0.9, 1.0])
def test_prefill_near_keys(near, dtype):
    """Keys that are nearly or quite the same: the inverse's powers would be huge."""
    def change(q, k, v, ld, beta, S):
        return q, k, v, ld, torch.ones_like(beta) if near == 1.0 else beta, S
    check_prefill("near", (1, 2, 128, 128), dtype, [64, 150], near=near, mu=-8.0, seed=4, change=change)
    check_prefill("near", (1, 2, 64, 64), dtype, [64, 150], near=near, mu=-8.0, seed=5, change=change)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("kind", ["beta 0", "beta 1", "beta 2", "beta mixed", "long keys", "no keys", "forget", "all",
                                  "growth", "strong", "none", "same decay and beta"])
def test_prefill_betas_and_decays(kind, dtype):
    def change(q, k, v, ld, beta, S):
        ld, beta = ld.clone(), beta.clone()
        if kind.startswith("beta"):
            beta[:] = {"0": 0.0, "1": 1.0, "2": 2.0}.get(kind[5:], 0.0)
            if kind == "beta mixed":
                beta[::3] = 1.0
        elif kind == "long keys":
            k = (k.float() * 1.3).to(k.dtype)
        elif kind == "no keys":
            k = k.clone()
            k[::2] = 0
        elif kind == "forget":   # the state is forgotten here and there, twice in a chunk too
            ld[[0, 10, 64, 70, 71, 130]] = -np.inf
        elif kind == "all":
            ld[:] = -np.inf
        elif kind == "growth":
            ld[:] = ld.abs() * 0.3
        elif kind == "strong":
            ld[:] = -60.0 + ld
        elif kind == "none":
            ld[:] = 0
        else:
            ld, beta = ld[:1].expand_as(ld), beta[:1].expand_as(beta)
        return q, k, v, ld, beta, S
    for heads in ((1, 2, 128, 128), (2, 4, 64, 48)):
        check_prefill(kind, heads, dtype, [150, 70], seed=8, change=change)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
def test_prefill_empty_and_missing(dtype):
    """Sequences of no rows, no slots, slots that cannot be used; rows of no sequence."""
    G, H, dk, dv = 1, 2, 64, 128
    check_prefill("empty", (G, H, dk, dv), dtype, [0, 5, 0, 0, 70, 0], carry=[0, 1, 1, 0, 0, 1], seed=1, tail=2)
    lens = [40, 30, 20, 10]
    q, k, v, ld, beta, S = (dev(t) for t in ref.inputs(100, G, H, dk, dv, dtype, True, 2, 4))
    pool = S.clone()
    y = ssd.delta_prefill(q, k, v, ld, beta, ids(offsets(lens)), pool, slots=ids([-1, 2, 2, 9]))
    assert bool(torch.isnan(y[70:]).all()) and bool(torch.isfinite(y[:70]).all())
    want, S1, ye, Se, ym = ref.rule(q[:70], k[:70], v[:70], ld[:70], beta[:70], offsets(lens[:2]), S, [-1, 2])
    assert beyond(y[:70], want, ref.y_bound(dtype, want, ye, ym)) <= 1
    assert beyond(pool, S1, Se + 1e-30) <= 1


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("where", ["q", "k", "v", "beta", "decay", "state"])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_prefill_infinities_and_nan(where, bad, dtype):
    """They reach the rows after them, in v only their column."""
    for heads, T in (((1, 2, 128, 128), 200), ((1, 2, 64, 64), 200), ((1, 2, 128, 64), 3000)):   # the last one cut
        G, H, dk, dv = heads
        q, k, v, ld, beta, S = ref.inputs(T, G, H, dk, dv, dtype, True, 9, 2)
        clean = [dev(t) for t in (q, k, v, ld, beta)], dev(S)
        want = ssd.delta_prefill(*clean[0], ids([0, 90, T]), clean[1])
        row, col = 131, 7
        t = {"q": q, "k": k, "v": v, "beta": beta, "decay": ld, "state": S}[where]
        if where in ("q", "k"):
            t[row, 0, col] = bad
        elif where == "v":
            t[row, 1, col] = bad
        elif where == "state":
            t[1, 1, 3, col] = bad
        else:
            t[row, 1] = bad
        say(f"delta_prefill {where} {bad} {heads} {dtype}")
        pool = dev(S)
        y = ssd.delta_prefill(*(dev(x) for x in (q, k, v, ld, beta)), ids([0, 90, T]), pool)
        y, want = y.cpu(), want.cpu()
        assert torch.equal(y[:90], want[:90])
        if where in ("v", "state"):
            rest = [c for c in range(dv) if c != col]
            assert torch.equal(y[:, 0], want[:, 0])
            # the other columns of the wave go row by row from there on: the same to rounding
            assert bool(torch.isfinite(y[:, 1][:, rest]).all())
            d = (y[:, 1][:, rest].double() - want[:, 1][:, rest].double()).abs().max()
            assert d < 0.05
        if where != "state":
            first = row if where != "q" else row
            assert bool(torch.isfinite(y[:first]).all())
            assert float((y[:first].double() - want[:first].double()).abs().max()) < 0.05
        if where == "q":
            assert bool(torch.isfinite(y[row + 1:]).all()) and bool(torch.isfinite(pool).all())
            assert not bool(torch.isfinite(y[row]).any())
        elif where == "state":
            assert not bool(torch.isfinite(pool[1, 1, 3, col]))
        else:
            assert not bool(torch.isfinite(pool[1, 1, :, col]).all())


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", HEADS + [(1, 3, 128, 68), (2, 2, 64, 32)])
def test_step_heads(heads, dtype):
    G, H, dk, dv = heads
    for N, slots in ((1, [2]), (5, [4, 6, 0, -1, 1]), (300, None)):
        if N == 300 and dk * dv > 20000:
            continue
        npool = 7 if N < 8 else 300
        q, k, v, ld, beta, S = ref.inputs(N, G, H, dk, dv, dtype, N != 5, 3 + N, npool)
        pool = dev(S)
        out = torch.full((N, H, dv), 7.0, dtype=dtype, device="cuda")
        say(f"delta_step {heads} {dtype} {N}")
        y = ssd.delta_step(*(dev(t) for t in (q, k, v, ld, beta)), pool, slots=None if slots is None else ids(slots),
                           out=out)
        rows = list(range(N)) if slots is None else slots
        want, S1, ye, Se, ym = ref.rule(q, k, v, ld, beta, list(range(N + 1)), S, rows)
        live = [n for n in range(N) if rows[n] >= 0]
        assert beyond(y[live], want[live], ref.y_bound(dtype, want, ye, ym, False)[live]) <= 1
        assert beyond(pool, S1, Se + 1e-30) <= 1
        assert bool((y[[n for n in range(N) if rows[n] < 0]] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_step_repeated_missing_and_padded_slots(dtype):
    G, H, dk, dv = 1, 3, 64, 96
    slots = [3, 1, 3, -1, 5, 3, 1, 99]
    q, k, v, ld, beta, S = ref.inputs(8, G, H, dk, dv, dtype, True, 6, 6)
    pool = dev(S)
    out = torch.full((8, H, dv), 7.0, dtype=dtype, device="cuda")
    y = ssd.delta_step(*(dev(t) for t in (q, k, v, ld, beta)), pool, slots=ids(slots), out=out)
    want, S1, ye, Se, ym = ref.rule(q[:7], k[:7], v[:7], ld[:7], beta[:7], list(range(8)), S, slots[:7])
    live = [0, 1, 2, 4, 5, 6]
    assert beyond(y[live], want[live], ref.y_bound(dtype, want, ye, ym, False)[live]) <= 1
    assert beyond(pool, S1, Se + 1e-30) <= 1
    assert bool((y[3] == 7.0).all()) and bool(torch.isnan(y[7]).all())


def test_steps_go_on_from_a_prefill():
    """A prompt at once, and its last rows one by one, give the same as the whole."""
    for dtype in (F32, BF):
        G, H, dk, dv = 2, 4, 64, 64
        q, k, v, ld, beta, S = ref.inputs(80, G, H, dk, dv, dtype, True, 12, 1)
        pool = dev(S)
        d = [dev(t) for t in (q, k, v, ld, beta)]
        ssd.delta_prefill(*(t[:70] for t in d), ids([0, 70]), pool)
        ys = [ssd.delta_step(*(t[i:i + 1] for t in d), pool) for i in range(70, 80)]
        want, S1, ye, Se, ym = ref.rule(q, k, v, ld, beta, [0, 80], S)
        assert beyond(torch.cat(ys), want[70:], ref.y_bound(dtype, want, ye, ym, False)[70:]) <= 1
        assert beyond(pool, S1, Se + 1e-30) <= 1


# ---- gradients


def check_bwd(name, heads, dtype, lens, per_token=True, entered=True, strided=False, tail=0, change=None, seed=0, **more):
    G, H, dk, dv = heads
    say(f"delta_bwd {name} {heads} {dtype} lens {lens[:6]} tail {tail}")
    N, cu = len(lens), offsets(lens)
    T = cu[-1] + tail
    q, k, v, ld, beta, S = ref.inputs(T, G, H, dk, dv, dtype, per_token, seed, N, strided, **more)
    g = torch.Generator().manual_seed(seed + 100)
    dy, dS = torch.randn(T, H, dv, generator=g).to(dtype), torch.randn(N, H, dk, dv, generator=g) * 0.5
    if change is not None:
        q, k, v, ld, beta, S, dy, dS = change(q, k, v, ld, beta, S, dy, dS)
    if not entered:
        S = dS = None
    move = fused if strided else dev
    opt = lambda t: None if t is None else dev(t)   # noqa: E731
    got = ssd.delta_bwd(move(q), move(k), move(v), dev(ld), dev(beta), ids(cu), dev(dy), states=opt(S), dstates=opt(dS))
    torch.cuda.synchronize()
    want, err = ref.gradients(q, k, v, ld, beta, cu, dy, S, dS)
    worst = {}
    for n, t in zip(("dq", "dk", "dv", "dlog_decay", "dbeta", "dstates"), got):
        if n == "dstates" and not entered:
            assert t is None
            continue
        kind = dtype if n in ("dq", "dk", "dv") else F32
        assert t.shape == want[n].shape and t.dtype == kind
        worst[n] = round(beyond(t, want[n], ref.gradient_bound(kind, want[n], err[n])), 4)
        # The bounds above add magnitudes over columns; the errors themselves do not line up.  As a whole, in the
        # 2-norm, a gradient is within its own rounding and 2^-15, which is 32 of the steps that the bounds count.
        size = float(want[n].norm())
        if size > 0:
            off = float((t.detach().cpu().double() - want[n]).norm()) / size
            assert off <= ref.HALF[kind] + 2.0 ** -15, (n, off)
    say(f"  {worst}")
    assert max(worst.values()) <= 1, worst
    return got


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", HEADS)
def test_bwd_heads(heads, dtype):
    check_bwd("heads", heads, dtype, [1, 64, 130, 63, 65], per_token=heads[2] != 64, entered=heads[3] != 64, tail=3,
              seed=heads[2] * 7 + heads[3])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 129, 200])
def test_bwd_lengths(n, dtype):
    check_bwd("length", (1, 2, 64, 128), dtype, [n], seed=n)
    check_bwd("length", (2, 2, 128, 64), dtype, [n, 3], per_token=False, seed=n)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_bwd_empty_sequences(dtype):
    check_bwd("empty", (1, 2, 64, 64), dtype, [0, 5, 0, 0, 70, 0], tail=2, seed=1)
    got = check_bwd("no rows", (1, 2, 16, 16), dtype, [0, 0], seed=1, per_token=False)
    assert bool((got[3] == 0).all())
    check_bwd("no rows", (1, 2, 16, 16), dtype, [0, 0], seed=1)
    check_bwd("no sequences", (1, 2, 16, 16), dtype, [], seed=1, per_token=False)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", [(2, 4, 48, 40), (1, 3, 128, 128), (1, 2, 33, 97)])
def test_bwd_slices_of_a_projection(heads, dtype):
    check_bwd("strides", heads, dtype, [70, 0, 100], strided=True, seed=3)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("kind", ["beta 0", "beta 1", "beta 2", "beta mixed", "long keys", "no keys", "near keys", "same keys",
                                  "forget", "all", "growth", "strong", "none", "same decay and beta", "one row of dy"])
def test_bwd_betas_and_decays(kind, dtype):
    def change(q, k, v, ld, beta, S, dy, dS):
        ld, beta = ld.clone(), beta.clone()
        if kind.startswith("beta"):
            beta[:] = {"0": 0.0, "1": 1.0, "2": 2.0}.get(kind[5:], 0.0)
            if kind == "beta mixed":
                beta[::3] = 1.0
        elif kind == "long keys":
            k = (k.float() * 1.3).to(k.dtype)
        elif kind == "no keys":
            k = k.clone()
            k[::2] = 0
        elif kind == "same keys":
            beta[:] = 1
        elif kind == "forget":
            ld[[0, 10, 64, 70, 71, 130]] = -np.inf
        elif kind == "all":
            ld[:] = -np.inf
        elif kind == "growth":
            ld[:] = ld.abs() * 0.3
        elif kind == "strong":
            ld[:] = -60.0 + ld
        elif kind == "none":
            ld[:] = 0
        elif kind == "one row of dy":
            dy = dy[:1].expand_as(dy)
        else:
            ld, beta = ld[:1].expand_as(ld), beta[:1].expand_as(beta)
        return q, k, v, ld, beta, S, dy, dS
    near = {"near keys": 0.9, "same keys": 1.0}.get(kind, 0.0)
    for heads in ((1, 2, 128, 128), (2, 4, 64, 48)):
        check_bwd(kind, heads, dtype, [150, 70], seed=8, change=change, near=near, mu=-8.0 if near else -4.0)


def test_bwd_against_differences():
    """The gradients against differences of delta_prefill itself, in float32."""
    G, H, dk, dv = 2, 4, 24, 20
    cu = [0, 70, 100]
    q, k, v, ld, beta, S = (dev(t) for t in ref.inputs(100, G, H, dk, dv, F32, True, 21, 2))
    g = torch.Generator().manual_seed(4)
    dy, dS = dev(torch.randn(100, H, dv, generator=g)), dev(torch.randn(2, H, dk, dv, generator=g))
    got = ssd.delta_bwd(q, k, v, ld, beta, ids(cu), dy, states=S, dstates=dS)

    def loss(x):
        pool = x[5].clone()
        y = ssd.delta_prefill(*x[:5], ids(cu), pool)
        return float((y.double() * dy).sum() + (pool.double() * dS).sum())

    x = [q, k, v, ld, beta, S]
    for i, grad in enumerate(got):
        d = dev(torch.randn(x[i].shape, generator=g))
        h = 2.0 ** -6 / float(d.norm() / x[i].norm()) / 8
        num = (loss(x[:i] + [x[i] + h * d] + x[i + 1:]) - loss(x[:i] + [x[i] - h * d] + x[i + 1:])) / (2 * h)
        want = float((grad.double() * d).sum())
        # the differences' own error: their third-order term, and float32's in the two losses
        assert abs(num - want) <= 2e-3 * float(grad.double().norm() * d.double().norm()), (i, num, want)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("where", ["q", "k", "v", "beta", "decay", "dy", "state", "dstate"])
def test_bwd_nan_stays_in_its_sequence(where, dtype):
    G, H, dk, dv = 2, 4, 64, 64
    cu = [0, 90, 200, 260]
    q, k, v, ld, beta, S = ref.inputs(260, G, H, dk, dv, dtype, True, 9, 3)
    g = torch.Generator().manual_seed(4)
    dy, dS = torch.randn(260, H, dv, generator=g).to(dtype), torch.randn(3, H, dk, dv, generator=g)
    x = {"q": q, "k": k, "v": v, "beta": beta, "decay": ld, "dy": dy, "state": S, "dstate": dS}
    run = lambda: [t.cpu() for t in ssd.delta_bwd(dev(q), dev(k), dev(v), dev(ld), dev(beta), ids(cu), dev(dy),   # noqa: E731
                                                  states=dev(S), dstates=dev(dS))]
    want = run()
    t = x[where]
    if where in ("state", "dstate"):
        t[1, 1, 3, 5] = NAN
    else:
        t[131, 0 if where == "q" or where == "k" else 1] = NAN
    got = run()
    for i, (a, b) in enumerate(zip(got, want)):
        if i == 5:
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, 2:], b[1, 2:])
            continue
        assert torch.equal(a[:90], b[:90]) and torch.equal(a[200:], b[200:])
        n = a.shape[1] // G   # the other group
        assert torch.equal(a[:, n:], b[:, n:])
    assert not bool(torch.isfinite(got[4][90:200]).all()) or where == "q"


def test_bwd_out_and_rows_of_no_sequence():
    G, H, dk, dv = 1, 3, 40, 24
    q, k, v, ld, beta, S = (dev(t) for t in ref.inputs(90, G, H, dk, dv, BF, True, 2, 2))
    cu = ids([5, 60, 80])
    dy = torch.ones_like(v)
    first = ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S)
    out = [torch.full_like(t, 7.0) for t in first]
    ws = torch.full((ssd.layer.delta_bwd_workspace_size(90, 2, G, H, dk, dv),), 255, dtype=torch.uint8, device="cuda")
    again = ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S, out=out, workspace=ws)
    for a, b, o in zip(first, again, out):
        assert b is o
        if a.shape[0] == 90:
            assert torch.equal(a[5:80], b[5:80]) and bool((a[:5] == 0).all()) and bool((a[80:] == 0).all())
            assert bool((b[:5] == 7).all()) and bool((b[80:] == 7).all())
        else:
            assert torch.equal(a, b)


# ---- as they are used


def problem(dtype, lens, heads=(2, 4, 64, 64), seed=0, slots=None):
    G, H, dk, dv = heads
    T = sum(lens)
    q, k, v, ld, beta, S = (dev(t) for t in ref.inputs(T, G, H, dk, dv, dtype, True, seed, slots or len(lens)))
    dy = dev(torch.randn(T, H, dv, generator=torch.Generator().manual_seed(seed + 9)).to(dtype))
    return q, k, v, ld, beta, ids(offsets(lens)), S, dy


@pytest.mark.parametrize("dtype", [F32, BF])
def test_training_step_of_a_layer(dtype):
    """The forward over a batch, the norm of its heads, and both gradients, chained as a training step does."""
    q, k, v, ld, beta, cu, S, _ = problem(dtype, [70, 58], seed=3)
    T, H, dv = v.shape
    pool = torch.zeros_like(S)
    y = ssd.delta_prefill(q, k, v, ld, beta, cu, pool, carry=ids([0, 0]))
    w, b = torch.ones(H * dv, device="cuda"), torch.zeros(H * dv, device="cuda")
    z, stats = ssd.gn_fwd(y.flatten(1), w, b, H, act="none")
    dz = torch.randn(T, H * dv, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dtype)
    dy, dw, db, _ = ssd.gn_bwd(y.flatten(1), w, b, H, stats, dz, act="none")
    got = ssd.delta_bwd(q, k, v, ld, beta, cu, dy.view(T, H, dv))
    want, err = ref.gradients(q, k, v, ld, beta, cu.tolist(), dy.view(T, H, dv))
    for n, t in zip(("dq", "dk", "dv", "dlog_decay", "dbeta"), got):
        kind = dtype if n in ("dq", "dk", "dv") else F32
        assert beyond(t, want[n], ref.gradient_bound(kind, want[n], err[n])) <= 1, n


def test_beam_search_over_recurrent_states():
    """A prompt, then steps in which beams are selected, their states reordered and stepped, against one state for each
    history that is stepped by itself."""
    G, H, dk, dv, K, V, steps = 1, 2, 32, 16, 4, 101, 6
    g = torch.Generator("cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)   # noqa: E731
    emb = [r(V, G, dk), r(V, G, dk), r(V, H, dv)]
    emb[0], emb[1] = (torch.nn.functional.normalize(x, dim=-1) for x in emb[:2])
    out = r(H * dv, V)
    ld, beta = -0.1 * torch.rand(H, device="cuda", generator=g), torch.full((1, H), 0.7, device="cuda")
    prompt = torch.randint(0, V, (9,), device="cuda", generator=g)

    def run(tokens):   # logits after these tokens, from nothing
        pool = torch.zeros(1, H, dk, dv, device="cuda")
        q, k, v = (x[tokens] for x in emb)
        y = ssd.delta_prefill(q, k, v, ld, beta.expand(len(tokens), H), ids([0, len(tokens)]), pool, carry=ids([0]))
        return y[-1].flatten() @ out

    pool = torch.zeros(7, H, dk, dv, device="cuda")
    slots = ids([5, 1, 6, 2])
    q, k, v = (x[prompt].repeat(K, 1, 1) for x in emb)
    y = ssd.delta_prefill(q, k, v, ld, beta.expand(9 * K, H), ids([0, 9, 18, 27, 36]), pool, slots=slots, carry=ids([0] * K))
    logits = (y[8::9].flatten(1) @ out).view(1, K, V)
    scores = torch.tensor([[0.0, -INF, -INF, -INF]], device="cuda")
    history = [prompt.tolist()] * K
    for _ in range(steps):
        scores, tokens, parents = ssd.beam_select(logits, scores, K)
        ssd.state_reorder(pool, parents, slots=slots)
        history = [history[p] + [t] for p, t in zip(parents[0].tolist(), tokens[0].tolist())]
        q, k, v = (x[tokens[0].long()] for x in emb)
        y = ssd.delta_step(q, k, v, ld, beta.expand(K, H), pool, slots=slots)
        logits = (y.flatten(1) @ out).view(1, K, V)
        for j in range(K):
            want = run(torch.tensor(history[j], device="cuda"))
            assert torch.allclose(logits[0, j], want, rtol=1e-3, atol=1e-3)
    assert len(set(map(tuple, history))) == K


@pytest.mark.parametrize("dtype", [F32, BF])
def test_same_results_on_any_workspace_and_every_run(dtype):
    for lens, heads in (([2000, 300], (1, 1, 128, 128)), ([130, 70], (2, 4, 48, 40))):
        q, k, v, ld, beta, cu, S, dy = problem(dtype, lens, heads, seed=7)
        args = (q, k, v, ld, beta, cu)
        T, N, (G, H, dk, dv) = sum(lens), len(lens), heads
        first = None
        for fill in (0, 255, 127):
            n = ssd.layer.delta_prefill_workspace_size(T, N, G, H, dk, dv, N)
            ws = torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")
            pool = S.clone()
            y = ssd.delta_prefill(*args, pool, workspace=ws)
            wb = torch.full((ssd.layer.delta_bwd_workspace_size(T, N, G, H, dk, dv),), fill, dtype=torch.uint8, device="cuda")
            all_ = [y, pool, *ssd.delta_bwd(*args, dy, states=S, dstates=S, workspace=wb)]
            torch.cuda.synchronize()
            first = first or all_
            assert all(torch.equal(a, b) for a, b in zip(all_, first))
    x = torch.randn(3, 4, 5001, device="cuda").to(dtype)
    sc = -torch.rand(3, 4, device="cuda")
    n = ssd.layer.beam_select_workspace_size(3, 4, 5001, 8)
    res = [ssd.beam_select(x, sc, 8, workspace=torch.full((n,), f, dtype=torch.uint8, device="cuda")) for f in (0, 255, 127)]
    assert all(torch.equal(a, b) for r in res[1:] for a, b in zip(r, res[0]))


def test_two_streams_at_once():
    """Two batches on streams of their own, each with its own workspace, give what each gives alone."""
    sets = [problem(BF, [2100, 65], (1, 2, 128, 64), seed=s) for s in (1, 2)]
    alone = []
    for q, k, v, ld, beta, cu, S, dy in sets:
        pool = S.clone()
        alone.append([ssd.delta_prefill(q, k, v, ld, beta, cu, pool), pool,
                      *ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    pools = [s[6].clone() for s in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (q, k, v, ld, beta, cu, S, dy) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                pools[i].copy_(S)
                got[i] = [ssd.delta_prefill(q, k, v, ld, beta, cu, pools[i]), pools[i],
                          *ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


def test_captured_calls_replayed():
    """Every call in two graphs, replayed in turn with eager work between, against the eager results."""
    def run(x):
        q, k, v, ld, beta, cu, S, dy, pool, logits, scores, parents = x
        pool.copy_(S)
        y = ssd.delta_prefill(q, k, v, ld, beta, cu, pool)
        z = ssd.delta_step(q[:2], k[:2], v[:2], ld[:2], beta[:2], pool)
        sel = ssd.beam_select(logits, scores, 2)
        ssd.state_reorder(pool, parents)
        return [y, z, pool, *sel, *ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S)]

    sets = []
    for s in (1, 2):
        p = problem(BF, [1700, 40], (1, 2, 128, 64), seed=s)
        g = torch.Generator("cuda").manual_seed(s)
        sets.append([*p, p[6].clone(), torch.randn(1, 2, 3000, device="cuda", generator=g),
                     torch.zeros(1, 2, device="cuda"), ids([[1, 0]])])
    eager = [[t.clone() for t in run(x)] for x in sets]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x in sets:
            run(x)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs.append(run(x))
            graphs.append(graph)
    torch.cuda.synchronize()
    for rep in range(3):
        for i in (0, 1, 1, 0):
            with torch.cuda.stream(side):
                for t in outs[i]:
                    t.fill_(0) if t.dtype != torch.bfloat16 else t.zero_()
                graphs[i].replay()
            torch.cuda.synchronize()
            run(sets[1 - i])   # eager work between
            torch.cuda.synchronize()
            for j, (a, b) in enumerate(zip(outs[i], eager[i])):
                assert torch.equal(a, b), (rep, i, j)


def test_offsets_past_32_bits():
    """Rows of v whose elements lie past 2^31, states past 2^32 bytes, beams whose states do."""
    H, dk, dv = 1, 8, 8
    big = 1 << 23                                        # row stride
    rows = 300
    base = torch.zeros(rows * big, dtype=BF, device="cuda")
    q, k, v, ld, beta, S = ref.inputs(rows, 1, H, dk, dv, BF, True, 4, 1)
    far = torch.as_strided(base, (rows, H, dv), (big, dv, 1))
    far.copy_(v)
    pool = dev(S)
    y = ssd.delta_prefill(dev(q), dev(k), far, dev(ld), dev(beta), ids([0, rows]), pool)
    want, S1, ye, Se, ym = ref.rule(q, k, v, ld, beta, [0, rows], S)
    assert beyond(y, want, ref.y_bound(BF, want, ye, ym)) <= 1 and beyond(pool, S1, Se + 1e-30) <= 1
    dy = torch.ones(rows, H, dv, dtype=BF, device="cuda")
    got = ssd.delta_bwd(dev(q), dev(k), far, dev(ld), dev(beta), ids([0, rows]), dy, states=dev(S))
    near = ssd.delta_bwd(dev(q), dev(k), dev(v), dev(ld), dev(beta), ids([0, rows]), dy, states=dev(S))
    assert all(torch.equal(a, b) for a, b in zip(got, near))
    del base, far
    slots = (1 << 32) // (128 * 128 * 4) + 3             # the last states begin past 2^32 bytes
    q, k, v, ld, beta, S = ref.inputs(2, 1, 1, 128, 128, BF, True, 4, 2)
    pool = torch.zeros(slots, 1, 128, 128, device="cuda")
    pool[-2:] = dev(S)
    ssd.delta_step(dev(q), dev(k), dev(v), dev(ld), dev(beta), pool, slots=ids([slots - 2, slots - 1]))
    want, S1, ye, Se, ym = ref.rule(q, k, v, ld, beta, [0, 1, 2], S)
    assert beyond(pool[-2:], S1, Se + 1e-30) <= 1
    before = pool[-2:].clone()
    ssd.state_reorder(pool, ids([[1, 0]]), slots=ids([slots - 2, slots - 1]))
    assert torch.equal(pool[-2:], before.flip(0)) and not bool(pool[:-2].any())


def test_another_streams_and_devices_tensors_are_refused_or_served():
    q, k, v, ld, beta, cu, S, dy = problem(F32, [20])
    with pytest.raises(ValueError):
        ssd.delta_prefill(q, k.cpu(), v, ld, beta, cu, S)
    with pytest.raises(ValueError):
        ssd.delta_prefill(q, k, v, ld, beta.cpu(), cu, S)
    with pytest.raises(TypeError):
        ssd.delta_prefill(q, k, v, ld, beta.double(), cu, S)
    with pytest.raises(ValueError):
        ssd.delta_bwd(q, k, v, ld, beta, cu, dy[:-1])
    with pytest.raises(ValueError):
        ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S[:, :, :, :-1])
    with pytest.raises(ValueError):
        ssd.beam_select(torch.zeros(1, 2, 9, device="cuda"), torch.zeros(1, 2), 2)
    with pytest.raises(ValueError):
        ssd.beam_select(torch.zeros(1, 2, 9, device="cuda"), torch.zeros(1, 2, device="cuda"), 2,
                        ended=torch.zeros(1, 2, dtype=torch.uint8, device="cuda"), end_token=9)
    with pytest.raises(ValueError):
        ssd.state_reorder(S, ids([[0, 1, 2]]).flatten())
    with pytest.raises(ssd.SsdError):
        ssd.state_reorder(S, ids([[0, 1, 2]]))   # more beams than slots


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads,stride", [((1, 1, 33, 20), (1 << 24) - 1), ((1, 2, 40, 24), (1 << 24) - 8),
                                          ((1, 1, 100, 72), (1 << 24) - 8), ((1, 1, 65, 33), 8521761),
                                          ((1, 1, 200, 40), (1 << 24) - 8)])
def test_largest_row_strides(heads, stride, dtype):
    """Rows as far apart as they may be, other values between them, against the same rows side by side."""
    G, H, dk, dv = heads
    T, cu = 97, [0, 20, 97]
    q, k, v, ld, beta, S = ref.inputs(T, G, H, dk, dv, dtype, True, 12, 2)
    dy = torch.randn(T, H, dv, generator=torch.Generator().manual_seed(2)).to(dtype)
    say(f"largest strides {heads} {stride} {dtype}")
    base, at, far = torch.full((T * stride,), 3.0, dtype=dtype, device="cuda"), 0, []
    near = [dev(x) for x in (q, k, v, dy, torch.zeros_like(dy))]
    for x in near:
        far.append(torch.as_strided(base, x.shape, (stride, x.shape[2], 1), at))
        far[-1].copy_(x)
        at += (x[0].numel() + 7) // 8 * 8
    ld, beta, S, cu = dev(ld), dev(beta), dev(S), ids(cu)
    got = []
    for q, k, v, dy, out in (near, far):
        pool = S.clone()
        y = ssd.delta_prefill(q, k, v, ld, beta, cu, pool, out=out)
        got.append([y, pool, *ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S, dstates=S)])
    torch.cuda.synchronize()
    assert len(got[0]) == 8
    for i, (a, b) in enumerate(zip(*got)):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b), i
    rows = base.view(T, stride)
    assert bool((rows[:, at:at + 4096] == 3.0).all())   # nothing written between


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,N", [(5, 0), (0, 0), (0, 2), (5, 2)])
def test_bwd_sums_over_no_rows(T, N, dtype):
    """dlog_decay [H] is the sum over the sequences' rows, of which there are none, whatever was in `out`."""
    G, H, dk, dv = 1, 300, 8, 8
    q, k, v, ld, beta, S = (dev(t) for t in ref.inputs(T, G, H, dk, dv, dtype, False, 3, N))
    out = [torch.full_like(t, 7.0) for t in (q, k, v, ld, beta, S)]
    say(f"delta_bwd sums over no rows T {T} N {N} {dtype}")
    ssd.delta_bwd(q, k, v, ld, beta, ids([0] * (N + 1)), torch.ones_like(v), states=S, dstates=S, out=out)
    assert bool((out[3] == 0).all())
    assert all(bool((t == 7.0).all()) for t in (*out[:3], out[4]))   # rows of no sequence, as they were
    assert torch.equal(out[5], S)


@pytest.mark.parametrize("heads,lens,mu", [((2, 4, 128, 128), [600, 33], -4.0), ((1, 2, 64, 128), [300], -4.0),
                                           ((1, 2, 128, 64), [300], 0.0), ((1, 1, 200, 64), [200], -8.0),
                                           ((2, 4, 33, 40), [130], -2.0), ((1, 1, 128, 128), [2500], -6.0)])
def test_prefill_in_bfloat16_rounds_y_once(heads, lens, mu):
    """Scores, states and u in y are sums of two bfloat16 numbers: 2^-18 off, and in a product of two such sums the
    least parts' product, 2^-18 at most, is left out.  So y is its own rounding and 3 2^-18 < 2^-16 of its magnitudes
    from the formula, besides what float32 sums leave."""
    G, H, dk, dv = heads
    cu = offsets(lens)
    q, k, v, ld, beta, S = ref.inputs(cu[-1], G, H, dk, dv, BF, True, 5, len(lens), mu=mu)
    say(f"delta_prefill rounds y once {heads} {lens}")
    y = ssd.delta_prefill(*(dev(t) for t in (q, k, v, ld, beta)), ids(cu), dev(S))
    want, _, ye, _, ym = ref.rule(q, k, v, ld, beta, cu, S)
    assert beyond(y, want, ref.y_bound(BF, want, ye + 2.0 ** -16 * ym, ym, rounded_inside=False)) <= 1


WHERE = ["q", "k", "v", "beta", "dy", "state", "dstate"]


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("where,bad,by_row", [(w, *c) for w in WHERE for c in ((INF, True), (-INF, True), (INF, False),
                                                                             (NAN, False))] + [("decay", INF, True)])
def test_bwd_infinities_stay_in_their_sequence(where, bad, by_row, dtype):
    """An infinity or a NaN reaches its own sequence's gradients in the heads of its group, and those heads' sums."""
    G, H, dk, dv = 2, 4, 40, 72
    cu = [0, 90, 200, 260]
    q, k, v, ld, beta, S = ref.inputs(260, G, H, dk, dv, dtype, by_row, 9, 3)
    g = torch.Generator().manual_seed(4)
    dy, dS = torch.randn(260, H, dv, generator=g).to(dtype), torch.randn(3, H, dk, dv, generator=g)
    x = {"q": q, "k": k, "v": v, "beta": beta, "decay": ld, "dy": dy, "state": S, "dstate": dS}
    say(f"delta_bwd {where} {bad} {by_row} {dtype}")
    run = lambda: [t.cpu() for t in ssd.delta_bwd(dev(q), dev(k), dev(v), dev(ld), dev(beta), ids(cu), dev(dy),   # noqa: E731
                                                  states=dev(S), dstates=dev(dS))]
    want = run()
    t = x[where]
    if where in ("state", "dstate"):
        t[1, 1, 3, 5] = bad
    else:
        t[131, 0 if where == "q" or where == "k" else 1] = bad
    got = run()
    finite = [torch.isfinite(a) for a in got]
    for i, (a, b, f) in enumerate(zip(got, want, finite)):
        if i == 5:
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, 2:], b[1, 2:])
        elif i == 3 and not by_row:
            assert torch.equal(a[2:], b[2:])
        else:
            assert torch.equal(a[:90], b[:90]) and torch.equal(a[200:], b[200:])
            n = a.shape[1] // G   # the other group
            assert torch.equal(a[:, n:], b[:, n:])
    assert not all(bool(f.all()) for f in finite)
    if not by_row:
        assert not bool(finite[3][:2].all())


def test_captured_calls_share_a_workspace():
    """Two graphs whose calls have one workspace between them, replayed in turn on one stream, against eager results."""
    heads, lens = (1, 2, 128, 64), [1700, 40]
    (G, H, dk, dv), T = heads, sum(lens)
    need = max(ssd.layer.delta_prefill_workspace_size(T, 2, G, H, dk, dv, 2), ssd.layer.delta_bwd_workspace_size(T, 2, G, H, dk, dv),
               ssd.layer.beam_select_workspace_size(2, 3, 3000, 4))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(x, ws):
        q, k, v, ld, beta, cu, S, dy, pool, logits, scores = x
        pool.copy_(S)
        y = ssd.delta_prefill(q, k, v, ld, beta, cu, pool, workspace=ws)
        sel = ssd.beam_select(logits, scores, 4, workspace=ws)
        return [y, pool, *sel, *ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S, dstates=S, workspace=ws)]

    sets = []
    for s in (1, 2):
        p = problem(BF, lens, heads, seed=s)
        g = torch.Generator("cuda").manual_seed(s)
        sets.append([*p, p[6].clone(), torch.randn(2, 3, 3000, device="cuda", generator=g), torch.zeros(2, 3, device="cuda")])
    eager = [[t.clone() for t in run(x, None)] for x in sets]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x in sets:
            run(x, ws)
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                outs.append(run(x, ws))
    torch.cuda.synchronize()
    for rep in range(3):
        ws.fill_(255)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for out in outs:
                for t in out:
                    t.zero_()
            for i in (0, 1, 1, 0):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            for j, (a, b) in enumerate(zip(outs[i], eager[i])):
                assert torch.equal(a, b), (rep, i, j)
        run(sets[rep % 2], None)   # eager work between
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_calls_follow_the_current_stream(dtype):
    """Tensors made on the default stream and handed to another one: a call waits for that stream's work alone."""
    q, k, v, ld, beta, cu, S, dy = problem(dtype, [700, 40], seed=4)
    x, sc = torch.randn(2, 3, 900, device="cuda").to(dtype), torch.zeros(2, 3, device="cuda")

    def run(v, S, x):
        pool = S.clone()
        y = ssd.delta_prefill(q, k, v, ld, beta, cu, pool)
        z = ssd.delta_step(q[:2], k[:2], v[:2], ld[:2], beta[:2], pool)
        sel = ssd.beam_select(x, sc, 2)
        ssd.state_reorder(pool, ids([[1, 0]]))
        return [y, z, pool, *sel, *ssd.delta_bwd(q, k, v, ld, beta, cu, dy, states=S)]

    want = run(v, S, x)
    late = [torch.zeros_like(t) for t in (v, S, x)]
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):   # what the stream has to do before the inputs are there
            b = a @ a
        for t, s in zip(late, (v, S, x)):
            t.copy_(s)
        got = run(*late)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(b).all())
    assert all(torch.equal(a, b) for a, b in zip(want, got))
