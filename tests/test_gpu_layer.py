"""The linear-attention layer's operators on the GPU, element by element
against their 64-bit forms (layer_ref)."""
import numpy as np
import pytest
import torch

import chunked_ssd_scan_fwd_amd as ssd
import layer_ref as ref
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def dev(t):
    return t.to("cuda")


def ids(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lens, skip=0):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32).tolist()


def fused(t):
    """A device copy of a view that keeps its strides (the slice of a projection)."""
    base = torch.empty(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype)
    base.set_(t.untyped_storage(), 0, base.shape)
    return base.to("cuda").as_strided(t.shape, t.stride(), t.storage_offset())


def check_prefill(name, heads, dtype, lens, per_token=True, carry=None, slots=None, npool=None, strided=False, tail=0,
                  max_seqlen=None, la=None, seed=0):
    G, H, dk, dv = heads
    say(f"prefill {name} {heads} {dtype} lens {lens[:6]} tail {tail} max {max_seqlen}")
    N = len(lens)
    cu = offsets(lens)
    T = cu[-1] + tail
    q, k, v, ld, S = ref.inputs(T, G, H, dk, dv, dtype, per_token, seed, npool or max(N, 1), strided)
    if la is not None:
        ld = la(ld)
    out = torch.full((T, H, dv), 7.0, dtype=dtype, device="cuda")
    pool = dev(S)
    move = fused if strided else dev
    got = ssd.lin_prefill(move(q), move(k), move(v), dev(ld), ids(cu), pool,
                          slots=None if slots is None else ids(slots), carry=None if carry is None else ids(carry),
                          max_seqlen=max(lens, default=0) if max_seqlen is None else max_seqlen, out=out)
    torch.cuda.synchronize()
    y, S1, ya, Sa = ref.scan(q, k, v, ld, cu, S, slots, carry)
    e = ref.beyond(got[:cu[-1]], y[:cu[-1]], ref.y_bound(dtype, y, ya)[:cu[-1]])
    es = ref.beyond(pool, S1, ref.state_bound(Sa))
    say(f"  y {e:.3f} states {es:.3f} of the bound")
    assert e <= 1 and es <= 1
    assert bool((got[cu[-1]:] == 7.0).all())
    untouched = sorted(set(range(S.shape[0])) - set(range(N) if slots is None else slots))
    assert torch.equal(pool.cpu()[untouched], S[untouched])
    return got, pool


HEADS = [(1, 1, 128, 128), (2, 4, 48, 40), (2, 8, 128, 128), (1, 6, 128, 64), (3, 3, 64, 64), (1, 2, 256, 128),
         (1, 2, 64, 256), (1, 1, 256, 256), (1, 2, 1, 1), (1, 3, 33, 97), (2, 2, 5, 200), (1, 1, 200, 3), (1, 1, 130, 129)]


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", HEADS)
def test_prefill_heads(heads, dtype):
    check_prefill("heads", heads, dtype, [1, 64, 130, 63, 65], per_token=heads[2] != 64, carry=[1, 0, 1, 0, 1],
                  slots=[4, 2, 0, 5, 1], npool=7, tail=3, seed=heads[2] * 7 + heads[3])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_prefill_lengths(n, dtype):
    check_prefill("length", (1, 2, 64, 128), dtype, [n], seed=n)
    check_prefill("length", (2, 2, 128, 64), dtype, [n, 3], per_token=False, seed=n)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", [(2, 4, 48, 40), (1, 3, 128, 128), (1, 2, 33, 97)])
def test_prefill_slices_of_a_projection(heads, dtype):
    check_prefill("strides", heads, dtype, [70, 0, 100], strided=True, seed=3)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("layout", ["aligned projection", "heads first", "one row repeated", "one group repeated",
                                    "states off 16 bytes", "everything off by one"])
def test_prefill_and_step_layouts(layout, dtype):
    """Strides and addresses that a caller may hand in, whole and cut."""
    for heads, lens in (((2, 4, 64, 48), [70, 0, 33]), ((1, 2, 128, 128), [600])):
        G, H, dk, dv = heads
        T, N = sum(lens), len(lens)
        q, k, v, ld, S = (dev(t) for t in ref.inputs(T, G, H, dk, dv, dtype, True, 11, N))
        out = torch.full((T, H, dv), 7.0, dtype=dtype, device="cuda")
        pool = S.clone()
        if layout == "aligned projection":
            p = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1), torch.full((T, 8), NAN, dtype=dtype, device="cuda")], 1)
            q, k, v, _ = p.split([G * dk, G * dk, H * dv, 8], 1)
            q, k, v = q.unflatten(1, (G, dk)), k.unflatten(1, (G, dk)), v.unflatten(1, (H, dv))
        elif layout == "heads first":
            q, k, v, out = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, out))
        elif layout == "one row repeated":
            k, ld = k[:1].expand(T, G, dk), ld[:1].expand(T, H)
        elif layout == "one group repeated":
            q = q[:, :1].expand(T, G, dk)
        elif layout == "states off 16 bytes":
            pool = torch.empty(S.numel() + 1, device="cuda")[1:].view(S.shape).copy_(S)
        else:
            def off(t):
                r = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
                return r.copy_(t)
            q, k, v, ld, out, pool = (off(t) for t in (q, k, v, ld, out, pool))
        say(f"layout {layout} {heads} {dtype}")
        want, S1, ya, Sa = ref.scan(q, k, v, ld, offsets(lens), S)
        y = ssd.lin_prefill(q, k, v, ld, ids(offsets(lens)), pool, out=out)
        ref.within(y, want, ref.y_bound(dtype, want, ya))
        ref.within(pool, S1, ref.state_bound(Sa))
        rows = min(T, N)
        before = pool.clone()
        y = ssd.lin_step(q[:rows], k[:rows], v[:rows], ld[:rows], pool, out=out[:rows])
        want, S1, ya, Sa = ref.scan(q[:rows], k[:rows], v[:rows], ld[:rows], list(range(rows + 1)), before)
        ref.within(y, want, ref.HALF[dtype] * want.abs() + 2e-5 * ya + (2.0 ** -25 if dtype == F16 else 0) + 1e-30)
        ref.within(pool, S1, ref.state_bound(Sa))


@pytest.mark.parametrize("heads,dtype", [((1, 1, 256, 130), BF), ((1, 2, 96, 200), F16), ((1, 1, 33, 17), F32), ((2, 2, 64, 64), BF)])
def test_prefill_cut_at_other_heads(heads, dtype):
    check_prefill("cut", heads, dtype, [1500, 700], carry=[0, 1], slots=[2, 0], npool=3, tail=2, seed=13)


@pytest.mark.parametrize("n", [2, 63, 65, 511, 512, 513])
@pytest.mark.parametrize("longest,hint", [(40, 40), (40, 1), (1700, 0)])
def test_prefill_many_ragged(n, longest, hint):
    """More blocks than the card has CUs, of lengths with gaps and ties, around the number of sequences that are
    put in order; whole (with a bound of the lengths, or one that is too low) and cut."""
    H = 8 if n > 40 else 160
    w = torch.rand(n, generator=torch.Generator().manual_seed(n)) ** 6
    lens = (w * 40).long().tolist()
    lens[n // 2], lens[n - 1] = longest, 640 if longest > 40 else 0
    got, pool = check_prefill("ragged", (2, H, 16, 8), BF, lens, carry=[i % 3 for i in range(n)],
                              slots=[(i * 7 + 3) % n if n % 7 else i for i in range(n)], max_seqlen=hint, seed=n, tail=1)


@pytest.mark.parametrize("n", [2, 3, 40, 63, 64, 65])
@pytest.mark.parametrize("hint", [700, 640, 0])
def test_prefill_ragged_long(n, hint):
    """Batches that start with their longest sequences: whole, with a bound or one that is too low, and by the
    number of rows alone."""
    H = 4096 // n
    w = torch.rand(n, generator=torch.Generator().manual_seed(n)) ** 3
    lens = (w * 300).long().tolist()
    lens[0], lens[n - 1], lens[n // 2] = 1, 700, 600 if n > 2 else 40
    check_prefill("ragged", (1, H, 8, 4), BF, lens, carry=[i % 2 for i in range(n)],
                  slots=[n - 1 - i for i in range(n)], max_seqlen=hint, seed=n, tail=3)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("lens", [[256, 128, 0, 1024, 384], [640, 640, 512], [0, 1300, 0, 0, 1]])
def test_prefill_segments_that_end_with_the_sequence(lens, dtype):
    """Lengths that are multiples of a segment's: no rest."""
    check_prefill("whole segments", (4, 64, 32, 32), dtype, lens, max_seqlen=0, seed=3, carry=[i % 2 for i in range(len(lens))])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens,max_seqlen", [([4500], 0), ([4500], 4500), ([3000, 17, 0, 1400], 0), ([2500], 5)])
def test_prefill_long(lens, max_seqlen, dtype):
    """Cut over the length: with no bound given, with the right one, and with one that is too small."""
    for heads, per_token in (((1, 1, 128, 128), True), ((1, 2, 64, 48), False)):
        check_prefill("long", heads, dtype, lens, per_token=per_token, max_seqlen=max_seqlen, seed=5,
                      carry=[1] * (len(lens) - 1) + [0] if len(lens) > 1 else None)


def test_prefill_many_short_sequences():
    lens = [(7 * i) % 5 for i in range(300)]
    check_prefill("many", (1, 2, 32, 32), BF, lens, carry=[i % 2 for i in range(300)], seed=8,
                  slots=[(i * 7) % 300 for i in range(300)])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("la", ["forget", "all", "growth", "strong", "none"])
def test_prefill_decays(la, dtype):
    def change(ld):
        ld = ld.clone()
        if la == "forget":   # the state is forgotten here and there, twice in a chunk too
            ld[[0, 10, 64, 70, 71, 130]] = -np.inf
        elif la == "all":
            ld[:] = -np.inf
        elif la == "growth":
            ld[:] = ld.abs() * 0.05
        elif la == "strong":
            ld[:] = -60.0 + ld
        else:
            ld[:] = 0
        return ld
    check_prefill("decay " + la, (1, 2, 64, 64), dtype, [150, 40], la=change, seed=2)


def test_prefill_nothing():
    q, k, v, ld, S = ref.inputs(0, 1, 2, 8, 8, BF, True, 0, 3)
    pool = dev(S)
    y = ssd.lin_prefill(dev(q), dev(k), dev(v), dev(ld), ids([0, 0, 0]), pool, carry=ids([1, 0]))
    assert y.shape == (0, 2, 8)
    S[1] = 0
    assert torch.equal(pool.cpu(), S)
    y = ssd.lin_prefill(dev(q), dev(k), dev(v), dev(ld), ids([0]), pool)
    assert y.shape == (0, 2, 8) and torch.equal(pool.cpu(), S)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("max_seqlen", [0, 1500])
def test_prefill_slots_that_cannot_be_used(max_seqlen, dtype):
    """A negative slot keeps nothing; a missing or repeated one gives NaN and writes nothing."""
    lens, slots = [70, 30, 1500, 20, 10], [-1, 2, 9, 2, 0]
    q, k, v, ld, S = ref.inputs(sum(lens), 1, 2, 64, 64, dtype, True, 4, 3)
    pool = dev(S)
    y = ssd.lin_prefill(dev(q), dev(k), dev(v), dev(ld), ids(offsets(lens)), pool, slots=ids(slots),
                        max_seqlen=max_seqlen).cpu()
    cu = offsets(lens)
    assert bool(torch.isnan(y[cu[2]:cu[4]]).all())
    for n in (0, 1, 4):
        a, b = cu[n], cu[n + 1]
        want, S1, ya, Sa = ref.scan(q[a:b], k[a:b], v[a:b], ld[a:b], [0, b - a], S, [slots[n]])
        ref.within(y[a:b], want, ref.y_bound(dtype, want, ya))
        if slots[n] >= 0:
            ref.within(pool[slots[n]], S1[slots[n]], ref.state_bound(Sa[slots[n]]))
    assert torch.equal(pool[1].cpu(), S[1])


def test_prefill_offsets_out_of_range_stay_inside():
    """Offsets below 0, past T or falling are clamped: no row outside is read or written."""
    q, k, v, ld, S = ref.inputs(50, 1, 1, 16, 16, F32, True, 4, 4)
    out = torch.full((50, 1, 16), 7.0, device="cuda")
    pool = dev(S)
    ssd.lin_prefill(dev(q), dev(k), dev(v), dev(ld), ids([-5, 20, 10, 45, 99]), pool, out=out)
    y, S1, ya, Sa = ref.scan(q, k, v, ld, [0, 20, 20, 45, 50], S)
    # sequence 2 begins at 10 although sequence 0 ended at 20: rows 10..44 are its own
    a = ref.scan(q[10:45], k[10:45], v[10:45], ld[10:45], [0, 35], S, [2])
    ref.within(pool[0], S1[0], ref.state_bound(Sa[0]))
    ref.within(pool[2], a[1][2], ref.state_bound(a[3][2]))
    ref.within(out[45:], y[45:], ref.y_bound(F32, y, ya)[45:])
    assert torch.equal(pool[1].cpu(), S[1])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_poison_stays_in_its_sequence(dtype):
    lens = [40, 33, 70]
    q, k, v, ld, S = ref.inputs(sum(lens) + 5, 1, 2, 64, 64, dtype, True, 6, 3)
    clean = [x.clone() for x in (q, k, v, ld)]
    for x in (q, k, v):
        x[40:73] = NAN
        x[143:] = np.inf
    v[73] = np.inf
    ld[143:] = NAN
    pool = dev(S)
    y = ssd.lin_prefill(dev(q), dev(k), dev(v), dev(ld), ids(offsets(lens)), pool)
    want, S1, ya, Sa = ref.scan(*clean, offsets(lens), S)
    ref.within(y[:40], want[:40], ref.y_bound(dtype, want, ya)[:40])
    ref.within(pool[0], S1[0], ref.state_bound(Sa[0]))
    assert bool(torch.isnan(y[40:73]).all()) and bool(torch.isnan(pool[1]).all())
    assert not bool(torch.isfinite(pool[2]).any())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_agrees_with_the_training_scan(dtype):
    """One sequence for each batch entry gives ssd_fwd's output."""
    B, G, H, T, dk, dv = 2, 2, 4, 300, 64, 64
    q, k, v, ld, S = ref.inputs(B * T, G, H, dk, dv, dtype, True, 9, B)
    y = ssd.lin_prefill(dev(q), dev(k), dev(v), dev(ld), ids([0, T, 2 * T]), dev(S), max_seqlen=T)
    f = lambda x: dev(x.float().view(B, T, x.shape[1], -1).transpose(1, 2).contiguous())   # noqa: E731
    want = ssd.fwd(f(q), f(k), f(v), dev(ld.view(B, T, H).transpose(1, 2).contiguous()), dev(S))
    want = want.transpose(1, 2).reshape(B * T, H, dv).cpu().double()
    _, _, ya, _ = ref.scan(q, k, v, ld, [0, T, 2 * T], S)
    ref.within(y, want, ref.y_bound(dtype, want, ya) + 2e-5 * ya)


# ---- step


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("N", [1, 5])
def test_step(N, heads, dtype):
    G, H, dk, dv = heads
    say(f"step {heads} {dtype} {N}")
    for per_token, strided in ((True, False), (False, True)):
        q, k, v, ld, S = ref.inputs(N, G, H, dk, dv, dtype, per_token, N, N + 2, strided)
        slots = [(3 * i + 1) % (N + 2) for i in range(N)] if N + 2 != 3 else [2]
        pool = dev(S)
        move = fused if strided else dev
        y = ssd.lin_step(move(q), move(k), move(v), dev(ld), pool, slots=ids(slots))
        want, S1, ya, Sa = ref.scan(q, k, v, ld, list(range(N + 1)), S, slots)
        bound = ref.HALF[dtype] * want.abs() + 2e-5 * ya + 1e-30 + (2.0 ** -25 if dtype == F16 else 0)
        ref.within(y, want, bound)
        ref.within(pool, S1, ref.state_bound(Sa))


def test_step_large_batch_and_no_slots():
    for N in (64, 65, 200):
        q, k, v, ld, S = ref.inputs(N, 1, 2, 32, 36, BF, True, N, N)
        pool = dev(S)
        y = ssd.lin_step(dev(q), dev(k), dev(v), dev(ld), pool)
        want, S1, ya, Sa = ref.scan(q, k, v, ld, list(range(N + 1)), S)
        ref.within(y, want, ref.HALF[BF] * want.abs() + 2e-5 * ya)
        ref.within(pool, S1, ref.state_bound(Sa))


@pytest.mark.parametrize("heads", [(1, 2, 64, 64), (1, 1, 33, 97), (2, 4, 128, 128)])
def test_step_padding_missing_and_repeated_slots(heads):
    G, H, dk, dv = heads
    N = 150
    q, k, v, ld, S = ref.inputs(N, G, H, dk, dv, F32, True, 4, 9)
    slots = [(i * 5) % 7 for i in range(N)]
    slots[3], slots[70], slots[149] = -1, 50, -7
    pool = dev(S)
    out = torch.full((N, H, dv), 7.0, device="cuda")
    ssd.lin_step(dev(q), dev(k), dev(v), dev(ld), pool, slots=ids(slots), out=out)
    live = [i for i in range(N) if 0 <= slots[i] < 9]
    want, S1, ya, Sa = ref.scan(q[live], k[live], v[live], ld[live], list(range(len(live) + 1)), S,
                                [slots[i] for i in live])
    ref.within(out[live], want, 2e-5 * ya + 1e-30)
    ref.within(pool, S1, ref.state_bound(Sa))
    assert bool((out[[3, 149]] == 7.0).all()) and bool(torch.isnan(out[70]).all())


def test_step_forgets():
    q, k, v, ld, S = ref.inputs(2, 1, 2, 8, 8, F32, True, 4, 2)
    ld[0] = -np.inf
    pool = dev(S)
    y = ssd.lin_step(dev(q), dev(k), dev(v), dev(ld), pool)
    want, S1, ya, Sa = ref.scan(q, k, v, ld, [0, 1, 2], S)
    ref.within(y, want, 2e-5 * ya)
    ref.within(pool, S1, ref.state_bound(Sa))


def test_steps_continue_a_prefill():
    """A prompt of 100, then 40 single tokens: the same as a prompt of 140."""
    q, k, v, ld, S = ref.inputs(140, 2, 4, 48, 40, F32, True, 4, 1)
    want, S1, ya, Sa = ref.scan(q, k, v, ld, [0, 140], S)
    pool = dev(S)
    y = [ssd.lin_prefill(dev(q[:100]), dev(k[:100]), dev(v[:100]), dev(ld[:100]), ids([0, 100]), pool)]
    for t in range(100, 140):
        y.append(ssd.lin_step(dev(q[t:t + 1]), dev(k[t:t + 1]), dev(v[t:t + 1]), dev(ld[t:t + 1]), pool))
    ref.within(torch.cat(y), want, ref.y_bound(F32, want, ya))
    ref.within(pool, S1, ref.state_bound(Sa))


def test_states_past_32_bits():
    """Slots whose states start more than 4 GiB into the pool."""
    H, dk, dv = 24, 128, 64
    per = H * dk * dv
    n = (1 << 32) // (4 * per) + 9
    say(f"pool of {n} states")
    pool = torch.zeros(n, H, dk, dv, device="cuda")
    q, k, v, ld, S = ref.inputs(70, 1, H, dk, dv, BF, True, 4, 2)
    pool[n - 1], pool[n - 5] = dev(S[0]), dev(S[1])
    y = ssd.lin_prefill(dev(q[:68]), dev(k[:68]), dev(v[:68]), dev(ld[:68]), ids([0, 68]), pool, slots=ids([n - 1]))
    y2 = ssd.lin_step(dev(q[68:]), dev(k[68:]), dev(v[68:]), dev(ld[68:]), pool, slots=ids([n - 1, n - 5]))
    want, S1, ya, Sa = ref.scan(q, k, v, ld, [0, 69, 70], S)
    y = torch.cat([y, y2])
    ref.within(y, want, ref.y_bound(BF, want, ya))
    ref.within(pool[[n - 1, n - 5]], S1, ref.state_bound(Sa))
    assert int(pool.count_nonzero()) == 2 * per
    cache = torch.zeros(n, H, dk, dv, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.zeros(n, H, dk, 2, dtype=torch.uint8, device="cuda")
    ssd.state_pack(pool, cache, scales, slots=ids([n - 1]), entries=ids([n - 2]))
    code, sc = ref.pack(pool[n - 1].cpu().numpy())
    assert np.array_equal(cache[n - 2].view(torch.uint8).cpu().numpy(), code)
    ssd.state_unpack(cache, scales, pool, slots=ids([n - 3]), entries=ids([n - 2]))
    assert np.array_equal(pool[n - 3].cpu().double().numpy(), ref.unpack(code, sc))


def test_rows_past_32_bits():
    """Rows of q, k, v and y more than 4 GiB apart from the first."""
    ld_ = (1 << 24) - 1
    n = 200
    big = torch.empty(n * ld_, dtype=BF, device="cuda")
    big2 = torch.empty(n * ld_, dtype=BF, device="cuda")
    q, k, v, la, S = ref.inputs(n, 1, 2, 64, 64, BF, True, 4, 1)
    view = lambda b, off, h: b.as_strided((n, h, 64), (ld_, 64, 1), off)   # noqa: E731
    Q, K, V, Y = view(big, 0, 1), view(big, 64, 1), view(big, 128, 2), view(big2, 3, 2)
    for to, x in ((Q, q), (K, k), (V, v)):
        to.copy_(dev(x))
    pool = dev(S)
    ssd.lin_prefill(Q, K, V, dev(la), ids([0, n]), pool, out=Y)
    want, S1, ya, Sa = ref.scan(q, k, v, la, [0, n], S)
    ref.within(Y, want, ref.y_bound(BF, want, ya))
    ref.within(pool, S1, ref.state_bound(Sa))
    x = big.as_strided((n, 128), (ld_, 1), 1)
    x.copy_(dev(torch.randn(n, 128, generator=torch.Generator().manual_seed(2))))
    check_gn(x, 2, None, "silu", "past 32 bits")


# ---- group norm


def gn_inputs(N, L, C, dtype, gated, seed=0, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    return ((r(N, L, C) * 1.5 + shift).to(dtype), r(C) * 0.3 + 1, r(C) * 0.3, r(N, L, C).to(dtype) if gated else None,
            r(N, L, C).to(dtype))


def check_gn(x, groups, gate, act, name, weight=None, bias=None, dy=None, eps=1e-5):
    """Forward, and with `dy` the gradients, against the 64-bit form and its derivatives."""
    say(f"gn {name} {tuple(x.shape)} groups {groups} {x.dtype} gate {gate is not None} {act}")
    dtype, C = x.dtype, x.shape[-1]
    w, b = (None if t is None else dev(t) for t in (weight, bias))
    y, stats = ssd.gn_fwd(x, w, b, groups, gate=gate, act=act, eps=eps)
    X = x.cpu().double().reshape(-1, x.shape[1] if x.dim() == 3 else 1, C).requires_grad_()
    N, L = X.shape[:2]
    W, B = (None if t is None else t.double().requires_grad_() for t in (weight, bias))
    Ga = None if gate is None else gate.cpu().double().reshape(X.shape).requires_grad_()
    want = ref.group_norm(X, W, B, groups, Ga, act, eps)
    # float32 sums over M values and a handful of operations on values of a
    # size with the results: 2e-5 of that size, besides the rounding at the
    # end.  The size is that of z's terms, before x - mu cancels.
    with torch.no_grad():
        xg = X.view(N, L, groups, -1)
        mu = xg.mean((1, 3), keepdim=True)
        rstd = ((xg - mu).square().mean((1, 3), keepdim=True) + eps).rsqrt()
        size = (((xg.abs() + mu.abs()) * rstd).reshape(X.shape) * (1 if W is None else W.abs()) + (0 if B is None else B.abs()))
        sg = 1.1 if Ga is None else ref.silu(Ga).abs() + 1e-3 if act == "silu" else Ga.abs()
        bound = ref.HALF[dtype] * want.abs() + 2e-5 * size * sg + (2.0 ** -25 if dtype == F16 else 0) + 1e-30
    ref.within(y.view(X.shape), want.detach(), bound)
    st = torch.stack((mu[:, 0, :, 0], rstd[:, 0, :, 0]), -1)
    amax = (xg.abs().amax((1, 3)) * rstd[:, 0, :, 0]).detach()
    ref.within(stats[..., 0], st[..., 0], 2e-6 * (xg.detach().abs().mean((1, 3)) + 1e-30))
    ref.within(stats[..., 1], st[..., 1], 2e-6 * st[..., 1] * (1 + amax))
    if dy is None:
        return
    got = ssd.gn_bwd(x, w, b, groups, stats, dy, gate=gate, act=act)
    D = dy.cpu().double().reshape(X.shape)
    ask = [X] + [t for t in (W, B, Ga) if t is not None]
    grads = dict(zip([id(t) for t in ask], torch.autograd.grad(want, ask, D)))
    with torch.no_grad():
        z = ((xg - mu) * rstd).reshape(X.shape)
        zz = z if W is None else z * W
        zz = zz if B is None else zz + B
        f = ref.silu if act == "silu" else (lambda u: u)
        u = zz if Ga is None else Ga
        sig = torch.sigmoid(u)
        df = sig * (1 + u * (1 - sig)) if act == "silu" else torch.ones_like(u)
        dz = (D * df if Ga is None else D * f(Ga)).abs()
        d = (dz * (1 if W is None else W.abs())).view_as(xg)
        # dx = rstd (d - mean d - xh mean d xh): each part's size
        part = rstd * (d + d.mean((1, 3), keepdim=True) + z.view_as(xg).abs() * (d * z.view_as(xg).abs()).mean((1, 3), keepdim=True))
        slack = 2e-5 * (1 + size)    # the relative error of xh, act' and their products
        bx = ref.HALF[dtype] * grads[id(X)].abs() + slack * (part.reshape(X.shape) + (rstd * D.view_as(xg).abs().mean((1, 3), keepdim=True)).expand_as(xg).reshape(X.shape)) + 1e-30 + (2.0 ** -25 if dtype == F16 else 0)
    ref.within(got[0].view(X.shape), grads[id(X)], bx)
    Dz = (D.abs() * (1.1 if Ga is None else f(Ga).abs())).detach()
    ones = torch.ones(C, dtype=torch.float64)
    ref.within(got[1], grads[id(W)] if W is not None else ((D * df if Ga is None else D * f(Ga)) * z).sum((0, 1)).detach(),
                      2e-5 * (Dz * size / (1 if W is None else W.abs().clamp(min=0.05)).detach() if W is not None else Dz * size).sum((0, 1)).detach() + 1e-30 * ones)
    wantb = grads[id(B)] if B is not None else (D * df if Ga is None else D * f(Ga)).sum((0, 1)).detach()
    ref.within(got[2], wantb, 2e-5 * (Dz * (1 + (size if Ga is None else 0))).sum((0, 1)).detach() + 1e-30)
    if Ga is None:
        assert got[3] is None
    else:
        bg = ref.HALF[dtype] * grads[id(Ga)].abs() + 2e-5 * D.abs() * size * 1.2 + 1e-30 + (2.0 ** -25 if dtype == F16 else 0)
        ref.within(got[3].view(X.shape), grads[id(Ga)], bg.detach())


GN = [(1, 1, 1, 1), (3, 1, 8, 8), (5, 1, 128, 1), (300, 1, 1536, 24), (33, 1, 2048, 16), (2, 1, 4104, 3), (7, 1, 30, 5),
      (4, 2, 64, 2), (2, 50, 320, 32), (3, 257, 30, 10), (1, 3000, 64, 4), (2, 9, 7, 7), (5, 5, 5, 1), (2, 1000, 3, 1),
      (1, 1, 10007, 1), (2, 3, 4096, 1), (70, 17, 96, 12), (3, 2, 8200, 8200)]


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("shape", GN)
def test_group_norm(shape, dtype):
    N, L, C, groups = shape
    for gated, act in ((True, "silu"), (False, "silu"), (True, "none"), (False, "none")):
        x, w, b, gate, dy = gn_inputs(N, L, C, dtype, gated, N + C)
        check_gn(dev(x), groups, None if gate is None else dev(gate), act, "shapes", w, b, dev(dy))


def test_group_norm_without_weights_and_two_axes():
    x, w, b, gate, dy = gn_inputs(9, 1, 48, BF, True)
    for W, Bi in ((None, None), (w, None), (None, b)):
        check_gn(dev(x[:, 0]), 6, dev(gate[:, 0]), "silu", "two axes", W, Bi, dev(dy[:, 0]))
        check_gn(dev(x.expand(9, 4, 48).contiguous()), 6, None, "silu", "no weights", W, Bi,
                 dev(dy.expand(9, 4, 48).contiguous()))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_group_norm_of_slices(dtype):
    """x, gate and dy as slices of wider rows, on boundaries of any kind."""
    for off, wide, C, groups in ((0, 200, 96, 12), (3, 251, 96, 12), (8, 128, 64, 4), (1, 67, 33, 3)):
        for L in (1, 5):
            x, w, b, gate, dy = gn_inputs(40, L, C, dtype, True, off)
            def slot(t):
                big = torch.full((40, L, wide + off), NAN, dtype=dtype, device="cuda")
                big[..., off:off + C] = dev(t)
                return big[..., off:off + C]
            check_gn(slot(x), groups, slot(gate), "silu", "slices", w, b, slot(dy))


def test_group_norm_far_mean_and_constant_groups():
    """A mean 300 deviations from zero, and groups of one value (variance 0)."""
    x, w, b, gate, dy = gn_inputs(20, 8, 64, F32, False, shift=450.0)
    check_gn(dev(x), 4, None, "silu", "far", w, b, dev(dy))
    x[:] = 3.0
    y, stats = ssd.gn_fwd(dev(x), dev(w), dev(b), 4, act="none")
    ref.within(y, b.double().expand(20, 8, 64), 2e-6 * torch.ones(1))
    ref.within(stats[..., 1], torch.full((20, 4), 1e-5, dtype=torch.float64).rsqrt(), torch.full((1,), 1e-3))


def test_group_norm_more_samples_than_a_launch_has_blocks():
    """Runs that are cut, of more samples than one grid holds: every sample's statistics and results."""
    N, L = 8_400_000, 257
    say(f"gn {N} samples of {L}")
    x = torch.empty(N, L, 1, dtype=F16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for part in x.split(1 << 20):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * 2 + 1)
    y, stats = ssd.gn_fwd(x, None, None, 1, act="none")
    dx, dw, db, _ = ssd.gn_bwd(x, None, None, 1, stats, y, act="none")
    for a in range(0, N, 1 << 20):
        X = x[a:a + (1 << 20)].float()
        var, mu = torch.var_mean(X, dim=1, correction=0, keepdim=True)
        z = (X - mu) * torch.rsqrt(var + 1e-5)
        assert float((y[a:a + (1 << 20)].float() - z).abs().max()) < 2.0 ** -11 * 8
        assert float((stats[a:a + (1 << 20), 0, 0] - mu[:, 0, 0]).abs().max()) < 1e-5
        # dy = y = xh up to its rounding: dx = rstd (xh - mean xh - xh mean xh^2) is that rounding's size
        assert float(dx[a:a + (1 << 20)].abs().max()) < 8 * 2.0 ** -10
    # sum of xh^2 over everything, N L up to roundings of y and sums of 2e9 terms
    assert abs(float(dw) / (N * L) - 1) < 1e-3


def test_group_norm_extreme_gates():
    """SiLU and its derivative where e^-u overflows or vanishes, and of infinite gates."""
    x, w, b, gate, dy = gn_inputs(4, 1, 32, F32, True)
    gate.view(-1)[:10] = torch.tensor([-1e30, -200.0, -90.0, -88.0, -20.0, 20.0, 88.0, 90.0, 200.0, 1e30])
    check_gn(dev(x), 4, dev(gate), "silu", "extreme gates", w, b, dev(dy))


def test_group_norm_poison_stays_in_its_group():
    x, w, b, gate, dy = gn_inputs(6, 3, 32, F32, False)
    clean = x.clone()
    x[2, 1, 9] = NAN
    x[4, 0, 31] = np.inf
    y, stats = ssd.gn_fwd(dev(x), dev(w), dev(b), 4)
    want, _ = ssd.gn_fwd(dev(clean), dev(w), dev(b), 4)
    bad = torch.zeros(6, 3, 32, dtype=torch.bool)
    bad[2, :, 8:16] = True
    bad[4, :, 24:] = True
    assert torch.equal(y.cpu()[~bad], want.cpu()[~bad]) and bool(torch.isnan(y.cpu()[2, :, 8:16]).all())


def test_group_norm_empty():
    w = torch.ones(8, device="cuda")
    x = torch.zeros(0, 3, 8, device="cuda")
    y, st = ssd.gn_fwd(x, w, w, 2)
    dx, dw, db, dg = ssd.gn_bwd(x, w, w, 2, st, x)
    assert y.shape == x.shape and not dw.any() and not db.any()
    x = torch.zeros(3, 0, 8, device="cuda")
    y, st = ssd.gn_fwd(x, w, w, 2)
    assert not st.any()
    dx, dw, db, dg = ssd.gn_bwd(x, w, w, 2, st, x)
    assert not dw.any() and not db.any()


def test_group_norm_gradients_against_differences():
    """The gradients of all four inputs, each by central differences in 64 bits of the same function."""
    for L, gated in ((1, True), (5, False)):
        x, w, b, gate, dy = gn_inputs(2, L, 12, F32, gated)
        _, st = ssd.gn_fwd(dev(x), dev(w), dev(b), 3, gate=None if gate is None else dev(gate))
        got = ssd.gn_bwd(dev(x), dev(w), dev(b), 3, st, dev(dy), gate=None if gate is None else dev(gate))
        args = [x.double(), w.double(), b.double()] + ([gate.double()] if gated else [])
        f = lambda a: float((ref.group_norm(a[0], a[1], a[2], 3, a[3] if gated else None, "silu", 1e-5) * dy.double()).sum())  # noqa: E731
        for i, have in zip(range(len(args)), got):
            for e in range(0, args[i].numel(), 5):
                hi, lo = [a.clone() for a in args], [a.clone() for a in args]
                hi[i].view(-1)[e] += 1e-5
                lo[i].view(-1)[e] -= 1e-5
                d = (f(hi) - f(lo)) / 2e-5
                assert abs(float(have.reshape(-1)[e]) - d) <= 1e-4 * (1 + abs(d)), (i, e)


# ---- the cache of states


def cache_of(E, H, dk, dv, fill=0):
    c = torch.full((E, H, dk, dv), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    return c, torch.full((E, H, dk, -(-dv // 32)), fill, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("heads", [(2, 128, 128), (24, 128, 64), (4, 48, 40), (1, 1, 1), (3, 33, 97), (1, 7, 31), (2, 5, 256),
                                   (1, 256, 33), (2, 3, 36)])
def test_cache(heads):
    H, dk, dv = heads
    say(f"cache {heads}")
    g = torch.Generator().manual_seed(dv)
    S = torch.randn(5, H, dk, dv, generator=g) * torch.exp(4 * torch.randn(5, H, dk, 1, generator=g))
    S[0, 0, 0] = 0
    S[1, 0, 0] = torch.tensor(1e-40)
    S[2, 0, 0, 0] = 3e38
    S[3, 0, 0, 0] = 448.0 * 2.0 ** 5
    pool = dev(S)
    cache, scales = cache_of(4, H, dk, dv, 1)
    ssd.state_pack(pool, cache, scales, slots=ids([3, 0, 1, 2]), entries=ids([1, 3, -1, 0]))
    code, sc = ref.pack(S[[2, 3, 0]].numpy())
    assert np.array_equal(cache.view(torch.uint8)[[0, 1, 3]].cpu().numpy(), code)
    assert np.array_equal(scales[[0, 1, 3]].cpu().numpy(), sc)
    assert bool((cache.view(torch.uint8)[2] == 1).all()) and bool((scales[2] == 1).all())
    ssd.state_unpack(cache, scales, pool, slots=ids([0, 4, -1, 9]), entries=ids([1, 1, 0, 0]))
    back = torch.from_numpy(ref.unpack(code[1], sc[1])).float()
    assert torch.equal(pool[0].cpu(), back) and torch.equal(pool[4].cpu(), back)
    assert torch.equal(pool[1:4].cpu(), S[1:4])


def test_cache_without_index_arrays_and_the_last_pair_counts():
    S = torch.randn(3, 2, 8, 40, generator=torch.Generator().manual_seed(1))
    cache, scales = cache_of(3, 2, 8, 40)
    ssd.state_pack(dev(S), cache, scales)
    code, sc = ref.pack(S.numpy())
    assert np.array_equal(cache.view(torch.uint8).cpu().numpy(), code) and np.array_equal(scales.cpu().numpy(), sc)
    pool = torch.zeros(3, 2, 8, 40, device="cuda")
    ssd.state_unpack(cache, scales, pool)
    assert np.array_equal(pool.cpu().double().numpy(), ref.unpack(code, sc))
    n = 150
    cache2, scales2 = cache_of(3, 2, 8, 40)
    ssd.state_pack(dev(S), cache2, scales2, slots=ids([i % 3 for i in range(n)]), entries=ids([1] * n))
    assert np.array_equal(cache2.view(torch.uint8)[1].cpu().numpy(), code[(n - 1) % 3])
    ssd.state_unpack(cache, scales, pool, slots=ids([2] * n), entries=ids([i % 3 for i in range(n)]))
    assert np.array_equal(pool[2].cpu().double().numpy(), ref.unpack(code, sc)[(n - 1) % 3])


def test_cache_of_what_is_not_finite_or_not_there():
    S = torch.ones(2, 1, 2, 64)
    S[0, 0, 0, 3], S[0, 0, 1, 40] = NAN, -np.inf
    pool = dev(S)
    cache, scales = cache_of(3, 1, 2, 64)
    ssd.state_pack(pool, cache, scales, slots=ids([0, 9]), entries=ids([0, 2]))
    ssd.state_unpack(cache, scales, pool, slots=ids([1]), entries=ids([0]))
    want = torch.ones(1, 2, 64)
    want[0, 0, :32], want[0, 1, 32:] = NAN, NAN
    assert torch.equal(torch.isnan(pool[1].cpu()), torch.isnan(want)) and float(pool[1].nan_to_num(1.0).min()) == 1.0
    assert scales[2].min() == 255
    ssd.state_unpack(cache, scales, pool, slots=ids([1]), entries=ids([5]))
    assert bool(torch.isnan(pool[1]).all())


def test_cache_rounds_ties_to_even_over_the_format():
    """Every e4m3 value, every midpoint between two, and its two neighbours in float32."""
    t = ref.e4m3_table()
    x = np.concatenate([t, (t[1:] + t[:-1]) / 2]).astype(np.float32)
    x = np.concatenate([x, np.nextafter(x, np.float32(1e9)), np.nextafter(x, np.float32(-1))])
    x = np.minimum(x, 448)
    x = np.pad(x, (0, -len(x) % 31)).reshape(-1, 31)
    S = np.concatenate([np.full((len(x), 1), 448, np.float32), x], 1)[None, None]
    S = np.concatenate([S, -S], 1)
    cache, scales = cache_of(1, *S.shape[1:])
    ssd.state_pack(dev(torch.from_numpy(S)), cache, scales)
    code, sc = ref.pack(S)
    assert np.array_equal(cache.view(torch.uint8).cpu().numpy(), code) and np.array_equal(scales.cpu().numpy(), sc)


# ---- together, graphs, streams


def layer_pass(d, pool, cache, scales, ws):
    """A prompt, its norm, its state to the cache and on to a second slot, then two tokens for both."""
    T, H, dv = d["v"].shape
    y = ssd.lin_prefill(d["q"], d["k"], d["v"], d["ld"], d["cu"], pool, slots=d["slots"], carry=d["carry"],
                        workspace=ws["prefill"])
    y = y[:d["live"]]   # the rows behind the last sequence are nobody's
    gate, dy = d["gate"][:d["live"]], d["dy"][:d["live"]]
    z, st = ssd.gn_fwd(y.view(-1, H * dv), d["w"], d["b"], H, gate=gate)
    g = ssd.gn_bwd(y.view(-1, H * dv), d["w"], d["b"], H, st, dy, gate=gate)
    ssd.state_pack(pool, cache, scales, slots=d["src"], entries=d["ent"])
    ssd.state_unpack(cache, scales, pool, slots=d["dst"], entries=d["ent"])
    s = [ssd.lin_step(d["q"][:2], d["k"][:2], d["v"][:2], d["ld"][:2], pool, slots=d["both"]) for _ in range(2)]
    z2, _ = ssd.gn_fwd(s[1].view(2, H * dv), d["w"], d["b"], H, gate=d["gate"][:2])
    return [y, z, *g, *s, z2]


def layer_data(seed, T=1300):
    q, k, v, ld, S = ref.inputs(T, 1, 2, 64, 64, BF, True, seed, 4)
    g = torch.Generator().manual_seed(seed)
    d = {"q": q, "k": k, "v": v, "ld": ld, "gate": torch.randn(T, 128, generator=g).to(BF),
         "dy": torch.randn(T, 128, generator=g).to(BF), "w": torch.rand(128, generator=g) + 0.5,
         "b": torch.randn(128, generator=g), "S": S}
    d = {n: dev(t) for n, t in d.items()}
    return d | {"live": T - 10, "cu": ids([0, T - 100, T - 10]), "slots": ids([0, 2]), "carry": ids([0, 1]), "src": ids([0]), "ent": ids([1]),
                "dst": ids([3]), "both": ids([0, 3])}


def test_the_operators_together():
    d = layer_data(1)
    pool = d["S"].clone()
    cache, scales = cache_of(2, 2, 64, 64)
    ws = {"prefill": None}
    out = layer_pass(d, pool, cache, scales, ws)
    c = {n: t.cpu() for n, t in d.items() if n != "live"}
    y, S1, ya, Sa = ref.scan(c["q"], c["k"], c["v"], c["ld"], c["cu"], c["S"], c["slots"], c["carry"])
    ref.within(out[0], y[:1290], ref.y_bound(BF, y, ya)[:1290])
    # from here on, each step against the reference on what the one before it gave
    yy = out[0].cpu().double().view(-1, 1, 128)
    z = ref.group_norm(yy, c["w"].double(), c["b"].double(), 2, c["gate"][:1290].double()[:, None], "silu", 1e-5)
    big = z.abs() + 1
    ref.within(out[1].view(z.shape), z, 2.0 ** -8 * z.abs() + 1e-3 * big * 2.0 ** -6)
    S = S1.float()
    code, sc = ref.pack(S[0].numpy())
    got = ref.unpack(cache[1].view(torch.uint8).cpu().numpy(), scales[1].cpu().numpy())
    step = np.repeat(2.0 ** (scales[1].cpu().numpy().astype(float) - 127), 32, -1)
    bound = np.maximum(2.0 ** -4 * np.abs(S[0].numpy()), 2.0 ** -10 * step) * 1.001 + 2e-5 * Sa[0].numpy()
    assert (np.abs(got - S1[0].numpy()) <= bound).all()
    S = S1.clone()
    S[3] = torch.from_numpy(got)
    Aa = S.abs() + Sa
    for i in range(2):
        y2, S, ya2, _ = ref.scan(c["q"][:2], c["k"][:2], c["v"][:2], c["ld"][:2], [0, 1, 2], S, c["both"])
        ya2 = ya2 + (c["q"][:2].double().abs().repeat_interleave(2, 1)[:, :, None, :] @ Aa[[0, 3]])[:, :, 0]
        have = out[6 + i]
        ref.within(have, y2, 2.0 ** -8 * y2.abs() + 1e-4 * ya2)
    ref.within(pool[[0, 3]], S[[0, 3]], 1e-4 * Aa[[0, 3]])


def test_results_repeat_whatever_the_workspace_held():
    d = layer_data(2, 5000)
    runs = []
    need = ssd.layer.lin_prefill_workspace_size(5000, 2, 1, 2, 64, 64, 4)
    for fill in (0, 255, 127):
        pool = d["S"].clone()
        cache, scales = cache_of(2, 2, 64, 64)
        ws = {"prefill": torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda")}
        runs.append(layer_pass(d, pool, cache, scales, ws) + [pool])
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_graphs_on_a_side_stream():
    """Two captured passes with workspaces of their own, replayed in turn with eager work between."""
    side = torch.cuda.Stream()
    sets = []
    with torch.cuda.stream(side):
        for seed in (3, 4):
            d = layer_data(seed)
            n = max(16, ssd.layer.lin_prefill_workspace_size(1300, 2, 1, 2, 64, 64, 4))
            ws = {"prefill": torch.empty(n, dtype=torch.uint8, device="cuda")}
            pool = d["S"].clone()
            cache, scales = cache_of(2, 2, 64, 64)
            layer_pass(d, pool, cache, scales, ws)   # warm
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = layer_pass(d, pool, cache, scales, ws)
            sets.append((d, ws, pool, cache, scales, graph, out))
    torch.cuda.synchronize()
    for again in range(4):
        for d, ws, pool, cache, scales, graph, out in sets:
            d["v"].mul_(0.9)
            p2 = d["S"].clone()
            c2, s2 = cache_of(2, 2, 64, 64)
            want = layer_pass(d, p2, c2, s2, {"prefill": None})
            pool.copy_(d["S"])
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out + [pool], want + [p2]):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    """The same calls on two streams, each with its own data, not ordered against each other."""
    sets = [layer_data(s, 3000) for s in (5, 6)]
    want = []
    for d in sets:
        pool, (cache, scales) = d["S"].clone(), cache_of(2, 2, 64, 64)
        want.append(layer_pass(d, pool, cache, scales, {"prefill": None}) + [pool])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for d, st in zip(sets, streams):
        with torch.cuda.stream(st):
            for _ in range(3):
                pool, (cache, scales) = d["S"].clone(), cache_of(2, 2, 64, 64)
                out = layer_pass(d, pool, cache, scales, {"prefill": None}) + [pool]
        got.append(out)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_cache_off_16_bytes():
    S = torch.randn(3, 2, 8, 64, generator=torch.Generator().manual_seed(1))
    pool = torch.empty(S.numel() + 1, device="cuda")[1:].view(S.shape).copy_(S)
    raw = torch.zeros(S.numel() + 3, dtype=torch.uint8, device="cuda")[3:].view(S.shape)
    cache, scales = raw.view(torch.float8_e4m3fn), torch.zeros(3, 2, 8, 2, dtype=torch.uint8, device="cuda")
    ssd.state_pack(pool, cache, scales)
    code, sc = ref.pack(S.numpy())
    assert np.array_equal(raw.cpu().numpy(), code) and np.array_equal(scales.cpu().numpy(), sc)
    ssd.state_unpack(cache, scales, pool)
    assert np.array_equal(pool.cpu().double().numpy(), ref.unpack(code, sc))


def test_binding_refuses():
    q, k, v, ld, S = (dev(t) for t in ref.inputs(6, 1, 2, 8, 8, BF, True, 0, 3))
    cu = ids([0, 6])
    ok = dict(q=q, k=k, v=v, log_decay=ld, cu_seqlens=cu, states=S)
    ssd.lin_prefill(**ok)
    for bad, err in ((dict(k=k.float()), TypeError), (dict(v=v[:5]), ValueError), (dict(states=S.half()), TypeError),
                     (dict(states=S.transpose(2, 3)), ValueError), (dict(cu_seqlens=cu.long()), TypeError),
                     (dict(cu_seqlens=cu.cpu()), ValueError), (dict(log_decay=ld[:5]), ValueError),
                     (dict(log_decay=ld.double()), TypeError), (dict(slots=ids([0, 1])), ValueError),
                     (dict(carry=ids([0]).float()), TypeError), (dict(max_seqlen=-3), ValueError),
                     (dict(out=torch.empty(6, 2, 8, device="cuda")), TypeError),
                     (dict(out=torch.empty(1, 2, 8, dtype=BF, device="cuda").expand(6, 2, 8)), ssd.SsdError),
                     (dict(q=q.transpose(0, 2).contiguous().transpose(0, 2)), ValueError),
                     (dict(cu_seqlens=ids([0, 1, 2, 3, 6])), ssd.SsdError)):   # four sequences, three slots
        with pytest.raises(err):
            ssd.lin_prefill(**(ok | bad))
    with pytest.raises(ssd.SsdError):
        ssd.lin_step(q, k, v, ld, S)   # six rows, three slots
    w = torch.ones(8, device="cuda")
    x = torch.ones(4, 3, 8, device="cuda")
    for bad, err in ((dict(groups=3), ValueError), (dict(weight=w[:7]), ValueError), (dict(weight=w.half()), TypeError),
                     (dict(gate=x[:3]), ValueError), (dict(act="relu"), ValueError), (dict(eps=-1.0), ValueError),
                     (dict(x=x.transpose(0, 1)), ValueError), (dict(x=x[:1].expand(4, 3, 8)), ValueError),
                     (dict(out=x[..., :4]), ValueError), (dict(stats=torch.empty(4, 2, device="cuda")), ValueError)):
        with pytest.raises(err):
            ssd.gn_fwd(**(dict(x=x, weight=w, bias=w, groups=2) | bad))
    with pytest.raises(TypeError):
        ssd.state_pack(S, torch.zeros(3, 2, 8, 8, device="cuda"), torch.zeros(3, 2, 8, 1, dtype=torch.uint8, device="cuda"))
    c, s = cache_of(3, 2, 8, 8)
    with pytest.raises(ValueError):
        ssd.state_pack(S, c, s, slots=ids([0, 1]), entries=ids([0]))


def test_cache_scales_past_32_bits():
    """Entries whose scales start 2^32 bytes into their array; the first entries' stay as they are."""
    H, dk, n = 16, 256, (1 << 20) + 2
    say(f"cache of {n} entries of {H} x {dk} x 1")
    cache, scales = cache_of(n, H, dk, 1)
    S = torch.randn(2, H, dk, 1, generator=torch.Generator().manual_seed(7)) * 3.0
    pool = dev(S)
    ssd.state_pack(pool, cache, scales, slots=ids([0, 1]), entries=ids([n - 2, n - 1]))
    code, sc = ref.pack(S.numpy())
    assert np.array_equal(cache[n - 2:].view(torch.uint8).cpu().numpy(), code)
    assert np.array_equal(scales[n - 2:].cpu().numpy(), sc)
    assert not bool(cache[:2].view(torch.uint8).any()) and not bool(scales[:2].any())
    pool.zero_()
    ssd.state_unpack(cache, scales, pool, slots=ids([1, 0]), entries=ids([n - 2, n - 1]))
    assert np.array_equal(pool.cpu().double().numpy(), ref.unpack(code, sc)[::-1])


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", [(1, 2, 64, 64), (1, 1, 128, 128), (1, 1, 200, 48)])
@pytest.mark.parametrize("T,at", [(90, 5), (90, 70), (1500, 5), (1500, 700), (1500, 1490)])
def test_prefill_state_of_one_row(T, at, heads, dtype):
    """float32 accuracy of a state that one row makes and nothing fades, whole and cut.

    The state is k v^T.  It may go through v times a decay of the chunk and
    back: the two factors, the products with them and the sum of the product's
    parts are a dozen roundings of 2^-24, within 2^-20.  v times a decay in two
    bfloat16 parts would be off by up to 2^-16."""
    G, H, dk, dv = heads
    say(f"one row {heads} {dtype} T {T} at {at}")
    q, k, v, _, S = ref.inputs(T, G, H, dk, dv, dtype, True, 21, 1)
    row = k[at].clone()
    k.zero_()
    k[at] = row
    ld = torch.zeros(T, H)
    ld[at] = -0.3
    pool = dev(S)
    ssd.lin_prefill(dev(q), dev(k), dev(v), dev(ld), ids([0, T]), pool, carry=ids([0]))
    want = ref.scan(q, k, v, ld, [0, T], S, carry=[0])[1]
    ref.within(pool, want, 2.0 ** -20 * want.abs() + 1e-30)


@pytest.mark.parametrize("la,dtype", [(la, d) for la in ("forget", "all", "growth", "strong", "none", "slow") for d in (F32, BF, F16)
                                      if (la, d) != ("growth", F16)])   # there y passes float16's 65504
def test_prefill_decays_of_cut_sequences(la, dtype):
    def change(ld):
        ld = ld.clone()
        if la == "forget":   # first, last and inner rows of chunks, segments and sequences
            ld[[0, 10, 64, 70, 71, 127, 128, 130, 255, 256, 800, 1499, 1500, 2000]] = -np.inf
        elif la == "all":
            ld[:] = -np.inf
        elif la == "growth":
            ld[:] = ld.abs() * 0.05
        elif la == "strong":
            ld[:] = -60.0 + ld
        else:
            ld[:] = -1e-4 if la == "slow" else 0
        return ld
    check_prefill("cut, decay " + la, (1, 2, 64, 64), dtype, [1500, 700], la=change, seed=2, max_seqlen=0)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("heads", [(1, 2, 64, 64), (1, 1, 64, 128), (1, 1, 128, 64), (1, 1, 128, 128), (1, 1, 256, 64), (1, 2, 33, 97)])
@pytest.mark.parametrize("T,rows", [(130, (0, 17, 63, 100)), (1100, (300, 1050))])
def test_prefill_poison_reaches_no_earlier_row(T, rows, heads, dtype):
    """One infinity or NaN among the inputs: rows before it, columns beside it in v and other heads' results are
    what they are without it; what it does reach is not finite; an infinite v makes the state infinite, by its sign."""
    G, H, dk, dv = heads
    base = dict(zip(("q", "k", "v", "ld", "S"), ref.inputs(T, G, H, dk, dv, dtype, True, 5, 1, la_mu=-5.0)))
    y0, S0, ya, Sa = ref.scan(*(base[n] for n in ("q", "k", "v", "ld")), [0, T], base["S"])
    yb, Sb = ref.y_bound(dtype, y0, ya), ref.state_bound(Sa)
    col, h = dv // 2, H - 1
    where = {"q": (0, 0), "k": (0, dk // 2), "v": (h, col), "ld": (h,)}
    others = [c for c in range(dv) if c != col]
    for at in rows:
        for name, bad in (("v", np.inf), ("v", -np.inf), ("v", NAN), ("k", np.inf), ("q", NAN), ("ld", NAN)):
            say(f"{bad} in {name} {heads} {dtype} T {T} row {at}")
            x = {n: t.clone() for n, t in base.items()}
            x[name][(at, *where[name])] = bad
            pool = dev(x["S"])
            y = ssd.lin_prefill(*(dev(x[n]) for n in ("q", "k", "v", "ld")), ids([0, T]), pool, max_seqlen=0).cpu()
            S = pool.cpu()
            ref.within(y[:at], y0[:at], yb[:at])
            if name == "v":
                ref.within(y[:, h, others], y0[:, h, others], yb[:, h, others])
                ref.within(S[0, h][:, others], S0[0, h][:, others], Sb[0, h][:, others])
                assert not bool(torch.isfinite(y[at:, h, col]).any())
                # k times it: infinities of either sign, or NaN
                np.testing.assert_array_equal(S[0, h, :, col].double().numpy(), (x["k"][at, 0].double() * bad).numpy())
            elif name == "k":
                rest = [r for r in range(dk) if r != dk // 2]
                ref.within(S[0][:, rest], S0[0][:, rest], Sb[0][:, rest])
                assert not bool(torch.isfinite(S[0][:, dk // 2]).any())
            elif name == "q":
                assert not bool(torch.isfinite(y[at]).any())
                ref.within(y[at + 1:], y0[at + 1:], yb[at + 1:])
                ref.within(S, S0, Sb)
            else:
                assert not bool(torch.isfinite(y[at:, h]).any()) and not bool(torch.isfinite(S[0, h]).any())
            if name in ("v", "ld"):   # the other heads
                ref.within(y[:, :h], y0[:, :h], yb[:, :h])
                ref.within(S[0, :h], S0[0, :h], Sb[0, :h])


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("L", [1, 5, 700])
def test_group_norm_of_infinite_gates(L, dtype):
    """SiLU of +infinity is infinite, of -infinity NaN, its derivative at both NaN; what belongs to other places,
    channels and runs stays as it is."""
    x, w, b, gate, dy = (dev(t) for t in gn_inputs(4, L, 32, dtype, True))
    bad = gate.clone()
    bad[1, 0, 3], bad[2, L - 1, 30] = np.inf, -np.inf

    def run(g):
        y, st = ssd.gn_fwd(x, w, b, 4, gate=g)
        return (y, *ssd.gn_bwd(x, w, b, 4, st, dy, gate=g))
    (y, dx, dw, db, dg), clean = run(bad), run(gate)
    place = torch.zeros(4, L, 32, dtype=torch.bool, device="cuda")
    place[1, 0, 3] = place[2, L - 1, 30] = True
    run_of = torch.zeros_like(place)
    run_of[1, :, :8] = run_of[2, :, 24:] = True
    channel = place.any(0).any(0)
    assert bool(torch.isinf(y[1, 0, 3])) and bool(torch.isnan(y[2, L - 1, 30])) and bool(torch.isnan(dg[place]).all())
    for got, want, where in zip((y, dx, dw, db, dg), clean, (place, run_of, channel, channel, place)):
        assert not bool(torch.isfinite(got[where]).any())
        assert torch.equal(got[~where], want[~where])


def test_cache_binding_refuses_index_arrays():
    """What is no tensor, of no axis or of more than one, of another type, on the host, or not dense."""
    S = torch.ones(4, 1, 2, 8, device="cuda")
    cache, scales = cache_of(4, 1, 2, 8)
    for bad, err in (([0, 1], TypeError), (np.zeros(2, np.int32), TypeError), (ids([0, 1]).long(), TypeError),
                     (ids([[0, 1]]), ValueError), (ids(0), ValueError), (ids([0, 1]).cpu(), ValueError),
                     (ids([0, 1, 2, 3])[::2], ValueError)):
        for name in ("slots", "entries"):
            other = {"slots": "entries", "entries": "slots"}[name]
            for given in ({name: bad}, {name: bad, other: ids([1, 0])}):
                with pytest.raises(err):
                    ssd.state_pack(S, cache, scales, **given)
                with pytest.raises(err):
                    ssd.state_unpack(cache, scales, S, **given)
    assert bool((S == 1).all()) and not bool(scales.any())
