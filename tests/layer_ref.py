"""Plain 64-bit forms of the linear-attention layer's operators, for its tests.

Each also gives what its result's error is measured in: the same sum over the
terms' magnitudes, since a rounding of a term or of a partial sum is relative
to the magnitudes that were added, whatever cancels in the result.
"""
import math

import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a rounding step


def scan(q, k, v, log_decay, cu, states, slots=None, carry=None):
    """(y, states, y_abs, states_abs) of the packed scan, row by row."""
    T, G, dk = q.shape
    H, dv = v.shape[1:]
    rep = H // G
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    la = log_decay.detach().cpu().double()
    la = la.expand(T, H) if la.dim() == 1 else la
    cu = [int(c) for c in cu]
    out = states.detach().cpu().double().clone()
    out_abs = out.abs()
    y = torch.zeros(T, H, dv, dtype=torch.float64)
    y_abs = torch.zeros_like(y)
    for n in range(len(cu) - 1):
        sl = n if slots is None else int(slots[n])
        fresh = sl < 0 or (carry is not None and int(carry[n]) == 0)
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if fresh else out[sl].clone()
        # magnitudes carry over from sequence to sequence of a slot, as the errors do
        A = torch.zeros_like(S) if fresh else out_abs[sl].clone()
        for t in range(cu[n], cu[n + 1]):
            a = torch.exp(la[t])[:, None, None]
            kv = k[t].repeat_interleave(rep, 0)[:, :, None] * v[t][:, None, :]
            qt = q[t].repeat_interleave(rep, 0)[:, None, :]
            S = a * S + kv
            A = a * A + kv.abs()
            y[t] = (qt @ S)[:, 0]
            y_abs[t] = (qt.abs() @ A)[:, 0]
        if sl >= 0:
            out[sl], out_abs[sl] = S, A
    return y, out, y_abs, out_abs


def silu(u):
    return u * torch.sigmoid(u)


def group_norm(x, weight, bias, groups, gate, act, eps):
    """y in 64 bits, differentiable."""
    N, L, C = x.shape
    xg = x.view(N, L, groups, C // groups)
    mu = xg.mean((1, 3), keepdim=True)
    var = (xg - mu).square().mean((1, 3), keepdim=True)
    z = ((xg - mu) / (var + eps).sqrt()).reshape(N, L, C)
    z = z if weight is None else z * weight
    z = z if bias is None else z + bias
    f = silu if act == "silu" else (lambda u: u)
    return f(z) if gate is None else z * f(gate)


def e4m3_table():
    """The finite e4m3 values by their bytes 0..126, from the format's definition."""
    return np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for b in range(127) for e, m in [(b >> 3, b & 7)]])


def pack(states):
    """(bytes, scales) of finite float32 states [..., dv], by search among the format's values."""
    x = np.asarray(states, dtype=np.float64)
    dv = x.shape[-1]
    nb = -(-dv // 32)
    xb = np.zeros(x.shape[:-1] + (nb * 32,))
    xb[..., :dv] = x
    xb = xb.reshape(x.shape[:-1] + (nb, 32))
    big = np.abs(xb).max(-1)
    s = np.full(big.shape, -127.0)
    nz = big > 0
    s[nz] = np.maximum(np.ceil(np.log2(big[nz] / 448.0)), -127)
    # ceil of a rounded logarithm may be one off: the definition decides
    s[nz] = np.where(big[nz] > 448 * 2.0 ** s[nz], s[nz] + 1, s[nz])
    s[nz] = np.where((s[nz] > -127) & (big[nz] <= 448 * 2.0 ** (s[nz] - 1)), s[nz] - 1, s[nz])
    tab = e4m3_table()
    val = np.abs(xb) * 2.0 ** -s[..., None]
    hi = np.clip(np.searchsorted(tab, val), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = val - tab[lo], tab[hi] - val
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(val >= tab[126], 126, code).astype(np.uint8) | (np.signbit(xb).astype(np.uint8) << 7)
    code = code.reshape(x.shape[:-1] + (nb * 32,))[..., :dv]
    return np.ascontiguousarray(code), (s + 127).astype(np.uint8)


def unpack(code, scales):
    tab = np.concatenate([e4m3_table(), [np.nan]])
    v = tab[code & 127] * np.where(code & 128, -1.0, 1.0)
    sc = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(sc, 32, axis=-1)[..., :code.shape[-1]]


def inputs(rows, G, H, dk, dv, dtype, per_token, seed, slots, fused=False, la_mu=-2.0):
    """q, k, v, log_decay, states on the CPU; `fused`: slices of one projection's rows."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    if fused:
        p = r(rows, 2 * G * dk + H * dv + 5)
        p[:, :2 * G * dk] *= dk ** -0.25
        p = p.to(dtype)
        q, k, v = p[:, :2 * G * dk + H * dv].split([G * dk, G * dk, H * dv], 1)
        q, k, v = q.unflatten(1, (G, dk)), k.unflatten(1, (G, dk)), v.unflatten(1, (H, dv))
    else:
        q, k, v = ((r(rows, G, dk) * dk ** -0.25).to(dtype), (r(rows, G, dk) * dk ** -0.25).to(dtype),
                   r(rows, H, dv).to(dtype))
    la = -torch.nn.functional.softplus(r(rows, H) + la_mu) if per_token else torch.log1p(
        -torch.exp2(-2.0 - 5.0 * torch.arange(H) / max(1, H - 1)))
    return q, k, v, la, r(slots, H, dk, dv)


def y_bound(dtype, y, y_abs):
    """How far y may be off: one rounding to its type; for 16-bit types the
    masked scores and the state that meet the products may be rounded to the
    type as well, once for each term (a term goes through one of them);
    2e-5 of the terms for float32 sums, exponentials and products of decays."""
    inner = HALF[dtype] * (1 + HALF[dtype]) if dtype == torch.bfloat16 else 0.0
    return (HALF[dtype] * (y.abs() + inner * y_abs) + inner * y_abs + 2e-5 * y_abs + 1e-30
            + (2.0 ** -25 if dtype == torch.float16 else 0.0))   # half the smallest float16


def state_bound(states_abs):
    return 2e-5 * states_abs + 1e-30


def within(got, want, bound):
    __tracebackhide__ = True
    r = beyond(got, want, bound)
    assert r <= 1, f"{r} of the bound"


def beyond(got, want, bound):
    """The largest excess over the bound, as a ratio (fails on NaN)."""
    d = (got.detach().cpu().double() - want).abs()
    r = (d / bound)
    return math.inf if bool(torch.isnan(r).any()) else float(r.max()) if r.numel() else 0.0
