"""Plain 64-bit forms of the gated delta rule for its tests, row by row, with
what the results' errors are measured in.

Errors.  With rho_t = max(1, |1 - beta_t |k_t|^2|), the 2-norm of
I - beta k k^T, an error that a column c of the state has before step t is at
most a_t rho_t times itself after it.  A step adds its own: float32 products,
sums over dk and over a chunk's rows, exponentials and differences of sums of
log decays, in all at most STEP of the 2-norms that it adds up,
    a_t |S_{t-1}(c)| + |k_t| beta_t (|v_t(c)| + a_t |k_t| |S_{t-1}(c)|).
`err` is that sum carried on.  y adds |q_t| err and one rounding; bfloat16
calls round what meets q too, the state as it entered the chunk and the
scores, each term in one of them: half a step of |q_t| H_t(c), where
H_t = a_t H_{t-1} + |k_t| |u_t| counts every term by its magnitude.
"""
import torch

from layer_ref import HALF

STEP = 2.0 ** -20   # 16 float32 half steps


def rule(q, k, v, log_decay, beta, cu, states, slots=None, carry=None):
    """(y, states, y's bound without its roundings, states' bound, y's magnitudes) of the packed batch."""
    T, G, dk = q.shape
    H, dv = v.shape[1:]
    q, k, v, beta = (x.detach().cpu().double() for x in (q, k, v, beta))
    q, k = (x.repeat_interleave(H // G, 1) for x in (q, k))
    la = log_decay.detach().cpu().double()
    la = la.expand(T, H) if la.dim() == 1 else la
    cu = [int(c) for c in cu]
    out = states.detach().cpu().double().clone()
    out_err = torch.zeros(out.shape[0], H, dv, dtype=torch.float64)
    out_mag = out.norm(dim=2)
    y = torch.zeros(T, H, dv, dtype=torch.float64)
    y_err, y_mag = torch.zeros_like(y), torch.zeros_like(y)
    for n in range(len(cu) - 1):
        sl = n if slots is None else int(slots[n])
        fresh = sl < 0 or (carry is not None and int(carry[n]) == 0)
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if fresh else out[sl].clone()
        err = torch.zeros(H, dv, dtype=torch.float64) if fresh else out_err[sl].clone()
        mag = torch.zeros(H, dv, dtype=torch.float64) if fresh else out_mag[sl].clone()
        for t in range(cu[n], cu[n + 1]):
            a, b, kt = la[t].exp()[:, None], beta[t][:, None], k[t]
            kn = kt.norm(dim=1)[:, None]
            size = a * S.norm(dim=1)
            rho = (1 - b * kn * kn).abs().clamp(min=1)
            err = a * rho * err + STEP * (size + kn * b.abs() * (v[t].abs() + kn * size))
            S = a[..., None] * S
            u = b * (v[t] - (kt[:, None, :] @ S)[:, 0])
            S = S + kt[..., None] * u[:, None, :]
            mag = a * mag + kn * u.abs()
            qn = q[t].norm(dim=1)[:, None]
            y[t] = (q[t][:, None, :] @ S)[:, 0]
            y_err[t], y_mag[t] = qn * (err + STEP * mag), qn * mag
        if sl >= 0:
            out[sl], out_err[sl], out_mag[sl] = S, err, mag
    return y, out, y_err, out_err[:, :, None, :].expand_as(out), y_mag


def y_bound(dtype, y, y_err, y_mag, rounded_inside=True):
    inner = HALF[dtype] * (1 + HALF[dtype]) if dtype == torch.bfloat16 and rounded_inside else 0.0
    bound = inner * y_mag + y_err
    return (HALF[dtype] * (y.abs() + bound) + bound + 1e-30
            + (2.0 ** -25 if dtype == torch.float16 else 0.0))   # half the smallest float16


def inputs(rows, G, H, dk, dv, dtype, per_token, seed, slots, fused=False, mu=-4.0, near=0.0):
    """q, k, v, log_decay, beta, states on the CPU, k of length 1; `fused`: slices of one projection's rows;
    `near`: how much all keys have in common."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    p = r(rows, 2 * G * dk + H * dv + (5 if fused else 0))
    qk = p[:, :2 * G * dk].unflatten(1, (2 * G, dk))
    if near:
        qk.mul_(1 - near).add_(near * r(1, 1, dk) * dk ** 0.5)
    qk.div_(qk.norm(dim=-1, keepdim=True).clamp(min=1e-6))
    p = p.to(dtype)
    q, k, v = p[:, :2 * G * dk + H * dv].split([G * dk, G * dk, H * dv], 1)
    q, k, v = q.unflatten(1, (G, dk)), k.unflatten(1, (G, dk)), v.unflatten(1, (H, dv))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    la = -torch.nn.functional.softplus(r(rows, H) + mu) if per_token else torch.log1p(
        -torch.exp2(-2.0 - 5.0 * torch.arange(H) / max(1, H - 1)))
    return q, k, v, la, torch.sigmoid(r(rows, H)), r(slots, H, dk, dv) * 0.5


def gradients(q, k, v, log_decay, beta, cu, dy, states=None, dstates=None):
    """({name: gradient}, {name: bound without the last rounding}) of sum(dy y) + sum(dstates last states), by the
    adjoint of each row's step.

    Bounds, by columns as in the forward's: an error of the adjoint state G goes through the transposed step, which
    grows it by a_t rho_t at most, and a step adds STEP of the norms that it adds up.  A gradient that is a product of
    two such values is off by each one's error times the other's norm.  dlog_decay is put together from products
    inside a chunk (of 64 rows at most), whose terms count by their magnitudes over all rows within 64 of its own."""
    T, G_, dk = q.shape
    H, dv = v.shape[1:]
    rep = H // G_
    q, k, v, beta, dy = (x.detach().cpu().double() for x in (q, k, v, beta, dy))
    q, k = (x.repeat_interleave(rep, 1) for x in (q, k))
    by_row = log_decay.dim() == 2
    la = log_decay.detach().cpu().double().expand(T, H)
    N = len(cu) - 1
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)   # noqa: E731
    g = {"dq": z(T, H, dk), "dk": z(T, H, dk), "dv": z(T, H, dv), "dlog_decay": z(T, H), "dbeta": z(T, H),
         "dstates": z(N, H, dk, dv)}
    e = {n: torch.zeros_like(x) for n, x in g.items()}
    for n in range(N):
        S = z(H, dk, dv) if states is None else states[n].detach().cpu().double()
        err, mag = z(H, dv), S.norm(dim=1)
        kept = []
        for t in range(int(cu[n]), int(cu[n + 1])):
            a, b, kt = la[t].exp()[:, None], beta[t][:, None], k[t]
            kn = kt.norm(dim=1)[:, None]
            rho = (1 - b * kn * kn).abs().clamp(min=1)
            aS = a[..., None] * S
            ev = v[t] - (kt[:, None, :] @ aS)[:, 0]
            size = aS.norm(dim=1)
            e_in = a * err + STEP * a * mag                         # of a S
            e_ev = kn * e_in + STEP * (v[t].abs() + kn * size)      # of v - a S^T k
            kept.append((aS, ev, e_in, e_ev, a * mag))
            err = a * rho * err + STEP * (size + kn * b.abs() * (v[t].abs() + kn * size))
            S = aS + kt[..., None] * (b * ev)[:, None, :]
            mag = a * mag + kn * (b * ev).abs()
        A = z(H, dk, dv) if dstates is None else dstates[n].detach().cpu().double()
        ge, gm = z(H, dv), A.norm(dim=1)
        rows = []
        for t in reversed(range(int(cu[n]), int(cu[n + 1]))):
            aS, ev, e_in, e_ev, mag = kept.pop()
            a, b, kt, d = la[t].exp()[:, None], beta[t][:, None], k[t], dy[t]
            kn, qn = kt.norm(dim=1)[:, None], q[t].norm(dim=1)[:, None]
            rho = (1 - b * kn * kn).abs().clamp(min=1)
            S = aS + kt[..., None] * (b * ev)[:, None, :]
            e_S, m_S = e_in + kn * b.abs() * e_ev, mag + kn * (b * ev).abs()
            A = A + q[t][..., None] * d[:, None, :]
            gm = gm + qn * d.abs()
            ge = ge + STEP * gm
            g["dq"][t] = (S @ d[..., None])[..., 0]
            e["dq"][t] = (d.abs() * (e_S + STEP * m_S)).sum(-1, keepdim=True)
            du = (kt[:, None, :] @ A)[:, 0]
            e_du = kn * (ge + STEP * gm)
            g["dbeta"][t] = (du * ev).sum(-1)
            e["dbeta"][t] = (e_du * ev.abs() + (du.abs() + e_du) * e_ev + STEP * kn * gm * (ev.abs() + e_ev)).sum(-1)
            de = b * du
            g["dv"][t], e["dv"][t] = de, b.abs() * e_du
            u, e_u = b * ev, b.abs() * e_ev
            g["dk"][t] = (A @ u[..., None])[..., 0] - (aS @ de[..., None])[..., 0]
            e["dk"][t] = (u.abs() * (ge + STEP * gm) + gm * e_u + de.abs() * (e_in + STEP * mag)
                          + b.abs() * e_du * mag).sum(-1, keepdim=True)
            An = A - kt[..., None] * de[:, None, :]
            gen = rho * ge + STEP * (gm + kn * b.abs() * kn * gm)
            g["dlog_decay"][t] = (An * aS).sum((-1, -2))
            e["dlog_decay"][t] = (gen * mag + gm * e_in).sum(-1)
            rows.append((STEP * (qn * d.abs() * m_S + kn * de.abs() * mag + kn * u.abs() * gm)).sum(-1))
            A, ge, gm = a[..., None] * An, a * gen, a * (gm + kn * b.abs() * kn * gm if bool((rho > 1).any()) else gm)
        if rows:
            c = torch.cat([z(1, H), torch.stack(rows[::-1]).cumsum(0)])
            L = len(rows)
            lo, hi = (torch.arange(L) - 64).clamp(min=0), (torch.arange(L) + 65).clamp(max=L)
            e["dlog_decay"][int(cu[n]):int(cu[n + 1])] += c[hi] - c[lo]
        g["dstates"][n] = A
        e["dstates"][n] = (ge + STEP * gm)[:, None, :]
    for n in ("dq", "dk"):
        g[n], e[n] = g[n].unflatten(1, (G_, rep)).sum(2), e[n].unflatten(1, (G_, rep)).sum(2)
    if not by_row:
        g["dlog_decay"], e["dlog_decay"] = g["dlog_decay"].sum(0), e["dlog_decay"].sum(0)
    return g, e


def gradient_bound(dtype, g, e):
    h = HALF[dtype]
    return h * (g.abs() + e) + e + 1e-30 + (2.0 ** -25 if dtype == torch.float16 else 0.0)
