"""Cases, inputs and plain forms of the gated delta rule and of beam search over
a pool of states.

The operators (float32 sums, states and statistics throughout):

* ``delta_prefill``: the gated delta rule over a packed batch of sequences,
  S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - a_t S_{t-1}^T k_t),
  y_t = S_t^T q_t,  a_t = exp(log_decay_t), continued from and written back to
  a pool of states.
* ``delta_step``: one step of the same recurrence for each running sequence.
* ``delta_bwd``: its gradients over a packed batch.
* ``beam_select``: the best continuations of a request's beams over beams and
  vocabulary.
* ``state_reorder``: the states of a request's beams after such a selection.

``own`` selects between the elementary torch operations below and the
framework's calls.  ``exact`` is the operators' definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
CHUNK = 64

# Head layouts (groups of q and k, heads, dk, dv): the scan workloads of this
# repository, and generic ones (as many groups as heads, wide and odd heads).
HEADS = [(2, 8, 128, 128), (1, 24, 128, 64), (2, 4, 48, 40), (1, 1, 128, 128),
         (16, 16, 64, 64), (16, 16, 128, 128), (4, 8, 256, 128), (3, 6, 33, 97)]
MOST_TOKENS = 131072
MOST_TRAINED = 32768


def listed():
    def scan(name, op, heads, dtype, seqs, tokens, per_token, **more):
        G, H, dk, dv = heads
        return {"name": name, "op": op, "dtype": dtype, "G": G, "H": H, "dk": dk, "dv": dv, "seqs": seqs,
                "tokens": tokens, "per_token": per_token, **more}

    def beams(name, dtype, requests, K, V, n):
        return {"name": name, "op": "beam", "dtype": dtype, "requests": requests, "beams": K, "vocabulary": V, "n": n}

    def reorder(name, requests, K, H, dk, dv):
        return {"name": name, "op": "reorder", "requests": requests, "beams": K, "H": H, "dk": dk, "dv": dv}

    return [
        # one short prompt: latency
        scan("delta_prefill_short_prompt", "prefill", (2, 8, 128, 128), "bf16", 1, 77, True, fresh=1),
        # a server's ordinary batch: prompts of mixed lengths, half of them continued
        scan("delta_prefill_mixed_batch", "prefill", (1, 24, 128, 64), "bf16", 20, 10007, True, fresh=10),
        # one long document: few heads, so the work has to be split over its length
        scan("delta_prefill_long_prompt", "prefill", (2, 8, 128, 128), "bf16", 1, 32768, True, fresh=1),
        # the largest: a batch of long prompts, a q and k for every head
        scan("delta_prefill_large_batch", "prefill", (16, 16, 128, 128), "bf16", 16, MOST_TOKENS, True, fresh=16),
        # one user's next token: latency
        scan("delta_step_one_user", "step", (2, 8, 128, 128), "bf16", 1, 1, False, slots=4),
        # a full server's next tokens: every state is read and written
        scan("delta_step_full_batch", "step", (16, 16, 128, 128), "bf16", 256, 256, True, slots=300),
        # a training step's batch of equal rows
        scan("delta_bwd_training", "bwd", (16, 16, 128, 128), "bf16", 4, 8192, True, entered=False),
        # documents of mixed lengths in one batch, odd heads in full precision, from states and with their gradients
        scan("delta_bwd_documents_fp32", "bwd", (2, 4, 48, 40), "fp32", 9, 4099, False, entered=True),
        # one request's four beams: latency
        beams("beam_select_one_request", "fp32", 1, 4, 32001, 8),
        # a server's requests over a large vocabulary
        beams("beam_select_full_batch", "bf16", 64, 4, 131072, 8),
        # one request's beams change places
        reorder("state_reorder_one_request", 1, 4, 8, 128, 128),
        # a server's
        reorder("state_reorder_full_batch", 64, 4, 16, 128, 128),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over the logarithm of its range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "step", "step", "bwd", "bwd", "bwd", "beam", "beam", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "beam":
        K, V = rng.choice([1, 2, 3, 4, 5, 8, 16]), _spread(rng, 100, 262144)
        most = max(1, min(256, 2 ** 25 // (K * V)))
        return {"op": op, "dtype": dtype, "requests": _spread(rng, 1, most), "beams": K, "vocabulary": V,
                "n": rng.choice([K, K, 2 * K, min(64, 4 * K)])}
    G, H, dk, dv = rng.choice(HEADS)
    if op == "reorder":
        K = rng.choice([2, 3, 4, 5, 8, 16])
        return {"op": op, "requests": _spread(rng, 1, max(1, min(128, 2 ** 28 // (4 * K * H * dk * dv)))), "beams": K,
                "H": H, "dk": dk, "dv": dv}
    if rng.random() < 0.25:   # heads of any size
        dk, dv = _spread(rng, 1, 256), _spread(rng, 1, 256)
    c = {"op": op, "dtype": dtype, "G": G, "H": H, "dk": dk, "dv": dv, "per_token": rng.random() < 0.5}
    if op == "step":
        c["seqs"] = c["tokens"] = _spread(rng, 1, max(1, min(512, 2 ** 29 // (8 * H * dk * dv))))
        c["slots"] = c["seqs"] + rng.randint(0, 32)
        return c
    if op == "prefill":
        most = min(MOST_TOKENS, 2 ** 31 // (16 * H * max(dk, dv)))
    else:   # and the states of its chunks fit
        most = min(MOST_TRAINED, 2 ** 24 // (H * max(dk, dv)), 2 ** 31 // (H * dk * dv))
    c["tokens"] = _spread(rng, 1, max(64, most))
    c["seqs"] = _spread(rng, 1, min(64, c["tokens"]))
    if op == "prefill":
        c["fresh"] = rng.randint(0, c["seqs"])
    else:
        c["entered"] = rng.random() < 0.5
    return c


# ---- inputs


def _lengths(case, seed):
    """Lengths of a packed batch: `seqs` of them, one or more tokens each, `tokens` in all, mixed."""
    n, total = case["seqs"], case["tokens"]
    if n == 1:
        return [total]
    if total % n == 0 and case.get("fresh", n) == n:   # a batch of equal rows
        return [total // n] * n
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(n, generator=g, dtype=torch.float64).mul_(2.0).exp_()
    ln = (w / w.sum() * (total - n)).floor().long() + 1
    ln[0] += total - int(ln.sum())
    return ln.tolist()


def _qkv(case, rows, dev, g):
    """q, k and v as the slices of one projection's output, with q and k of length 1 (q scaled)."""
    G, H, dk, dv = (case[n] for n in ("G", "H", "dk", "dv"))
    p = torch.randn(rows, 2 * G * dk + H * dv, device=dev, generator=g)
    qk = p[:, :2 * G * dk].unflatten(1, (2 * G, dk))
    qk.div_(qk.square().sum(-1, keepdim=True).sqrt_().add_(1e-6))
    p[:, :G * dk].mul_(dk ** -0.5)
    p = p.to(DTYPES[case["dtype"]])
    q, k, v = p.split([G * dk, G * dk, H * dv], dim=1)
    return q.unflatten(1, (G, dk)), k.unflatten(1, (G, dk)), v.unflatten(1, (H, dv))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    new = lambda *sh: torch.randn(*sh, device=dev, generator=g)   # noqa: E731
    if op in ("prefill", "step", "bwd"):
        H, dk, dv, n, rows = (case[x] for x in ("H", "dk", "dv", "seqs", "tokens"))
        if op != "step":
            ln = _lengths(case, seed)
            cu = torch.zeros(n + 1, dtype=torch.int64)
            cu[1:] = torch.tensor(ln).cumsum(0)
            s["cu"] = cu.to(torch.int32).to(dev)
            s["max_len"] = max(ln)
        s["q"], s["k"], s["v"] = _qkv(case, rows, dev, g)
        if case["per_token"]:
            s["log_decay"] = -torch.nn.functional.softplus(new(rows, H) - 4.0)
        else:   # one for each head, from fast to slow
            h = torch.arange(H, device=dev, dtype=torch.float32)
            s["log_decay"] = torch.log1p(-torch.exp2(-3.0 - 6.0 * h / max(1, H - 1)))
        s["beta"] = torch.sigmoid(new(rows, H))
        if op == "bwd":
            s["dy"] = new(rows, H, dv).to(DTYPES[case["dtype"]])
            s["states"] = new(n, H, dk, dv) * 0.3 if case["entered"] else None
            s["dstates"] = new(n, H, dk, dv) * 0.3 if case["entered"] else None
            return s
        if op == "prefill":
            s["carry"] = torch.ones(n, dtype=torch.int32)
            s["carry"][torch.randperm(n, generator=torch.Generator().manual_seed(seed + 1))[:case["fresh"]]] = 0
            s["carry"] = s["carry"].to(dev)
        slots = case.get("slots", n)
        s["states"] = new(slots, H, dk, dv) * 0.3
        s["slots"] = torch.randperm(slots, device=dev, generator=g)[:n].to(torch.int32)
        return s
    R, K = case["requests"], case["beams"]
    if op == "beam":
        s["n"], s["end"] = case["n"], 2
        s["logits"] = (new(R, K, case["vocabulary"]) * 2.5).to(DTYPES[case["dtype"]])
        s["scores"] = -10.0 * torch.rand(R, K, device=dev, generator=g)
        s["ended"] = torch.rand(R, K, device=dev, generator=g) < 0.1
        return s
    s["states"] = new(R * K + 8, case["H"], case["dk"], case["dv"])
    s["slots"] = torch.randperm(R * K + 8, device=dev, generator=g)[:R * K].to(torch.int32)
    s["parents"] = torch.randint(0, K, (R, K), device=dev, generator=g).to(torch.int32)
    return s


# ---- one pass


def run(s):
    if own:
        return _run_own(s)
    return {"prefill": _prefill, "step": _step, "bwd": _bwd, "beam": _beam, "reorder": _reorder}[s["op"]](s)


def _run_own(s):
    import chunked_ssd_scan_fwd_amd as ssd
    op = s["op"]
    if op == "prefill":
        y = ssd.delta_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["cu"], s["states"], slots=s["slots"],
                              carry=s["carry"], max_seqlen=s["max_len"])
        return {"y": y, "states": s["states"]}
    if op == "step":
        y = ssd.delta_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["states"], slots=s["slots"])
        return {"y": y, "states": s["states"]}
    if op == "bwd":
        got = ssd.delta_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["cu"], s["dy"], states=s["states"],
                            dstates=s["dstates"], max_seqlen=s["max_len"])
        return dict(zip(("dq", "dk", "dv", "dlog_decay", "dbeta", "dstates"), got))
    if op == "beam":
        scores, tokens, parents = ssd.beam_select(s["logits"], s["scores"], s["n"], ended=s["ended"],
                                                  end_token=s["end"])
        return {"scores": scores, "tokens": tokens, "parents": parents}
    ssd.state_reorder(s["states"], s["parents"], slots=s["slots"])
    return {"states": s["states"]}


def _inverse(A):
    """(I + A)^-1 of strictly lower matrices [..., C, C], C a power of two, joined from halves: stable as a
    substitution is."""
    C = A.shape[-1]
    T = torch.ones_like(A[..., :, :1]).unsqueeze(-1)                      # [..., C, 1, 1]
    while T.shape[-1] < C:
        h = T.shape[-1]
        n = C // (2 * h)
        low = A.unflatten(-2, (n, 2 * h)).unflatten(-1, (n, 2 * h)).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        low = low[..., h:, :h].contiguous()
        T1, T2 = T[..., 0::2, :, :].contiguous(), T[..., 1::2, :, :].contiguous()
        X = -(T2 @ (low @ T1))
        T = torch.cat((torch.cat((T1, torch.zeros_like(T1)), -1), torch.cat((X, T2), -1)), -2)
    return T[..., 0, :, :].contiguous()


class _Chunks:
    """A packed batch as chunks [n, H, nc, C, .] of its sequences, filled up with rows that change nothing."""

    def __init__(self, s):
        cu = s["cu"].long()
        self.T, self.G, self.dk = s["q"].shape
        self.H, self.dv = s["v"].shape[1:]
        self.n, dev = cu.numel() - 1, cu.device
        self.nc = -(-s["max_len"] // CHUNK)
        start, ln = cu[:-1], cu[1:] - cu[:-1]
        pos = torch.arange(self.nc * CHUNK, device=dev)
        self.live = pos < ln[:, None]                                     # [n, nc C]
        self.at = torch.where(self.live, start[:, None] + pos, 0)
        t = torch.arange(self.T, device=dev)
        seq = torch.searchsorted(cu, t, right=True) - 1
        self.back = seq * (self.nc * CHUNK) + t - cu[seq]
        self.q, self.k, self.v = self.tiles(s["q"]), self.tiles(s["k"]), self.tiles(s["v"])
        self.beta = self.tiles(s["beta"][..., None])                      # [n, H, nc, C, 1]
        la = s["log_decay"]
        la = la if la.dim() == 2 else la.expand(self.T, self.H)
        b = self.tiles(la[..., None], torch.float64)[..., 0].cumsum(-1)   # [n, H, nc, C]
        tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
        D = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(~tri, -math.inf)).float()
        self.enter = torch.exp(b).float()[..., None]                      # e^{b_t}
        self.leave = torch.exp(b[..., -1:] - b).float()[..., None]        # e^{b_L - b_t}
        self.all = torch.exp(b[..., -1]).float()[..., None, None]         # e^{b_L}
        kt = self.k.transpose(-1, -2).contiguous()
        self.P = (self.q @ kt) * D
        self.M = (self.k @ kt) * (D - torch.eye(CHUNK, device=dev))       # below the diagonal
        self.D = D
        self.inv = _inverse(self.beta * self.M)

    def tiles(self, x, dtype=torch.float32):                              # [T, h, d] -> [n, H, nc, C, d]
        x = torch.where(self.live[..., None, None], x.to(dtype)[self.at], 0.0)
        x = x.repeat_interleave(self.H // x.shape[2], dim=2) if x.shape[2] != self.H else x
        return x.unflatten(1, (self.nc, CHUNK)).permute(0, 3, 1, 2, 4).contiguous()

    def rows(self, x):                                                    # [n, H, nc, C, d] -> [T, H, d]
        return x.permute(0, 2, 3, 1, 4).flatten(0, 2)[self.back]

    def walk(self, S, visit):
        """The states that enter the chunks, one chunk after the other, each with what its rows write; the last state."""
        W, U0 = self.inv @ (self.beta * self.enter * self.k), self.inv @ (self.beta * self.v)
        kt = (self.k * self.leave).transpose(-1, -2).contiguous()
        for c in range(self.nc):
            U = U0[:, :, c] - W[:, :, c] @ S
            visit(c, S, U)
            S = self.all[:, :, c] * S + kt[:, :, c] @ U
        return S


def _prefill(s):
    x = _Chunks(s)
    qe = x.q * x.enter
    y = torch.empty_like(x.v)

    def visit(c, S, U):
        y[:, :, c] = qe[:, :, c] @ S + x.P[:, :, c] @ U

    slots = s["slots"].long()
    S0 = s["states"][slots] * s["carry"][:, None, None, None]
    s["states"][slots] = x.walk(S0, visit)
    return {"y": x.rows(y).to(s["v"].dtype), "states": s["states"]}


def _step(s):
    q, k, v = (s[x].float() for x in "qkv")
    H = v.shape[1]
    q, k = (x.repeat_interleave(H // x.shape[1], dim=1) for x in (q, k))
    slots = s["slots"].long()
    S = torch.exp(s["log_decay"]).expand(q.shape[0], H)[..., None, None] * s["states"][slots]
    u = s["beta"][..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    y = (S * q[..., None]).sum(-2).to(s["v"].dtype)
    s["states"][slots] = S
    return {"y": y, "states": s["states"]}


def _bwd(s):
    """The chunks again with the states that enter them, the adjoints from the last chunk to the first, and the
    products inside all chunks at once."""
    x = _Chunks(s)
    S = torch.empty(x.n, x.H, x.nc, x.dk, x.dv, device=x.q.device)
    U = torch.empty_like(x.v)

    def visit(c, S_c, U_c):
        S[:, :, c], U[:, :, c] = S_c, U_c

    x.walk(torch.zeros_like(S[:, :, 0]) if s["states"] is None else s["states"], visit)
    dy = x.tiles(s["dy"])
    tr = lambda a: a.transpose(-1, -2).contiguous()   # noqa: E731
    dU0 = tr(x.P) @ dy
    dS = torch.empty_like(S)                                              # of the states that leave the chunks
    dG = torch.empty_like(U)
    A = torch.zeros_like(S[:, :, 0]) if s["dstates"] is None else s["dstates"]
    qt, kt, kl, it = tr(x.q * x.enter), tr(x.k * x.enter), x.k * x.leave, tr(x.inv)
    for c in reversed(range(x.nc)):
        dS[:, :, c] = A
        dG[:, :, c] = it[:, :, c] @ (dU0[:, :, c] + kl[:, :, c] @ A)
        A = x.all[:, :, c] * A + qt[:, :, c] @ dy[:, :, c] - kt[:, :, c] @ (x.beta[:, :, c] * dG[:, :, c])
    dR = x.beta * dG
    St, Ut = tr(S), tr(U)
    dyS, dRS, UdS = x.enter * (dy @ St), x.enter * (dR @ St), x.leave * (U @ tr(dS))
    dP = (dy @ Ut) * x.D                                                  # of q k^T, on and below the diagonal
    dM = -(dR @ Ut) * (x.D - torch.eye(CHUNK, device=x.q.device))         # of k k^T, below it
    dq = dyS + dP @ x.k
    dk = UdS - dRS + tr(dP) @ x.q + (dM + tr(dM)) @ x.k
    Z = x.v - x.enter * (x.k @ S) - x.M @ U                               # U / beta
    dbeta = (dG * Z).sum(-1, keepdim=True)
    # the decays: of what leaves, by the rows before; of what enters, by the rows from there on; of pairs across
    N = ((dP * (x.q @ tr(x.k))) + (dM * (x.k @ tr(x.k)))).double()
    f = ((dyS * x.q).sum(-1) - (dRS * x.k).sum(-1)).double()
    e = (UdS * x.k).sum(-1).double()
    pairs = N.sum(-2) - N.sum(-1)                                         # by column less by row
    before = (e + pairs).cumsum(-1) - (e + pairs)
    dla = f.flip(-1).cumsum(-1).flip(-1) + before + (x.all[..., 0, 0] * (S * dS).sum((-1, -2))).double()[..., None]
    # a group's heads share its q and k
    share = lambda a: x.rows(a).unflatten(1, (x.G, -1)).sum(2).to(s["q"].dtype)   # noqa: E731
    dla = x.rows(dla[..., None])[..., 0]
    dla = (dla if s["log_decay"].dim() == 2 else dla.sum(0)).float()
    return {"dq": share(dq), "dk": share(dk), "dv": x.rows(dR).to(s["v"].dtype), "dlog_decay": dla,
            "dbeta": x.rows(dbeta)[..., 0], "dstates": None if s["states"] is None else A}


def _beam(s):
    """In 64 bits: candidates next to each other are closer than float32 tells apart."""
    x, n = s["logits"].double(), s["n"]
    R, K, V = x.shape
    m = x.amax(-1, keepdim=True)
    lse = m + (x - m).exp().sum(-1, keepdim=True).log()
    c = s["scores"].double()[..., None] + (x - lse)
    ended = s["ended"][..., None]
    end = torch.arange(V, device=x.device) == s["end"]
    c = torch.where(ended, torch.where(end, s["scores"].double()[..., None], -math.inf), c).flatten(1)
    n_ = min(n, K * V)
    last = c.topk(n_).values[:, -1:]
    # those above the last of the best, and as many of its equals as there is room for, by their index
    at = torch.arange(K * V, device=x.device, dtype=torch.int32)
    far = torch.full_like(at, 2 ** 31 - 1)
    above = torch.where(c > last, at, far).topk(n_, largest=False, sorted=True).values
    equal = torch.where(c == last, at, far).topk(n_, largest=False, sorted=True).values
    both = torch.cat((above, equal), 1).sort(-1).values                   # by index, then by value
    val = torch.where(both == far[0], -math.inf, c.gather(1, both.long().clamp(max=K * V - 1)))
    val, order = val.sort(dim=-1, descending=True, stable=True)
    at = both.gather(1, order)[:, :n].long()
    val = val[:, :n]
    val, at = (torch.nn.functional.pad(a, (0, n - a.shape[1]), value=w) for a, w in ((val, -math.inf), (at, 0)))
    none = val == -math.inf
    return {"scores": val.float(), "tokens": torch.where(none, -1, at % V).int(),
            "parents": torch.where(none, -1, at // V).int()}


def _reorder(s):
    K = s["parents"].shape[1]
    slots = s["slots"].long()
    of = (torch.arange(s["parents"].shape[0], device=slots.device)[:, None] * K + s["parents"]).flatten()
    s["states"][slots] = s["states"][slots[of]]
    return {"states": s["states"]}


# ---- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "beam":
        elems = case["requests"] * case["beams"] * case["vocabulary"]
        return {"bytes": elems * SIZE[case["dtype"]] + 12 * case["requests"] * case["n"], "flops": 4 * elems}
    if op == "reorder":
        K = case["beams"]
        moved = K - 1                                       # of K beams with parents drawn evenly
        read = K * (1 - (1 - 1 / K ** 2) ** moved) if K < 3 else K * (1 - (1 - 1 / K) ** moved)
        state = 4 * case["H"] * case["dk"] * case["dv"]
        return {"bytes": case["requests"] * state * (moved + read), "flops": 0}
    G, H, dk, dv = (case[n] for n in ("G", "H", "dk", "dv"))
    rows, n, e = case["tokens"], case["seqs"], SIZE[case["dtype"]]
    state, decays = n * H * dk * dv * 4, (rows if case["per_token"] else 1) * H * 4
    if op == "bwd":
        byt = rows * (4 * G * dk + 3 * H * dv) * e + 2 * decays + 2 * rows * H * 4
        return {"bytes": byt + (3 * state if case["entered"] else 0), "flops": 16 * rows * H * dk * dv}
    byt = rows * (2 * G * dk + 2 * H * dv) * e + decays + rows * H * 4
    reads = (n - case["fresh"]) / n if op == "prefill" else 1
    return {"bytes": byt + state * (1 + reads), "flops": 6 * rows * H * dk * dv}


# ---- the definitions, in 64 bits


def _padded(case, s):
    """The batch as [n, longest, ...] in 64 bits, filled up with rows that change nothing."""
    rows, n, H, rep = case["tokens"], case["seqs"], case["H"], case["H"] // case["G"]
    cu = s["cu"].long() if "cu" in s else torch.arange(n + 1, device="cuda")
    ln = cu.diff()
    L = int(ln.max())
    t = torch.arange(rows, device="cuda")
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), ln)
    place = seq * L + t - cu[seq]

    def fill(x):
        out = torch.zeros(n * L, *x.shape[1:], dtype=torch.float64, device="cuda")
        out[place] = x.double()
        return out.unflatten(0, (n, L))

    la = s["log_decay"]
    la = la if la.dim() == 2 else la.expand(rows, H)
    q, k = (fill(s[x].repeat_interleave(rep, 1)) for x in "qk")
    return L, place, q, k, fill(s["v"]), fill(la).exp(), fill(s["beta"]), fill


def exact(case, seed):
    op = case["op"]
    if op in ("prefill", "step", "bwd"):
        H, dk, dv, n = (case[x] for x in ("H", "dk", "dv", "seqs"))
        steps = 1 if op == "step" else max(_lengths(case, seed))
        one = n * H * dk * dv * 8
        if steps * (max(1.5e-4, one * 12 / 2e12) if op != "bwd" else max(6e-4, one * 40 / 2e12)) > 18:
            return None
        if n * steps * H * (2 * dk + 4 * dv) * 8 > 5e10 or (op == "bwd" and one * (64 + steps / 64) > 6e10):
            return None
    s = prepare(case, seed)
    if op in ("prefill", "step"):
        L, place, q, k, v, a, beta, _ = _padded(case, s)
        slots = s["slots"].long()
        S = s["states"][slots].double()
        if op == "prefill":
            S[s["carry"] == 0] = 0
        y = torch.zeros(n, L, H, dv, dtype=torch.float64, device="cuda")
        for t in range(L):
            S.mul_(a[:, t, :, None, None])
            u = v[:, t] - torch.matmul(k[:, t, :, None, :], S)[..., 0, :]
            S.addcmul_(k[:, t][..., None], (u * beta[:, t][..., None])[..., None, :])
            y[:, t] = torch.matmul(q[:, t, :, None, :], S)[..., 0, :]
        states = s["states"].double()
        states[slots] = S
        return {"y": y.flatten(0, 1)[place], "states": states}
    if op == "bwd":
        return _exact_bwd(case, s)
    if op == "beam":
        x, n = s["logits"].double(), s["n"]
        R, K, V = x.shape
        c = s["scores"].double()[..., None] + torch.log_softmax(x, -1)
        for r, k in s["ended"].nonzero().tolist():
            c[r, k] = -math.inf
            c[r, k, s["end"]] = s["scores"][r, k].double()
        val, at = c.flatten(1).sort(dim=-1, descending=True, stable=True)
        val = torch.nn.functional.pad(val[:, :n], (0, max(0, n - K * V)), value=-math.inf)
        return {"scores": val, "tokens": None, "parents": None}
    K = case["beams"]
    states, slots, parents = s["states"].double(), s["slots"].tolist(), s["parents"].tolist()
    old = states.clone()
    for r, of in enumerate(parents):
        for j, p in enumerate(of):
            states[slots[r * K + j]] = old[slots[r * K + p]]
    return {"states": states}


def _exact_bwd(case, s):
    """Row by row, forward and then back, the states recomputed from every 64th."""
    H, dk, dv, n = (case[x] for x in ("H", "dk", "dv", "seqs"))
    L, place, q, k, v, a, beta, fill = _padded(case, s)
    # rows past a sequence's end keep the state: their decay is exp(0)
    dy = fill(s["dy"])
    zero = torch.zeros(n, H, dk, dv, dtype=torch.float64, device="cuda")

    def step(S, t):
        S = S * a[:, t, :, None, None]
        e = v[:, t] - torch.matmul(k[:, t, :, None, :], S)[..., 0, :]
        return S, e, S + k[:, t][..., None] * (beta[:, t][..., None] * e)[..., None, :]

    S = zero if s["states"] is None else s["states"].double()
    kept = []
    for t in range(L):
        if t % 64 == 0:
            kept.append(S)
        S = step(S, t)[2]
    G = zero.clone() if s["dstates"] is None else s["dstates"].double().clone()
    dq, dkey, dval, dla, dbeta = (torch.zeros_like(x) for x in (q, k, v, a, beta))
    for t0 in reversed(range(0, L, 64)):
        S, run_ = kept.pop(), []
        for t in range(t0, min(L, t0 + 64)):
            run_.append(step(S, t))
            S = run_[-1][2]
        for t in reversed(range(t0, min(L, t0 + 64))):
            aS, e, S = run_.pop()
            G.addcmul_(q[:, t][..., None], dy[:, t][..., None, :])
            dq[:, t] = torch.matmul(S, dy[:, t][..., None])[..., 0]
            du = torch.matmul(k[:, t][..., None, :], G)[..., 0, :]
            b = beta[:, t][..., None]
            dbeta[:, t] = (du * e).sum(-1)
            de = b * du
            dval[:, t] = de
            dkey[:, t] = torch.matmul(G, (b * e)[..., None])[..., 0] - torch.matmul(aS, de[..., None])[..., 0]
            G = G - k[:, t][..., None] * de[..., None, :]                 # of a S
            dla[:, t] = (G * aS).sum((-1, -2))
            G = G * a[:, t, :, None, None]
    pick = lambda x: x.flatten(0, 1)[place]   # noqa: E731
    share = lambda x: pick(x).unflatten(1, (case["G"], -1)).sum(2)   # noqa: E731
    dla = pick(dla)
    return {"dq": share(dq), "dk": share(dkey), "dv": pick(dval), "dlog_decay": dla if case["per_token"] else dla.sum(0),
            "dbeta": pick(dbeta), "dstates": None if s["states"] is None else G}
