"""Cases, inputs and plain forms of the linear-attention layer's operators.

The operators (float32 sums, states and statistics throughout):

* ``lin_prefill``: chunked linear attention with a decay for each head over a
  packed batch of sequences, S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T,
  y_t = S_t^T q_t, continued from and written back to a pool of states.
* ``lin_step``: one step of the same recurrence for each running sequence.
* ``gn_fwd`` / ``gn_bwd``: group norm, channels last, with an activation on
  the normalised value or on a gate that multiplies it.
* ``state_pack`` / ``state_unpack``: states of the pool written to a cache in
  8 bits (e4m3) with one power-of-two scale for 32 values, and read back.

``own`` selects between the elementary torch operations below and the
framework's calls.  ``exact`` is the operators' definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5

# Head layouts (groups of q and k, heads, dk, dv): the scan workloads of this
# repository, and generic ones (as many groups as heads, wide and odd heads).
HEADS = [(2, 8, 128, 128), (1, 24, 128, 64), (2, 4, 48, 40), (1, 1, 128, 128),
         (16, 16, 64, 64), (16, 16, 128, 128), (4, 8, 256, 128), (3, 6, 33, 97)]
MOST_TOKENS = 131072


def listed():
    def prefill(name, heads, dtype, seqs, tokens, per_token, fresh):
        G, H, dk, dv = heads
        return {"name": name, "op": "prefill", "dtype": dtype, "G": G, "H": H, "dk": dk, "dv": dv, "seqs": seqs,
                "tokens": tokens, "per_token": per_token, "fresh": fresh}

    def step(name, heads, dtype, seqs, slots, per_token):
        G, H, dk, dv = heads
        return {"name": name, "op": "step", "dtype": dtype, "G": G, "H": H, "dk": dk, "dv": dv, "seqs": seqs,
                "slots": slots, "per_token": per_token}

    def norm(name, op, dtype, N, L, C, groups, gate):
        return {"name": name, "op": op, "dtype": dtype, "N": N, "L": L, "C": C, "groups": groups, "gate": gate}

    def cache(name, op, slots, H, dk, dv, entries):
        return {"name": name, "op": op, "slots": slots, "H": H, "dk": dk, "dv": dv, "entries": entries}

    return [
        # one short prompt: latency
        prefill("prefill_short_prompt", (2, 8, 128, 128), "bf16", 1, 77, True, 1),
        # a server's ordinary batch: prompts of mixed lengths, half of them continued
        prefill("prefill_mixed_batch", (1, 24, 128, 64), "bf16", 20, 10007, True, 10),
        # one long document: few heads, so the work has to be split over its length
        prefill("prefill_long_prompt", (2, 8, 128, 128), "bf16", 1, 65536, False, 0),
        # odd head sizes in full precision
        prefill("prefill_odd_heads_fp32", (2, 4, 48, 40), "fp32", 6, 4099, True, 3),
        # the largest: a batch of long prompts, a q and k for every head
        prefill("prefill_large_batch", (16, 16, 128, 128), "bf16", 16, MOST_TOKENS, False, 16),
        # one user's next token: latency
        step("step_one_user", (2, 8, 128, 128), "bf16", 1, 4, False),
        # a full server's next tokens: every state is read and written
        step("step_full_batch", (1, 24, 128, 64), "bf16", 256, 300, True),
        # a gated layer's output, normalised for each head of each token, forward
        norm("gn_fwd_gated_tokens", "gn_fwd", "bf16", 16384, 1, 2048, 16, True),
        # the same layer's backward, 24 heads of 64, odd number of tokens
        norm("gn_bwd_gated_tokens", "gn_bwd", "bf16", 5001, 1, 1536, 24, True),
        # channels-last feature maps of a convolutional stem, ten channels to a group
        norm("gn_bwd_feature_maps", "gn_bwd", "fp16", 4, 4001, 320, 32, False),
        # states of finished prompts kept for reuse
        cache("state_pack_prompts", "state_pack", 96, 24, 128, 64, 64),
        # and handed to new requests, several of them from one entry
        cache("state_unpack_prompts", "state_unpack", 96, 24, 128, 64, 40),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over the logarithm of its range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "step", "step", "gn_fwd", "gn_bwd", "gn_bwd", "state_pack",
                     "state_unpack"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("prefill", "step"):
        G, H, dk, dv = rng.choice(HEADS)
        if rng.random() < 0.25:   # heads of any size
            dk, dv = _spread(rng, 1, 256), _spread(rng, 1, 256)
        c = {"op": op, "dtype": dtype, "G": G, "H": H, "dk": dk, "dv": dv, "per_token": rng.random() < 0.5}
        if op == "prefill":
            c["tokens"] = _spread(rng, 1, max(1, min(MOST_TOKENS, 2 ** 31 // (16 * H * max(dk, dv)))))
            c["seqs"] = _spread(rng, 1, min(64, c["tokens"]))
            c["fresh"] = rng.randint(0, c["seqs"])
        else:
            c["seqs"] = _spread(rng, 1, max(1, min(512, 2 ** 29 // (8 * H * dk * dv))))
            c["slots"] = c["seqs"] + rng.randint(0, 32)
        return c
    if op in ("gn_fwd", "gn_bwd"):
        groups = rng.choice([1, 4, 8, 16, 24, 32])
        C = groups * _spread(rng, 1, 128)
        most = 2 ** 25 // C
        L = 1 if rng.random() < 0.5 else _spread(rng, 2, min(16384, most))
        return {"op": op, "dtype": dtype, "N": _spread(rng, 1, max(1, most // L)), "L": L, "C": C, "groups": groups,
                "gate": rng.random() < 0.5}
    _, H, dk, dv = rng.choice(HEADS)
    entries = _spread(rng, 1, max(1, min(256, 2 ** 28 // (4 * H * dk * dv))))
    return {"op": op, "slots": entries + rng.randint(0, 16), "H": H, "dk": dk, "dv": dv, "entries": entries}


# ---- inputs


def _lengths(case, seed):
    """Lengths of a packed batch: `seqs` of them, one or more tokens each, `tokens` in all, mixed."""
    n, total = case["seqs"], case["tokens"]
    g = torch.Generator().manual_seed(seed)
    if n == 1:
        return [total]
    if total % n == 0 and case["fresh"] == n:   # a batch of equal prompts
        return [total // n] * n
    w = torch.rand(n, generator=g, dtype=torch.float64).mul_(2.0).exp_()
    ln = (w / w.sum() * (total - n)).floor().long() + 1
    ln[0] += total - int(ln.sum())
    return ln.tolist()


def _log_decay(case, rows, dev, g):
    """Either one decay for each head, from fast to slow, or one for each token and head."""
    if case["per_token"]:
        z = torch.randn(rows, case["H"], device=dev, generator=g)
        return -torch.nn.functional.softplus(z - 2.0)
    h = torch.arange(case["H"], device=dev, dtype=torch.float32)
    return torch.log1p(-torch.exp2(-3.0 - 6.0 * h / max(1, case["H"] - 1)))


def _qkv(case, rows, dev, g):
    """q, k and v as the slices of one projection's output."""
    G, H, dk, dv = (case[n] for n in ("G", "H", "dk", "dv"))
    p = torch.randn(rows, 2 * G * dk + H * dv, device=dev, generator=g)
    p[:, :2 * G * dk].mul_(dk ** -0.25)
    p = p.to(DTYPES[case["dtype"]])
    q, k, v = p.split([G * dk, G * dk, H * dv], dim=1)
    return q.unflatten(1, (G, dk)), k.unflatten(1, (G, dk)), v.unflatten(1, (H, dv))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op in ("prefill", "step"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        if op == "prefill":
            n = case["seqs"]
            ln = _lengths(case, seed)
            cu = torch.zeros(n + 1, dtype=torch.int64)
            cu[1:] = torch.tensor(ln).cumsum(0)
            s["cu"] = cu.to(torch.int32).to(dev)
            s["max_len"] = max(ln)
            s["carry"] = torch.ones(n, dtype=torch.int32)
            s["carry"][torch.randperm(n, generator=torch.Generator().manual_seed(seed + 1))[:case["fresh"]]] = 0
            s["carry"] = s["carry"].to(dev)
            rows, slots = case["tokens"], n
        else:
            rows, slots, n = case["seqs"], case["slots"], case["seqs"]
        s["q"], s["k"], s["v"] = _qkv(case, rows, dev, g)
        s["log_decay"] = _log_decay(case, rows, dev, g)
        s["states"] = torch.randn(slots, H, dk, dv, device=dev, generator=g)
        s["slots"] = torch.randperm(slots, device=dev, generator=g)[:n].to(torch.int32)
        return s
    if op in ("gn_fwd", "gn_bwd"):
        N, L, C = case["N"], case["L"], case["C"]
        dt = DTYPES[case["dtype"]]
        new = lambda *sh: torch.randn(*sh, device=dev, generator=g)   # noqa: E731
        s |= {"groups": case["groups"], "x": (new(N, L, C) * 1.5 + 0.5).to(dt), "weight": new(C) * 0.1 + 1.0, "bias": new(C) * 0.1,
              "gate": new(N, L, C).to(dt) if case["gate"] else None}
        if op == "gn_bwd":
            s["dy"] = new(N, L, C).to(dt)
            # what the forward hands to the backward: each group's mean and 1 / deviation
            x = s["x"].view(N, L, case["groups"], -1).double()
            var, mean = torch.var_mean(x, dim=(1, 3), correction=0)
            s["stats"] = torch.stack((mean, torch.rsqrt(var + EPS)), -1).float()
        return s
    H, dk, dv = case["H"], case["dk"], case["dv"]
    # rows of a state differ in size by powers of ten
    s["states"] = torch.randn(case["slots"], H, dk, dv, device=dev, generator=g) * torch.exp(
        2.0 * torch.randn(case["slots"], H, dk, 1, device=dev, generator=g))
    nb = -(-dv // 32)
    s["cache"] = torch.zeros(case["entries"], H, dk, dv, dtype=torch.float8_e4m3fn, device=dev)
    s["scales"] = torch.zeros(case["entries"], H, dk, nb, dtype=torch.uint8, device=dev)
    if op == "state_pack":
        s["slots"] = torch.randperm(case["slots"], device=dev, generator=g)[:case["entries"]].to(torch.int32)
        s["entries"] = torch.randperm(case["entries"], device=dev, generator=g).to(torch.int32)
    else:
        s["cache"].copy_((torch.randn(case["entries"], H, dk, dv, device=dev, generator=g) * 100).clamp_(-448, 448))
        s["scales"].copy_(torch.randint(100, 140, s["scales"].shape, device=dev, generator=g))
        s["slots"] = torch.randperm(case["slots"], device=dev, generator=g).to(torch.int32)
        s["entries"] = torch.randint(0, case["entries"], (case["slots"],), device=dev, generator=g).to(torch.int32)
    return s


# ---- one pass


def run(s):
    if own:
        return _run_own(s)
    return {"prefill": _prefill, "step": _step, "gn_fwd": _gn_fwd, "gn_bwd": _gn_bwd, "state_pack": _pack,
            "state_unpack": _unpack}[s["op"]](s)


def _run_own(s):
    import chunked_ssd_scan_fwd_amd as ssd
    op = s["op"]
    if op == "prefill":
        y = ssd.lin_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["cu"], s["states"], slots=s["slots"],
                            carry=s["carry"], max_seqlen=s["max_len"])
        return {"y": y, "states": s["states"]}
    if op == "step":
        y = ssd.lin_step(s["q"], s["k"], s["v"], s["log_decay"], s["states"], slots=s["slots"])
        return {"y": y, "states": s["states"]}
    if op == "gn_fwd":
        y, stats = ssd.gn_fwd(s["x"], s["weight"], s["bias"], s["groups"], gate=s["gate"], act="silu", eps=EPS)
        return {"y": y, "stats": stats}
    if op == "gn_bwd":
        dx, dw, db, dg = ssd.gn_bwd(s["x"], s["weight"], s["bias"], s["groups"], s["stats"], s["dy"], gate=s["gate"],
                                    act="silu")
        return {"dx": dx, "dweight": dw, "dbias": db, "dgate": dg}
    if op == "state_pack":
        ssd.state_pack(s["states"], s["cache"], s["scales"], slots=s["slots"], entries=s["entries"])
        return {"cache": s["cache"], "scales": s["scales"]}
    ssd.state_unpack(s["cache"], s["scales"], s["states"], entries=s["entries"], slots=s["slots"])
    return {"states": s["states"]}


def _prefill(s):
    """The chunked form: products inside chunks of 64, and a lower-triangular product over the chunks' states."""
    Ck = 64
    q, k, v, cu, states = s["q"], s["k"], s["v"], s["cu"].long(), s["states"]
    T, G, dk = q.shape
    H, dv = v.shape[1:]
    n, dev = cu.numel() - 1, q.device
    nc = -(-s["max_len"] // Ck)
    start, ln = cu[:-1], cu[1:] - cu[:-1]
    pos = torch.arange(nc * Ck, device=dev)
    live = pos < ln[:, None]                                             # [n, nc C]
    at = torch.where(live, start[:, None] + pos, 0)

    def tiles(x):                                                        # [T, h, d] -> [n, H, nc, C, d]
        x = torch.where(live[..., None, None], x.float()[at], 0.0)
        x = x.repeat_interleave(H // x.shape[2], dim=2) if x.shape[2] != H else x
        return x.unflatten(1, (nc, Ck)).permute(0, 3, 1, 2, 4).contiguous()

    q, k, v = tiles(q), tiles(k), tiles(v)
    la = s["log_decay"].double()
    la = la[at] if la.dim() == 2 else la.expand(n, nc * Ck, H)
    la = torch.where(live[..., None], la, 0.0).unflatten(1, (nc, Ck)).permute(0, 3, 1, 2)
    b = la.cumsum(-1)                                                    # [n, H, nc, C]
    tri = torch.ones(Ck, Ck, dtype=torch.bool, device=dev).tril()
    D = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(~tri, -math.inf)).float()
    y = ((q @ k.transpose(-1, -2)) * D) @ v
    X = (k * torch.exp(b[..., -1:] - b).float()[..., None]).transpose(-1, -2) @ v   # [n, H, nc, dk, dv]
    cb = b[..., -1].cumsum(-1)                                           # decay up to each chunk's end
    before = torch.cat((torch.zeros_like(cb[..., :1]), cb), -1)          # and up to each chunk's start, and the end
    low = torch.ones(nc + 1, nc, dtype=torch.bool, device=dev).tril(-1)
    M = torch.exp((before[..., :, None] - cb[..., None, :]).masked_fill(~low, -math.inf)).float()
    slots = s["slots"].long()
    S0 = states[slots] * s["carry"][:, None, None, None]
    S = (M @ X.flatten(-2)).unflatten(-1, (dk, dv)) + torch.exp(before).float()[..., None, None] * S0[:, :, None]
    y = y + (q * torch.exp(b).float()[..., None]) @ S[:, :, :-1]
    y = y.permute(0, 2, 3, 1, 4).flatten(0, 2)                           # [n nc C, H, dv]
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    y = y[seq * (nc * Ck) + t - cu[seq]].to(s["v"].dtype)
    states[slots] = S[:, :, -1]
    return {"y": y, "states": states}


def _step(s):
    q, k, v = (s[x].float() for x in "qkv")
    H = v.shape[1]
    q, k = (x.repeat_interleave(H // x.shape[1], dim=1) for x in (q, k))
    slots = s["slots"].long()
    a = torch.exp(s["log_decay"]).expand(q.shape[0], H)[..., None, None]
    S = a * s["states"][slots] + k[..., None] * v[..., None, :]
    y = (S * q[..., None]).sum(-2).to(s["v"].dtype)
    s["states"][slots] = S
    return {"y": y, "states": s["states"]}


def _gn_fwd(s):
    x, w, b, gate, groups = s["x"].float(), s["weight"], s["bias"], s["gate"], s["groups"]
    N, L, C = x.shape
    xg = x.view(N, L, groups, C // groups)
    mean = xg.mean((1, 3))
    xc = xg - mean[:, None, :, None]
    rstd = torch.rsqrt(xc.square().mean((1, 3)) + EPS)
    z = (xc * rstd[:, None, :, None]).view(N, L, C) * w + b
    u = z if gate is None else gate.float()
    u = u / (1 + torch.exp(-u))
    y = u if gate is None else z * u
    return {"y": y.to(s["x"].dtype), "stats": torch.stack((mean, rstd), -1)}


def _gn_bwd(s):
    x, w, b, gate, groups, dy = s["x"].float(), s["weight"], s["bias"], s["gate"], s["groups"], s["dy"].float()
    N, L, C = x.shape
    mean, rstd = s["stats"][:, None, :, None, 0], s["stats"][:, None, :, None, 1]
    xh = ((x.view(N, L, groups, -1) - mean) * rstd)
    z = xh.view(N, L, C) * w + b
    u = z if gate is None else gate.float()
    sg = 1 / (1 + torch.exp(-u))
    du = sg * (1 + u * (1 - sg))
    if gate is None:
        dz, dgate = dy * du, None
    else:
        dz, dgate = dy * (u * sg), (dy * z * du).to(s["x"].dtype)
    dxh = (dz * w).view_as(xh)
    m1, m2 = dxh.mean((1, 3), keepdim=True), (dxh * xh).mean((1, 3), keepdim=True)
    dx = rstd * (dxh - m1 - xh * m2)
    dw, db = (dz * xh.view(N, L, C)).sum((0, 1)), dz.sum((0, 1))
    return {"dx": dx.view(N, L, C).to(s["x"].dtype), "dweight": dw, "dbias": db, "dgate": dgate}


def _blocks(x):
    """The last axis in blocks of 32, the last one filled up with zeros."""
    n = x.shape[-1]
    return torch.nn.functional.pad(x, (0, -n % 32)).unflatten(-1, (-1, 32))


def _pack(s):
    """The smallest power of two under which a block's values stay within 448."""
    x = _blocks(s["states"][s["slots"].long()])
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, torch.where(m <= 0.875, e - 9, e - 8), -127).clamp(min=-127)
    half = torch.div(-e, 2, rounding_mode="floor")
    f = torch.exp2(half.float())[..., None] , torch.exp2((-e - half).float())[..., None]
    vals = (x * f[0] * f[1]).flatten(-2)[..., :s["states"].shape[-1]].to(torch.float8_e4m3fn)
    at = s["entries"].long()
    s["cache"].view(torch.uint8)[at] = vals.view(torch.uint8)
    s["scales"][at] = (e + 127).to(torch.uint8)
    return {"cache": s["cache"], "scales": s["scales"]}


def _unpack(s):
    at = s["entries"].long()
    x = s["cache"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    e = s["scales"][at].float() - 127
    half = torch.floor(e / 2)
    n = x.shape[-1]
    x = (_blocks(x) * torch.exp2(half)[..., None] * torch.exp2(e - half)[..., None]).flatten(-2)[..., :n]
    s["states"][s["slots"].long()] = x
    return {"states": s["states"]}


# ---- what a pass cannot do without


def work(case):
    op = case["op"]
    if op in ("prefill", "step"):
        G, H, dk, dv = (case[n] for n in ("G", "H", "dk", "dv"))
        rows, n = case["tokens"] if op == "prefill" else case["seqs"], case["seqs"]
        byt = rows * (2 * G * dk + 2 * H * dv) * SIZE[case["dtype"]] + (rows if case["per_token"] else 1) * H * 4
        reads = n - case["fresh"] if op == "prefill" else n
        return {"bytes": byt + (n + reads) * H * dk * dv * 4, "flops": 4 * rows * H * dk * dv}
    if op in ("gn_fwd", "gn_bwd"):
        elems = case["N"] * case["L"] * case["C"]
        tensors = 2 + case["gate"] if op == "gn_fwd" else 3 + 2 * case["gate"]
        return {"bytes": elems * tensors * SIZE[case["dtype"]] + 8 * case["N"] * case["groups"] + 8 * case["C"] * (1 if op == "gn_fwd" else 2),
                "flops": elems * (12 if op == "gn_fwd" else 30)}
    per = case["H"] * case["dk"] * (5 * case["dv"] + -(-case["dv"] // 32))
    return {"bytes": per * (case["entries"] if op == "state_pack" else case["slots"]),
            "flops": case["H"] * case["dk"] * case["dv"] * case["entries"]}


# ---- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prefill", "step"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        steps, n = (s["max_len"] if op == "prefill" else 1), case["seqs"]
        if steps * max(1e-4, n * H * dk * dv * 8 * 8 / 2e12) > 18:
            return None
        head = torch.arange(H, device="cuda") // (H // case["G"])
        slots = s["slots"].long()
        S = s["states"][slots].double()
        la = s["log_decay"].double()
        rows = case["tokens"] if op == "prefill" else n
        y = torch.zeros(rows, H, dv, dtype=torch.float64, device="cuda")
        if op == "prefill":
            S[s["carry"] == 0] = 0
            first = s["cu"][:-1].long()
            order = torch.argsort(s["cu"].diff(), descending=True)
            ln = sorted(s["cu"].diff().tolist(), reverse=True)
        else:
            first, order, ln = torch.arange(n, device="cuda"), torch.arange(n, device="cuda"), [1] * n
        S, first = S[order], first[order]
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        m = n
        for t in range(steps):
            while m and ln[m - 1] <= t:
                m -= 1
            at = first[:m] + t
            a = torch.exp(la[at] if la.dim() == 2 else la.expand(m, H))
            live = S[:m]
            live.mul_(a[..., None, None])
            live.addcmul_(k[at][:, head][..., None], v[at][..., None, :])
            y[at] = torch.matmul(q[at][:, head][..., None, :], live)[..., 0, :]
        states = s["states"].double()
        states[slots[order]] = S
        return {"y": y, "states": states}
    if op in ("gn_fwd", "gn_bwd"):
        N, L, C, groups = case["N"], case["L"], case["C"], case["groups"]
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        gate = s["gate"].double() if case["gate"] else None
        if op == "gn_bwd":
            x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
            if gate is not None:
                gate.requires_grad_()
        with torch.enable_grad():
            xg = x.transpose(1, 2).reshape(N, groups, -1)
            var, mean = torch.var_mean(xg, dim=-1, correction=0, keepdim=True)
            z = ((xg - mean) / (var + EPS).sqrt()).view(N, C, L).transpose(1, 2) * w + b
            y = z * torch.sigmoid(z) if gate is None else z * (gate * torch.sigmoid(gate))
            if op == "gn_fwd":
                return {"y": y, "stats": torch.cat((mean, (var + EPS).rsqrt()), -1)}
            ask = [x, w, b] + ([gate] if gate is not None else [])
            got = list(torch.autograd.grad(y, ask, s["dy"].double())) + [None]
        return {"dx": got[0], "dweight": got[1], "dbias": got[2], "dgate": got[3]}
    if op == "state_pack":
        return None   # roundings to 8 bits, which the scales fix
    states = s["states"].double()
    sc = torch.exp2(s["scales"].double() - 127).repeat_interleave(32, dim=-1)[..., :case["dv"]]
    states[s["slots"].long()] = (s["cache"].double() * sc)[s["entries"].long()]
    return {"states": states}
