"""Operators of a linear-attention layer: Python binding of the lin_, gn_ and
state_ calls of ``ssd.h``.

Like the rest of the binding it only marshals arguments: every step runs in
the library's HIP kernels, on PyTorch's current stream of the inputs' device,
and there is no fallback.  Nothing here waits for the device, so every call
can be captured into a graph (pass ``workspace`` and outputs that outlive it,
or let the graph's own memory pool hold them).

Element types of q, k, v, y, x, gate, dy: float32, bfloat16 or float16, the
same for all of a call.  States, log decays, weights, statistics: float32.
Index arrays: int32, on the device.
"""
from __future__ import annotations

import ctypes

__all__ = ["lin_prefill", "lin_step", "gn_fwd", "gn_bwd", "state_pack", "state_unpack", "lin_prefill_workspace_size",
           "gn_workspace_size", "STATE_CACHE_BLOCK"]

STATE_CACHE_BLOCK = 32   # values of a state's row that share a scale byte
_i64, _vp, _sz, _int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_torch = None
_library = None   # the package's library()
_stream_of = _current = None
_dtypes = {}
_ACTS = {None: 0, "none": 0, "silu": 1}


class LinShapeArg(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("T", "N", "G", "H", "dk", "dv", "slots")]


class LinStridesArg(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("q_t", "q_g", "k_t", "k_g", "v_t", "v_h", "y_t", "y_h")]


class GnShapeArg(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("N", "L", "C", "groups")]


class StateCacheShapeArg(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("n", "slots", "entries", "H", "dk", "dv")]


def declare(lib):
    """The argument types of the layer's calls."""
    lp, tp, gp, cp = (ctypes.POINTER(c) for c in (LinShapeArg, LinStridesArg, GnShapeArg, StateCacheShapeArg))
    lib.lin_prefill_workspace_size.argtypes = [lp, _i64]
    lib.lin_prefill_workspace_size.restype = _sz
    lib.lin_prefill.argtypes = [lp, _int, tp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _vp]
    lib.lin_step.argtypes = [lp, _int, tp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp]
    for fn in (lib.gn_fwd_workspace_size, lib.gn_bwd_workspace_size):
        fn.argtypes = [gp]
        fn.restype = _sz
    lib.gn_fwd.argtypes = [gp, _int, _int, ctypes.c_float, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _vp]
    lib.gn_bwd.argtypes = [gp, _int, _int, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _sz,
                           _vp]
    lib.state_pack.argtypes = [cp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.state_unpack.argtypes = [cp, _vp, _vp, _vp, _vp, _vp, _vp]
    for fn in (lib.lin_prefill, lib.lin_step, lib.gn_fwd, lib.gn_bwd, lib.state_pack, lib.state_unpack):
        fn.restype = _int


def _init():
    global _torch, _stream_of, _current
    import torch
    _dtypes.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    # a call's own time counts where the work takes microseconds: the raw
    # stream and device, without the objects around them
    _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    _current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch


def _lib():
    if _torch is None:
        _init()
    return _library()


_args = {}


def _arg(cls, *fields):
    """A reference to a struct of these fields; those of recent calls are kept."""
    key = (cls, fields)
    r = _args.get(key)
    if r is None:
        if len(_args) >= 1024:
            _args.clear()
        r = _args[key] = ctypes.byref(cls(*fields))
    return r


def _dtype_of(t, name):
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _dtypes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    return code


def _is(t, name, shape, dtype, device):
    """`t` is a tensor of this shape (a tuple) and type, on HIP device `device` (its number)."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype == dtype and t.shape == shape and t.get_device() == device:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on HIP device {device}, got {t.device}")


def _dense(t, name, shape, dtype, device):
    _is(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _rows(t, name):
    """Strides of a [rows, heads, d] tensor whose last axis is dense."""
    a, b, c = t.stride()
    n, h, d = t.shape
    if c != 1 and d > 1:
        raise ValueError(f"the last axis of {name} must be dense")
    return (a if n > 1 else 0), (b if h > 1 else 0)


def _ids(t, name, n, device):
    """An index array's pointer (None for none)."""
    return None if t is None else _dense(t, name, (n,), _torch.int32, device)


def _call(fn, where, device, *args):
    """fn(*args, stream) with device number `device` current, on its current stream."""
    if device != _current():
        with _torch.cuda.device(device):
            rc = fn(*args, _stream_of(device))
    else:
        rc = fn(*args, _stream_of(device))
    if rc != 0:
        from . import SsdError
        raise SsdError(rc, where)


def _bytes(need, device, workspace):
    """Pointer and size of the caller's workspace, or of a new one."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _torch.empty(need, dtype=_torch.uint8, device=device)
        return workspace.data_ptr(), need, workspace
    from . import _workspace_bytes
    workspace, _ = _workspace_bytes(need, _torch.device("cuda", device), workspace)
    return workspace.data_ptr() or None, workspace.numel() * workspace.element_size(), workspace


def _lin_args(q, k, v, log_decay, states, out, rows_name):
    code = _dtype_of(q, "q")
    dev, dt = q.get_device(), q.dtype
    for t, name, dims in ((v, "v", 3), (states, "states", 4), (log_decay, "log_decay", 0)):
        if not isinstance(t, _torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if dims and t.dim() != dims or q.dim() != 3:
            raise ValueError(f"q must be [{rows_name},G,dk], v [{rows_name},H,dv] and states [slots,H,dk,dv]")
    R, G, dk = q.shape
    _, H, dv = v.shape
    _is(k, "k", (R, G, dk), dt, dev)
    _is(v, "v", (R, H, dv), dt, dev)
    S = states.shape[0]
    sp = _dense(states, "states", (S, H, dk, dv), _torch.float32, dev)
    ld = 0
    if log_decay.dim() == 1:
        _is(log_decay, "log_decay", (H,), _torch.float32, dev)
    else:
        _is(log_decay, "log_decay", (R, H), _torch.float32, dev)
        if R > 1:   # 0: the same decays for every row
            ld = log_decay.stride(0)
    if H > 1 and log_decay.stride(-1) != 1:
        raise ValueError("the last axis of log_decay must be dense")
    if out is None:
        out = v.new_empty((R, H, dv))
        st = (H * dv, dv)
    else:
        _is(out, "out", (R, H, dv), dt, dev)
        st = _rows(out, "out")
    st = _arg(LinStridesArg, *_rows(q, "q"), *_rows(k, "k"), *_rows(v, "v"), *st)
    return code, dev, (R, G, H, dk, dv, S), sp, ld, log_decay.data_ptr() or None, out, st


def lin_prefill_workspace_size(T, N, G, H, dk, dv, slots, max_seqlen=0) -> int:
    """Workspace bytes of `lin_prefill` for T rows, N sequences and a pool of `slots` states."""
    n = _lib().lin_prefill_workspace_size(ctypes.byref(LinShapeArg(T, N, G, H, dk, dv, slots)), max_seqlen)
    if n == _sz(-1).value:
        raise ValueError(f"unsupported or invalid shape {(T, N, G, H, dk, dv, slots)}")
    return int(n)


def lin_prefill(q, k, v, log_decay, cu_seqlens, states, *, slots=None, carry=None, max_seqlen=0, out=None,
                workspace=None):
    """y[T,H,dv] of the scan over a packed batch: q, k [T,G,dk], v [T,H,dv]
    (their last axis dense), log_decay float32 [H] or [T,H], cu_seqlens int32
    [N+1].  Sequence n continues the state in states[slots[n]] (float32
    [slots,H,dk,dv]; slots None: n) where carry[n] is not 0 (None: always),
    and leaves its last state there.  max_seqlen: an upper bound of the
    lengths, which lets short batches run in one pass.  Rows of no sequence
    are left as they are in ``out``.  See lin_prefill in ssd.h for what
    becomes of negative, missing and repeated slots."""
    lib = _lib()
    code, dev, (T, G, H, dk, dv, S), sp, ld, lp, out, st = _lin_args(q, k, v, log_decay, states, out, "T")
    if not isinstance(cu_seqlens, _torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be a tensor of N+1 offsets")
    N = cu_seqlens.shape[0] - 1
    cu = _dense(cu_seqlens, "cu_seqlens", (N + 1,), _torch.int32, dev)
    max_seqlen = int(max_seqlen or 0)
    if max_seqlen < 0:
        raise ValueError("max_seqlen must not be negative")
    s = _arg(LinShapeArg, T, N, G, H, dk, dv, S)
    need = lib.lin_prefill_workspace_size(s, max_seqlen)
    if need == _sz(-1).value:
        raise ValueError(f"unsupported or invalid shape: T {T}, N {N}, G {G}, H {H}, dk {dk}, dv {dv}")
    wp, wn, _keep = _bytes(need, dev, workspace)
    _call(lib.lin_prefill, "lin_prefill", dev, s, code, st, q.data_ptr() or None,
          k.data_ptr() or None, v.data_ptr() or None, lp, ld, cu, _ids(slots, "slots", N, dev),
          _ids(carry, "carry", N, dev), max_seqlen, sp, out.data_ptr() or None, wp, wn)
    return out


def lin_step(q, k, v, log_decay, states, *, slots=None, out=None):
    """y[N,H,dv] of one step for each row: q, k [N,G,dk], v [N,H,dv],
    log_decay float32 [H] or [N,H]; row n updates states[slots[n]] (slots
    None: n) in place.  Rows of one slot take effect in their order; rows of
    a negative slot are skipped and leave ``out`` as it is."""
    lib = _lib()
    code, dev, (N, G, H, dk, dv, S), sp, ld, lp, out, st = _lin_args(q, k, v, log_decay, states, out, "N")
    s = _arg(LinShapeArg, 0, N, G, H, dk, dv, S)
    _call(lib.lin_step, "lin_step", dev, s, code, st, q.data_ptr() or None,
          k.data_ptr() or None, v.data_ptr() or None, lp, ld, _ids(slots, "slots", N, dev), sp,
          out.data_ptr() or None)
    return out


def _gn_rows(t, name, shape, dtype, device):
    """Pointer and row stride (0: dense) of x, gate or dy, [N,L,C] or [N,C]."""
    _is(t, name, shape, dtype, device)
    if t.is_contiguous():
        return t.data_ptr() or None, 0
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last axis of {name} must be dense")
    if len(shape) == 2:
        ld = t.stride(0) if shape[0] > 1 else 0
    elif shape[1] > 1:
        ld = t.stride(1)
        if shape[0] > 1 and t.stride(0) != shape[1] * ld:
            raise ValueError(f"the rows of {name} must be evenly spaced over samples")
    else:
        ld = t.stride(0) if shape[0] > 1 else 0
    if ld == 0 and t.numel() > shape[-1]:
        raise ValueError(f"{name} must not repeat one row")
    return t.data_ptr() or None, ld


def _gn_args(x, weight, bias, groups, gate):
    code = _dtype_of(x, "x")
    if x.dim() not in (2, 3):
        raise ValueError("x must be [N,L,C], or [N,C] for L = 1")
    C = x.shape[-1]
    N, L = x.shape[0], (x.shape[1] if x.dim() == 3 else 1)
    groups = int(groups)
    if groups < 1 or C < 1 or C % groups:
        raise ValueError(f"{C} channels cannot be cut into {groups} groups")
    dev, shape = x.get_device(), tuple(x.shape)
    xp, ldx = _gn_rows(x, "x", shape, x.dtype, dev)
    wp = None if weight is None else _dense(weight, "weight", (C,), _torch.float32, dev)
    bp = None if bias is None else _dense(bias, "bias", (C,), _torch.float32, dev)
    gp, ldg = (None, 0) if gate is None else _gn_rows(gate, "gate", shape, x.dtype, dev)
    return code, dev, shape, (N, L, C, groups), xp, ldx, wp, bp, gp, ldg


def _act(act):
    if act not in _ACTS:
        raise ValueError(f"act must be 'silu' or 'none', got {act!r}")
    return _ACTS[act]


def gn_workspace_size(N, L, C, groups, backward: bool = False) -> int:
    """Workspace bytes of `gn_fwd` or `gn_bwd`."""
    lib = _lib()
    n = (lib.gn_bwd_workspace_size if backward else lib.gn_fwd_workspace_size)(
        ctypes.byref(GnShapeArg(N, L, C, groups)))
    if n == _sz(-1).value:
        raise ValueError(f"invalid shape {(N, L, C, groups)}")
    return int(n)


def gn_fwd(x, weight, bias, groups, *, gate=None, act="silu", eps=1e-5, out=None, stats=None, workspace=None):
    """(y, stats): group norm of x [N,L,C] (or [N,C], L = 1), channels last,
    over the L rows and C / groups channels of each group, times weight plus
    bias (float32 [C] or None).  y = act(z), or z act(gate) with a gate of x's
    shape; act is "silu" or "none".  stats float32 [N,groups,2] holds mean and
    1 / deviation for `gn_bwd`."""
    lib = _lib()
    code, dev, shape, s, xp, ldx, wp, bp, gp, ldg = _gn_args(x, weight, bias, groups, gate)
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    act = _act(act)
    st_shape = (s[0], s[3], 2)
    if out is None:
        out = x.new_empty(shape)
        op = out.data_ptr() or None
    else:
        op = _dense(out, "out", shape, x.dtype, dev)
    if stats is None:
        stats = x.new_empty(st_shape, dtype=_torch.float32)
        stp = stats.data_ptr() or None
    else:
        stp = _dense(stats, "stats", st_shape, _torch.float32, dev)
    ref = _arg(GnShapeArg, *s)
    wsp, wsn, _keep = _bytes(lib.gn_fwd_workspace_size(ref), dev, workspace)
    _call(lib.gn_fwd, "gn_fwd", dev, ref, code, act, eps, xp, ldx, wp, bp, gp, ldg, op, stp, wsp, wsn)
    return out, stats


def gn_bwd(x, weight, bias, groups, stats, dy, *, gate=None, act="silu", out=None, workspace=None):
    """(dx, dweight, dbias, dgate): the gradients of sum(dy * y) for `gn_fwd`
    of the same arguments, which returned `stats`; dgate is None without a
    gate.  ``out``: the four (or, without a gate, three) tensors to write."""
    lib = _lib()
    code, dev, shape, s, xp, ldx, wp, bp, gp, ldg = _gn_args(x, weight, bias, groups, gate)
    act = _act(act)
    dyp, ldy = _gn_rows(dy, "dy", shape, x.dtype, dev)
    stp = _dense(stats, "stats", (s[0], s[3], 2), _torch.float32, dev)
    C = s[2]
    if out is None:
        dx = x.new_empty(shape)
        dg = None if gate is None else x.new_empty(shape)
        dw, db = x.new_empty((2, C), dtype=_torch.float32).unbind()
        dxp, dwp, dgp = dx.data_ptr() or None, dw.data_ptr(), None if dg is None else dg.data_ptr() or None
        dbp = dwp + 4 * C
    else:
        dx, dw, db, dg = tuple(out) if gate is not None else (*tuple(out)[:3], None)
        dxp = _dense(dx, "dx", shape, x.dtype, dev)
        dwp, dbp = _dense(dw, "dweight", (C,), _torch.float32, dev), _dense(db, "dbias", (C,), _torch.float32, dev)
        dgp = None if dg is None else _dense(dg, "dgate", shape, x.dtype, dev)
    ref = _arg(GnShapeArg, *s)
    wsp, wsn, _keep = _bytes(lib.gn_bwd_workspace_size(ref), dev, workspace)
    _call(lib.gn_bwd, "gn_bwd", dev, ref, code, act, xp, ldx, wp, bp, gp, ldg, stp, dyp, ldy, dxp, dwp, dbp, dgp, wsp, wsn)
    return dx, dw, db, dg


def _cache_args(states, cache, scales, slots, entries):
    if not isinstance(states, _torch.Tensor) or states.dim() != 4 or not states.is_cuda:
        raise ValueError("states must be a [slots,H,dk,dv] tensor on a HIP device")
    dev = states.get_device()
    S, H, dk, dv = states.shape
    sp = _dense(states, "states", (S, H, dk, dv), _torch.float32, dev)
    if not isinstance(cache, _torch.Tensor) or cache.dim() != 4:
        raise ValueError("cache must be an [entries,H,dk,dv] tensor")
    E = cache.shape[0]
    cp = _dense(cache, "cache", (E, H, dk, dv), _torch.float8_e4m3fn, dev)
    ep = _dense(scales, "scales", (E, H, dk, -(-dv // STATE_CACHE_BLOCK)), _torch.uint8, dev)
    for t, name in ((slots, "slots"), (entries, "entries")):
        if t is not None and not isinstance(t, _torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t is not None and t.dim() != 1:
            raise ValueError(f"{name} must be a tensor of indexes, one for each pair")
    n = slots.shape[0] if slots is not None else entries.shape[0] if entries is not None else min(S, E)
    if (slots is None and n > S) or (entries is None and n > E):
        raise ValueError(f"{n} pairs, {S} slots and {E} entries")
    return (dev, _arg(StateCacheShapeArg, n, S, E, H, dk, dv), sp, cp, ep, _ids(slots, "slots", n, dev),
            _ids(entries, "entries", n, dev))


def state_pack(states, cache, scales, *, slots=None, entries=None):
    """Writes states[slots[i]] (float32 [slots,H,dk,dv]) to the cache's entry
    entries[i] in 8 bits: cache float8_e4m3fn [entries,H,dk,dv] and scales
    uint8 [entries,H,dk,ceil(dv/32)], a power of two for each 32 values of a
    row.  Without an index array, 0, 1, 2, ...  Pairs with a negative index
    are skipped; of pairs with one entry the last counts."""
    lib = _lib()
    dev, s, sp, cp, ep, ids, ide = _cache_args(states, cache, scales, slots, entries)
    _call(lib.state_pack, "state_pack", dev, s, sp, ids, ide, cp, ep)


def state_unpack(cache, scales, states, *, entries=None, slots=None):
    """Writes the cache's entry entries[i], as `state_pack` left it, to
    states[slots[i]].  One entry may go to several slots.  Index arrays as for
    `state_pack`; an entry that does not exist gives NaN."""
    lib = _lib()
    dev, s, sp, cp, ep, ids, ide = _cache_args(states, cache, scales, slots, entries)
    _call(lib.state_unpack, "state_unpack", dev, s, cp, ep, ide, ids, sp)
