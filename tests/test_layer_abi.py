"""CPU checks of the linear-attention layer's calls: every one is exported
and refuses bad arguments on the host, before anything touches a device; and
the tests' own references against second formulations."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import chunked_ssd_scan_fwd_amd as ssd
from chunked_ssd_scan_fwd_amd.layer import GnShapeArg, LinShapeArg, LinStridesArg, StateCacheShapeArg
import layer_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = range(6)
P = 0x10000   # a pointer that is never followed


def test_every_declared_call_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ssd.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:lin|gn|state)_[a-z_0-9]+)\s*\(", text))
    assert {"lin_prefill", "lin_step", "gn_fwd", "gn_bwd", "state_pack", "state_unpack"} <= names
    for n in names:
        assert hasattr(ssd.library(), n), n


def lin(shape, step=False, dtype=1, strides=None, ptr=P, ld=0, max_len=0, ws=(None, 0), **other):
    lib = ssd.library()
    p = dict(q=ptr, k=ptr, v=ptr, la=ptr, cu=ptr, slots=ptr, carry=ptr, states=ptr, y=ptr) | other
    st = ctypes.byref(strides) if strides is not None else None
    if step:
        return lib.lin_step(ctypes.byref(shape), dtype, st, p["q"], p["k"], p["v"], p["la"], ld, p["slots"],
                            p["states"], p["y"], None)
    return lib.lin_prefill(ctypes.byref(shape), dtype, st, p["q"], p["k"], p["v"], p["la"], ld, p["cu"], p["slots"],
                           p["carry"], max_len, p["states"], p["y"], *ws, None)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("shape,code", [
    ((5, 2, 3, 4, 8, 8, 4), SHAPE),              # H % G
    ((5, 2, 0, 4, 8, 8, 4), SHAPE),
    ((5, -1, 1, 4, 8, 8, 4), SHAPE),
    ((5, 2, 1, 4, 0, 8, 4), SHAPE),
    ((5, 2, 1, 4, 8, 8, -1), SHAPE),
    ((5, 2, 1, 4, 257, 8, 4), UNSUPPORTED),
    ((5, 2, 1, 4, 8, 300, 4), UNSUPPORTED),
    ((5, 1 << 24, 1, 4, 8, 8, 4), SHAPE),
    ((5, 2, 1, 1 << 16, 8, 8, 4), SHAPE),
    ((5, (1 << 24) - 1, 1, 4096, 8, 8, 4), SHAPE),   # more blocks than a grid holds
    ((5, 1 << 23, 1, 1, 8, 8, 4), SHAPE),
    ((5, 1 << 21, 1, 1, 8, 97, 4), SHAPE),
])
def test_lin_shapes_refused(step, shape, code):
    assert lin(LinShapeArg(*shape), step) == code


def test_lin_arguments_refused():
    s = LinShapeArg(5, 2, 1, 4, 8, 8, 4)
    big = 1 << 24
    assert lin(LinShapeArg(-1, 2, 1, 4, 8, 8, 4)) == SHAPE
    assert lin(LinShapeArg(1 << 30, 2, 1, 4, 8, 8, 4)) == SHAPE
    assert lin(s, max_len=-1) == SHAPE
    for step in (False, True):
        assert lin(s, step, dtype=3) == UNSUPPORTED and lin(s, step, dtype=-1) == UNSUPPORTED
        assert lin(s, step, ld=-1) == SHAPE and lin(s, step, ld=big) == SHAPE
        assert lin(s, step, strides=LinStridesArg(8, 8, 8, 8, big, 8, 32, 8)) == SHAPE
        assert lin(s, step, strides=LinStridesArg(8, -8, 8, 8, 32, 8, 32, 8)) == SHAPE
        assert lin(s, step, strides=LinStridesArg(8, 8, 8, 8, 32, 8, 31, 8)) == SHAPE   # rows of y overlap
        assert lin(s, step, strides=LinStridesArg(8, 8, 8, 8, 32, 8, 0, 8)) == SHAPE
        assert lin(s, step, strides=LinStridesArg(8, 8, 8, 8, 32, 8, 32, 7)) == SHAPE   # heads of y overlap
        for name in ("q", "k", "v", "la", "states", "y") + (() if step else ("cu",)):
            assert lin(s, step, **{name: None}) == NULL, name
            assert lin(s, step, **{name: P + 1}) == ALIGN, name
        for name in ("slots",) + (() if step else ("carry",)):
            assert lin(s, step, **{name: P + 2}) == ALIGN, name
        assert lin(LinShapeArg(5, 5, 1, 4, 8, 8, 4), step, slots=None) == SHAPE   # sequence 4 has no slot
        assert lin(LinShapeArg(0, 0, 1, 4, 8, 8, 0), step, ptr=None) == OK        # nothing to do
    assert lib_null() == NULL
    assert ssd.library().lin_prefill_workspace_size(ctypes.byref(s), -1) == ctypes.c_size_t(-1).value
    with pytest.raises(ValueError):
        ssd.layer.lin_prefill_workspace_size(5, 2, 3, 4, 8, 8, 4)


def lib_null():
    lib = ssd.library()
    a = lib.lin_prefill(None, 0, None, *[None] * 4, 0, None, None, None, 0, None, None, None, 0, None)
    b = lib.lin_step(None, 0, None, *[None] * 4, 0, None, None, None, None)
    assert a == b
    return a


def test_prefill_workspace_is_checked():
    s = LinShapeArg(1 << 17, 1, 1, 1, 128, 128, 1)
    need = ssd.layer.lin_prefill_workspace_size(1 << 17, 1, 1, 1, 128, 128, 1)
    if need:
        assert lin(s, ws=(P, need - 1)) == WORKSPACE
        assert lin(s, ws=(None, need)) == NULL
        assert lin(s, ws=(P + 8, need)) == ALIGN
    assert ssd.layer.lin_prefill_workspace_size(1 << 17, 1, 1, 1, 128, 128, 1, 40) == 0


def gn(shape, bwd=False, dtype=1, act=1, eps=1e-5, ptr=P, ws=(P, 1 << 40), ld=(0, 0, 0), **other):
    p = dict(x=ptr, w=ptr, b=ptr, gate=ptr, y=ptr, stats=ptr, dy=ptr, dx=ptr, dw=ptr, db=ptr, dgate=ptr) | other
    lib = ssd.library()
    if bwd:
        return lib.gn_bwd(ctypes.byref(shape), dtype, act, p["x"], ld[0], p["w"], p["b"], p["gate"], ld[1], p["stats"],
                          p["dy"], ld[2], p["dx"], p["dw"], p["db"], p["dgate"], *ws, None)
    return lib.gn_fwd(ctypes.byref(shape), dtype, act, eps, p["x"], ld[0], p["w"], p["b"], p["gate"], ld[1], p["y"],
                      p["stats"], *ws, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_gn_arguments_refused(bwd):
    s = GnShapeArg(3, 4, 12, 3)
    for bad in ((3, 4, 12, 5), (3, 4, 12, 0), (-1, 4, 12, 3), (3, -1, 12, 3), (3, 4, 0, 3), (3, 4, 1 << 24, 1),
                (3, 1 << 30, 12, 3), (1 << 40, 1 << 20, 12, 3)):
        assert gn(GnShapeArg(*bad), bwd) == SHAPE, bad
    assert gn(s, bwd, dtype=7) == UNSUPPORTED and gn(s, bwd, act=2) == UNSUPPORTED
    assert gn(s, bwd, ld=(-1, 0, 0)) == SHAPE and gn(s, bwd, ld=(0, 1 << 24, 0)) == SHAPE
    for name in ("x", "stats") + (("dy",) if bwd else ("y",)):
        assert gn(s, bwd, **{name: None}) == NULL, name
    for name in ("x", "stats", "w", "b", "gate") + (("dy", "dx", "dgate", "dw", "db") if bwd else ("y",)):
        assert gn(s, bwd, **{name: P + 1}) == ALIGN, name
    if bwd:
        need = ssd.layer.gn_workspace_size(3, 4, 12, 3, True)
        assert need > 0 and gn(s, True, ws=(P, need - 1)) == WORKSPACE
        assert gn(s, True, ws=(None, need)) == NULL and gn(s, True, ws=(P + 4, need)) == ALIGN
        assert gn(s, True, gate=None) == NULL   # a gradient of a gate that is not there
    else:
        assert gn(s, eps=-1.0) == SHAPE and gn(s, eps=float("nan")) == SHAPE
        assert gn(GnShapeArg(0, 4, 12, 3), ptr=None) == OK
    lib = ssd.library()
    assert lib.gn_fwd(None, 0, 0, 0.0, None, 0, None, None, None, 0, None, None, None, 0, None) == NULL
    assert lib.gn_bwd(None, 0, 0, None, 0, None, None, None, 0, None, None, 0, *[None] * 5, 0, None) == NULL
    with pytest.raises(ValueError):
        ssd.layer.gn_workspace_size(3, 4, 12, 5)


def cache(shape, unpack=False, **other):
    p = dict(states=P, cache=P, scales=P, slots=P, entries=P) | other
    lib = ssd.library()
    if unpack:
        return lib.state_unpack(ctypes.byref(shape), p["cache"], p["scales"], p["entries"], p["slots"], p["states"], None)
    return lib.state_pack(ctypes.byref(shape), p["states"], p["slots"], p["entries"], p["cache"], p["scales"], None)


@pytest.mark.parametrize("unpack", [False, True])
def test_cache_arguments_refused(unpack):
    s = StateCacheShapeArg(2, 3, 4, 1, 8, 8)
    for bad, code in (((-1, 3, 4, 1, 8, 8), SHAPE), ((2, -3, 4, 1, 8, 8), SHAPE), ((2, 3, 4, 0, 8, 8), SHAPE),
                      ((2, 3, 4, 1, 0, 8), SHAPE), ((2, 3, 4, 1, 257, 8), UNSUPPORTED),
                      ((2, 3, 4, 1, 8, 257), UNSUPPORTED), ((1 << 24, 3, 4, 1, 8, 8), SHAPE),
                      (((1 << 24) - 1, 3, 4, 4096, 256, 256), SHAPE)):
        assert cache(StateCacheShapeArg(*bad), unpack) == code, bad
    for name in ("states", "cache", "scales"):
        assert cache(s, unpack, **{name: None}) == NULL
    for name in ("states", "slots", "entries"):
        assert cache(s, unpack, **{name: P + 2}) == ALIGN
    assert cache(StateCacheShapeArg(4, 3, 4, 1, 8, 8), unpack, slots=None) == SHAPE
    assert cache(StateCacheShapeArg(4, 4, 3, 1, 8, 8), unpack, entries=None) == SHAPE
    assert cache(StateCacheShapeArg(0, 3, 4, 1, 8, 8), unpack, states=None, cache=None, scales=None) == OK
    lib = ssd.library()
    assert (lib.state_unpack if unpack else lib.state_pack)(None, *[None] * 6) == NULL


def test_binding_refuses_host_tensors_and_wrong_types():
    q, k, v, la, S = layer_ref.inputs(4, 1, 2, 8, 8, torch.float32, False, 0, 2)
    with pytest.raises(ValueError):
        ssd.lin_step(q, k, v, la, S)
    with pytest.raises(TypeError):
        ssd.lin_step(q.double(), k, v, la, S)
    with pytest.raises(ValueError):
        ssd.lin_prefill(q, k, v, la, torch.tensor([0, 4], dtype=torch.int32), S)
    with pytest.raises(ValueError):
        ssd.gn_fwd(torch.zeros(3, 8), None, None, 2)
    with pytest.raises(TypeError):
        ssd.gn_fwd(None, None, None, 2)
    with pytest.raises(ValueError):
        ssd.state_pack(S, torch.zeros(2, 2, 8, 8, dtype=torch.float8_e4m3fn), torch.zeros(2, 2, 8, 1, dtype=torch.uint8))


# ---- the references themselves


def test_scan_reference_against_the_quadratic_form():
    q, k, v, la, S = layer_ref.inputs(9, 1, 2, 3, 4, torch.float32, True, 5, 2)
    y, out, y_abs, _ = layer_ref.scan(q, k, v, la, [0, 0, 9], S, carry=[1, 1])
    for h in range(2):
        B = la.double()[:, h].cumsum(0)
        for t in range(9):
            want = sum(torch.exp(B[t] - B[j]) * (q[t, 0].double() @ k[j, 0].double()) * v[j, h].double()
                       for j in range(t + 1)) + torch.exp(B[t]) * (q[t, 0].double() @ S[1, h].double())
            assert torch.allclose(y[t, h], want, rtol=1e-12)
    assert torch.equal(out[0], S[0].double()) and bool((y_abs >= y.abs()).all())


def test_group_norm_reference_against_torch():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 5, 12, generator=g, dtype=torch.float64)
    w, b = torch.randn(12, generator=g, dtype=torch.float64), torch.randn(12, generator=g, dtype=torch.float64)
    y = layer_ref.group_norm(x, w, b, 4, None, "none", 1e-5)
    want = torch.nn.functional.group_norm(x.transpose(1, 2), 4, w, b, 1e-5).transpose(1, 2)
    assert torch.allclose(y, want, rtol=1e-11, atol=1e-12)


def test_cache_reference_against_the_format():
    g = np.random.default_rng(3)
    x = (g.standard_normal((2, 3, 40)) * np.exp(3 * g.standard_normal((2, 3, 40)))).astype(np.float32)
    x[0, 0] = 0
    x[0, 1, 0], x[0, 1, 1:32] = 448.0, 1.0
    x[0, 2, :32] = np.float32(1e-40)
    code, sc = layer_ref.pack(x)
    back = layer_ref.unpack(code, sc)
    s = np.repeat(2.0 ** (sc.astype(float) - 127), 32, axis=-1)[..., :40]
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)).all()
    assert sc[0, 0, 0] == 0 and sc[0, 1, 0] == 127 and (code[0, 0] == 0).all()
    t8 = torch.from_numpy(code.copy()).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(t8 * s, back)
    again = torch.from_numpy((x / s).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(again, code)
