"""CPU checks of the gated delta rule's calls: exported, refusing bad arguments
on the host, and the tests' own references against second formulations."""
import ctypes
import os
import re

import pytest
import torch

import chunked_ssd_scan_fwd_amd as ssd
from chunked_ssd_scan_fwd_amd.layer import LinShapeArg, LinStridesArg
import delta_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = range(6)
P, BIG = 0x10000, (0x10000, 1 << 60)   # a pointer that is never followed


def test_every_declared_call_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ssd.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(delta_[a-z_0-9]+)\s*\(", text))
    assert {"delta_prefill", "delta_step", "delta_bwd"} <= names
    for n in names:
        assert hasattr(ssd.library(), n), n


def call(shape, which, dtype=1, strides=None, ptr=P, ld=0, lb=8, max_len=0, ws=BIG, by_row=1, **other):
    lib = ssd.library()
    names = ("q", "k", "v", "la", "beta", "cu", "slots", "carry", "states", "y", "dy", "dlast", "dq", "dk", "dv", "dla",
             "dbeta", "d0")
    p = dict.fromkeys(names, ptr) | other
    st = ctypes.byref(strides) if strides is not None else None
    s = ctypes.byref(shape)
    if which == "step":
        return lib.delta_step(s, dtype, st, p["q"], p["k"], p["v"], p["la"], ld, p["beta"], lb, p["slots"], p["states"],
                              p["y"], None)
    if which == "prefill":
        return lib.delta_prefill(s, dtype, st, p["q"], p["k"], p["v"], p["la"], ld, p["beta"], lb, p["cu"], p["slots"],
                                 p["carry"], max_len, p["states"], p["y"], *ws, None)
    return lib.delta_bwd(s, dtype, st, p["q"], p["k"], p["v"], p["la"], ld, p["beta"], lb, p["cu"], p["states"], p["dy"],
                         p["dlast"], p["dq"], p["dk"], p["dv"], p["dla"], by_row, p["dbeta"], p["d0"], 0, *ws, None)


@pytest.mark.parametrize("which", ["prefill", "step", "bwd"])
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
])
def test_shapes_refused(which, shape, code):
    assert call(LinShapeArg(*shape), which) == code


@pytest.mark.parametrize("dk,rows", [(256, 32), (8, 64)])
def test_bwd_refuses_more_chunks_than_a_grid_holds(dk, rows):
    size = ssd.layer.delta_bwd_workspace_size
    most = (1 << 23) - 1   # chunks, one of them for the sequence's remainder
    assert size((most - 1) * rows, 1, 1, 1, dk, 1) > 0
    with pytest.raises(ValueError):
        size(most * rows, 1, 1, 1, dk, 1)
    assert call(LinShapeArg(most * rows, 1, 1, 1, dk, 1, 1), "bwd") == SHAPE


@pytest.mark.parametrize("which", ["prefill", "step", "bwd"])
def test_arguments_refused(which):
    s = LinShapeArg(5, 2, 1, 4, 8, 8, 4)
    big = 1 << 24
    assert call(s, which, dtype=3) == UNSUPPORTED and call(s, which, dtype=-1) == UNSUPPORTED
    assert call(s, which, ld=-1) == SHAPE and call(s, which, ld=big) == SHAPE
    assert call(s, which, lb=-1) == SHAPE and call(s, which, lb=big) == SHAPE
    assert call(s, which, strides=LinStridesArg(8, 8, 8, 8, big, 8, 32, 8)) == SHAPE
    assert call(s, which, strides=LinStridesArg(8, -8, 8, 8, 32, 8, 32, 8)) == SHAPE
    if which != "bwd":
        assert call(s, which, strides=LinStridesArg(8, 8, 8, 8, 32, 8, 31, 8)) == SHAPE   # rows of y overlap
        assert call(LinShapeArg(5, 5, 1, 4, 8, 8, 4), which, slots=None) == SHAPE   # sequence 4 has no slot
        assert call(LinShapeArg(0, 0, 1, 4, 8, 8, 0), which, ptr=None) == OK        # nothing to do
    need = {"prefill": ("q", "k", "v", "la", "beta", "cu", "states", "y"), "step": ("q", "k", "v", "la", "beta", "states", "y"),
            "bwd": ("q", "k", "v", "la", "beta", "cu", "dy", "dq", "dk", "dv", "dla", "dbeta")}[which]
    for name in need:
        assert call(s, which, **{name: None}) == NULL, name
    may = {"prefill": ("slots", "carry"), "step": ("slots",), "bwd": ("states", "dlast", "d0")}[which]
    for name in need + may:
        assert call(s, which, **{name: P + 1}) == ALIGN, name
    if which != "step":
        assert call(LinShapeArg(-1, 2, 1, 4, 8, 8, 4), which) == SHAPE
        assert call(LinShapeArg(1 << 30, 2, 1, 4, 8, 8, 4), which) == SHAPE
        assert call(LinShapeArg((1 << 30) - 1, 2, 1, 1, 8, 8, 4), which) == SHAPE   # more chunks than a grid holds
        n = (ssd.layer.delta_prefill_workspace_size(5, 2, 1, 4, 8, 8, 4) if which == "prefill" else
             ssd.layer.delta_bwd_workspace_size(5, 2, 1, 4, 8, 8))
        if which == "bwd" or n > 0:
            assert n > 0 and call(s, which, ws=(P, n - 1)) == WORKSPACE
            assert call(s, which, ws=(None, n)) == NULL and call(s, which, ws=(P + 8, n)) == ALIGN
    if which == "prefill":
        assert call(s, which, max_len=-1) == SHAPE
    if which == "bwd":
        assert call(LinShapeArg(0, 0, 1, 4, 8, 8, 0), which, ptr=None) == OK
        assert call(LinShapeArg(0, 0, 1, 4, 8, 8, 0), which, ptr=None, by_row=0) == NULL   # dlog_decay [H] is written


def test_null_shapes_and_sizes():
    lib = ssd.library()
    assert lib.delta_prefill(None, 0, None, *[None] * 4, 0, None, 0, *[None] * 3, 0, *[None] * 3, 0, None) == NULL
    assert lib.delta_step(None, 0, None, *[None] * 4, 0, None, 0, *[None] * 4) == NULL
    assert lib.delta_bwd(None, 0, None, *[None] * 4, 0, None, 0, *[None] * 8, 0, None, None, 0, None, 0, None) == NULL
    with pytest.raises(ValueError):
        ssd.layer.delta_prefill_workspace_size(5, 2, 3, 4, 8, 8, 4)
    with pytest.raises(ValueError):
        ssd.layer.delta_bwd_workspace_size(5, 2, 3, 4, 8, 8)
    assert lib.delta_prefill_workspace_size(ctypes.byref(LinShapeArg(5, 2, 1, 4, 8, 8, 4)), -1) == ctypes.c_size_t(-1).value


def test_binding_refuses_host_tensors_and_wrong_types():
    q, k, v, la, beta, S = ref.inputs(4, 1, 2, 8, 8, torch.float32, False, 0, 2)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        ssd.delta_step(q, k, v, la, beta, S)
    with pytest.raises(TypeError):
        ssd.delta_step(q.double(), k, v, la, beta, S)
    with pytest.raises(ValueError):
        ssd.delta_prefill(q, k, v, la, beta, cu, S)
    with pytest.raises(ValueError):
        ssd.delta_bwd(q, k, v, la, beta, cu, v)
    with pytest.raises(TypeError):
        ssd.delta_bwd(None, k, v, la, beta, cu, v)


# ---- the references themselves


def small(seed=0, rows=9, G=1, H=2, dk=3, dv=4):
    q, k, v, la, beta, S = (t.double() for t in ref.inputs(rows, G, H, dk, dv, torch.float32, True, seed, 2, mu=-1.0))
    g = torch.Generator().manual_seed(seed + 1)
    return q, k, v, la, beta, S, torch.randn(rows, H, dv, generator=g).double(), torch.randn(2, H, dk, dv, generator=g).double()


def test_rule_reference_against_the_transition_matrices():
    q, k, v, la, beta, S, _, _ = small()
    y, out, ye, Se, ym = ref.rule(q, k, v, la, beta, [0, 0, 9], S)
    for h in range(2):
        X = S[1, h].clone()
        for t in range(9):
            kt = k[t, 0][:, None]
            X = la[t, h].exp() * (torch.eye(3).double() - beta[t, h] * kt @ kt.T) @ X + beta[t, h] * kt @ v[t, h][None]
            assert torch.allclose(y[t, h], X.T @ q[t, 0], rtol=1e-11, atol=1e-13)
        assert torch.allclose(out[1, h], X, rtol=1e-11, atol=1e-13)
    assert torch.equal(out[0], S[0])


@pytest.mark.parametrize("by_row", [True, False])
def test_gradient_reference_against_differences(by_row):
    q, k, v, la, beta, S, dy, dS = small(3)
    la = la if by_row else la[0]
    cu = [0, 4, 9]
    x = {"dq": q, "dk": k, "dv": v, "dlog_decay": la, "dbeta": beta, "dstates": S}

    def loss(**at):
        z = x | at
        y, out, *_ = ref.rule(z["dq"], z["dk"], z["dv"], z["dlog_decay"], z["dbeta"], cu, z["dstates"])
        return float((y * dy).sum() + (out * dS).sum())

    g, e = ref.gradients(q, k, v, la, beta, cu, dy, S, dS)
    for name, t in x.items():
        gen = torch.Generator().manual_seed(5)
        for _ in range(3):
            d = torch.randn(t.shape, generator=gen, dtype=torch.float64)
            h = 1e-5
            num = (loss(**{name: t + h * d}) - loss(**{name: t - h * d})) / (2 * h)
            assert abs(num - float((g[name] * d).sum())) <= 1e-6 * (1 + abs(num)), name
        assert bool((e[name] >= 0).all())


@pytest.mark.parametrize("T", [0, 5])
def test_sum_over_no_sequence_is_written(T):
    """dlog_decay [H] is an output for a batch without sequences too; nothing else is."""
    s = LinShapeArg(T, 0, 1, 4, 8, 8, 0)
    assert call(s, "bwd", ptr=None, by_row=0) == NULL
    assert call(s, "bwd", ptr=None, by_row=0, dla=P + 1) == ALIGN
    assert call(s, "bwd", ptr=None, by_row=1) == OK
