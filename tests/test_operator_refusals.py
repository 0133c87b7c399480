"""What the recurrence, the multi-axis rotation and the gradient norm refuse, at the C entry points and in
the binding; every check runs before any CUDA call, so this file needs no GPU."""
import ctypes
import os

import numpy as np
import pytest
import torch

import tree_masked_attention_plan_gb300 as tam


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tam.LIB_PATH):
        from tree_masked_attention_plan_gb300 import build_lib
        build_lib.build()
    return tam._lib()


@pytest.fixture(scope="module")
def plan(lib):
    """A plan's descriptor over an address that is never read."""
    par, nl = np.array([-1, 0], np.int32), np.array([100, 60], np.int32)
    info, c = tam.PlanInfo(), tam.PlanT()
    assert lib.tree_plan_query(par.ctypes.data, nl.ctypes.data, 2, ctypes.byref(info)) == 0
    assert lib.tree_plan_bind(ctypes.byref(info), ctypes.c_void_p(1 << 20), ctypes.byref(c)) == 0
    return c


A = 1 << 30                                             # stands for device memory; no check reads it
SHAPE, ARG = -2, -6


def test_scan(lib, plan):
    ok = dict(plan=ctypes.byref(plan), parent=A, node_len=A, gate=A, x=A, init=A, C=64, dtype=0, kind=0, ws=A, y=A, states=A)

    def fwd(**kw):
        a = {**ok, **kw}
        return lib.tree_scan_fwd(a["plan"], a["parent"], a["node_len"], a["gate"], a["x"], a["init"], a["C"], a["dtype"],
                                 a["kind"], a["ws"], a["y"], a["states"], None, None)

    def bwd(**kw):
        a = {**dict(ok, dy=A, dfin=A, dg=A, dx=A, di=A), **kw}
        return lib.tree_scan_bwd(a["plan"], a["parent"], a["node_len"], a["gate"], a["x"], a["init"], a["states"], a["dy"],
                                 a["dfin"], a["C"], a["dtype"], a["kind"], a["ws"], a["dg"], a["dx"], a["di"], None, None)

    for call in (fwd, bwd):
        assert call(plan=None) == ARG
        for name in ("parent", "node_len", "gate", "x", "ws", "states"):
            assert call(**{name: None}) == ARG, name
        for name in ("gate", "x", "ws", "states", "init"):
            assert call(**{name: A + 4}) == ARG, name
        for C in (0, -8, 4, 12):
            assert call(C=C) == SHAPE
        assert call(dtype=2) == SHAPE and call(dtype=-1) == SHAPE and call(kind=2) == SHAPE and call(kind=-1) == SHAPE
    assert fwd(y=None) == ARG and fwd(y=A + 8) == ARG
    for name in ("dy", "dg", "dx"):
        assert bwd(**{name: None}) == ARG and bwd(**{name: A + 2}) == ARG
    assert bwd(di=A + 4) == ARG and bwd(dfin=A + 4) == ARG
    assert lib.tree_scan_workspace(None, 64) == 0 and lib.tree_scan_workspace(ctypes.byref(plan), 0) == 0
    assert lib.tree_scan_workspace(ctypes.byref(plan), 64) > 0


def test_scan_buffers_that_overlap(lib, plan):
    """Outputs overlap nothing but a per-token input as a whole (that is let through to the check of the device)."""
    M = 1 << 22
    names = ("parent", "node_len", "gate", "x", "init", "ws", "y", "states", "dy", "dfin", "dg", "dx", "di")
    at = {n: A + i * M for i, n in enumerate(names)}
    tokens, nodes = 160 * 64 * 2, 2 * 64 * 4

    def fwd(**kw):
        a = {**at, **kw}
        return lib.tree_scan_fwd(ctypes.byref(plan), a["parent"], a["node_len"], a["gate"], a["x"], a["init"], 64, 0, 0,
                                 a["ws"], a["y"], a["states"], None, None)

    def bwd(**kw):
        a = {**at, **kw}
        return lib.tree_scan_bwd(ctypes.byref(plan), a["parent"], a["node_len"], a["gate"], a["x"], a["init"], a["states"],
                                 a["dy"], a["dfin"], 64, 0, 0, a["ws"], a["dg"], a["dx"], a["di"], None, None)

    for name in ("gate", "x", "init", "y"):
        size = nodes if name == "init" else tokens
        for off in (0, 16, size - 16):
            assert fwd(states=at[name] + off) == ARG and fwd(ws=at[name] + off) == ARG
    assert fwd(init=at["states"]) == ARG and fwd(y=at["x"] + 16) == ARG and fwd(y=at["gate"] + tokens - 16) == ARG
    for name in ("gate", "x", "dy", "init", "dfin", "states", "dg", "dx"):
        assert bwd(di=at[name]) == ARG and bwd(ws=at[name]) == ARG, name
    assert bwd(dg=at["dx"]) == ARG and bwd(dx=at["dy"] + 16) == ARG and bwd(dg=at["states"]) == ARG
    if not torch.cuda.is_available():                  # what is allowed gets as far as the device, of which there is none
        for call in (fwd(), fwd(y=at["x"]), fwd(y=at["gate"]), bwd(), bwd(dx=at["dy"]), bwd(dg=at["gate"], dx=at["x"])):
            assert call not in (0, ARG, SHAPE)


def test_rope_axes(lib, plan):
    def call(fn, sections=(16, 24, 24), inter=0, n=None, pos=A, q=A, Hq=4, Hkv=2, d=128, theta=1e4):
        s = (ctypes.c_int32 * max(1, len(sections)))(*sections)
        return fn(ctypes.byref(plan), pos, s, len(sections) if n is None else n, inter, q, A, A, A, Hq, Hkv, d, theta, None)

    for fn in (lib.tree_rope_axes_fwd, lib.tree_rope_axes_bwd):
        assert call(fn, pos=None) == ARG and call(fn, pos=A + 2) == ARG and call(fn, q=None) == ARG and call(fn, q=A + 8) == ARG
        for bad in ((16, 24, 23), (16, 24, 25), (-1, 41, 24), (2 ** 31 - 1, 2 ** 31 - 1, 66)):
            assert call(fn, bad) == SHAPE, bad
        assert call(fn, (0, 0, 64), inter=1) == SHAPE and call(fn, (20, 22, 22), inter=1) == SHAPE
        assert call(fn, (), n=0) == SHAPE and call(fn, (16, 16, 16, 8, 8)) == SHAPE
        assert call(fn, d=96, sections=(16, 16, 16)) == SHAPE and call(fn, Hq=3) == SHAPE and call(fn, Hkv=0) == SHAPE
        assert call(fn, theta=0.0) == SHAPE and call(fn, theta=float("nan")) == SHAPE and call(fn, theta=float("inf")) == SHAPE


def _list(*entries):
    c = (tam.GradT * len(entries))()
    for i, e in enumerate(entries):
        c[i] = tam.GradT(*e, 0)
    return c


def test_grads(lib):
    good = (A, A, 100, 0)

    def norm(lst, n=None, ws=A, out=A):
        return lib.tree_grad_norm(lst, len(lst) if n is None else n, ws, out, None)

    def clip(lst, max_norm=1.0, n=None, ws=A, out=A):
        return lib.tree_grad_clip(lst, len(lst) if n is None else n, max_norm, ws, out, None)

    for call in (norm, clip):
        assert call(_list(good), n=0) == SHAPE and call(_list(good), n=-1) == SHAPE
        assert call(_list((A, A, -1, 0))) == SHAPE and call(_list((A, A, 100, 2))) == SHAPE
        assert call(_list((A, A, 2 ** 60, 0))) == SHAPE
        assert call(_list((None, A, 100, 0))) == ARG and call(_list((A + 1, A + 1, 100, 0))) == ARG
        assert call(_list((A + 2, A + 2, 100, 1))) == ARG
        assert call(_list(good), ws=None) == ARG and call(_list(good), ws=A + 8) == ARG and call(_list(good), out=None) == ARG
        assert call(_list(good), out=A + 2) == ARG
    assert lib.tree_grad_norm(None, 1, A, A, None) == ARG
    assert clip(_list((A, None, 100, 0))) == ARG
    for bad in (-1.0, float("nan")):
        assert clip(_list(good), bad) == SHAPE
    overlaps = [_list(good, good),                                        # the same one twice, in place
                _list(good, (A + 100, A + 100, 100, 0)),                  # two that share elements, in place
                _list((A, A + 2, 100, 0)),                                # its own gradient, moved by one
                _list((A, A + 4096, 100, 0), (A + 8192, A + 4100, 100, 0)),   # two targets
                _list((A, A + 4096, 100, 0), (A + 4200, A + 8192, 100, 0)),   # a target on another's gradient
                _list((A + 4200, A + 8192, 100, 0), (A, A + 4096, 100, 0))]
    for lst in overlaps:
        assert clip(lst) == ARG
    assert lib.tree_grad_workspace(0) == 0 and lib.tree_grad_workspace(5) > 0


def test_the_binding(plan):
    t = torch.zeros(4)
    with pytest.raises(ValueError):
        tam.tree_grad_list([])
    with pytest.raises(ValueError):
        tam.tree_grad_list([t])                                           # not on a GPU
    with pytest.raises(ValueError):
        tam.tree_grad_list([t], out=[t, t])
    with pytest.raises(ValueError):
        tam.tree_grad_list([torch.zeros(4, dtype=torch.float16)])
    p = tam.TreePlan(info=tam.PlanInfo(n_nodes=2, n_tokens=160, n_tiles=2), buf=None, c=plan, device=torch.device("cuda", 0))
    x = torch.zeros(160, 64)
    with pytest.raises(ValueError, match="gate_kind"):
        tam.tree_scan_fwd(p, (None, None), x, x, gate_kind="relu")
    with pytest.raises(ValueError, match="x must be"):
        tam.tree_scan_fwd(p, (None, None), x, x.half())
    with pytest.raises(ValueError, match="expected contiguous CUDA"):
        tam.tree_scan_fwd(p, (None, None), x, x)


def test_axis_positions():
    parent, lens = [-1, 0, 1, 0, -1], [3, 4, 2, 1, 2]
    local = np.zeros((2, 12), int)
    local[:, :3] = [0, 1, 2]
    local[:, 3:7] = [[0, 0, 1, 1], [0, 1, 0, 1]]       # a 2 x 2 image
    local[:, 7:9] = [0, 1]
    local[:, 10:] = [0, 1]
    got = tam.tree_axis_positions(parent, lens, [3, 2, 2, 1, 2], local, base=10)
    assert got.dtype == np.int32
    assert got.tolist() == [[10, 11, 12, 13, 13, 14, 14, 15, 16, 13, 10, 11], [10, 11, 12, 13, 14, 13, 14, 15, 16, 13, 10, 11]]
    with pytest.raises(ValueError):
        tam.tree_axis_positions(parent, lens, [3, 2], local)
    with pytest.raises(ValueError):
        tam.tree_axis_positions(parent, lens, [3, 2, 2, 1, 2], local[:, :5])
    with pytest.raises(ValueError):
        tam.tree_axis_positions(parent, lens, [3, 2, 2, 1, 2], local, base=2 ** 31 - 3)
