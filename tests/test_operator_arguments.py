"""Sizes and arguments that the entry points take or refuse, in addition to test_operator_refusals.py; no GPU needed."""
import ctypes
import os

import numpy as np
import pytest
import torch

import tree_masked_attention_plan_gb300 as tam

SHAPE, ARG = -2, -6


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tam.LIB_PATH):
        from tree_masked_attention_plan_gb300 import build_lib
        build_lib.build()
    return tam._lib()


@pytest.mark.parametrize("parent,lens,longest", [([-1], [7], 7), ([-1, 0, -1], [3, 0, 9], 9), ([-1, 0], [0, 1], 1)])
def test_the_longest_node(lib, parent, lens, longest):
    par, nl = np.array(parent, np.int32), np.array(lens, np.int32)
    info, c = tam.PlanInfo(), tam.PlanT()
    assert lib.tree_plan_query(par.ctypes.data, nl.ctypes.data, len(lens), ctypes.byref(info)) == 0
    assert lib.tree_plan_bind(ctypes.byref(info), ctypes.c_void_p(1 << 20), ctypes.byref(c)) == 0
    assert info.max_len == c.max_len == longest


def test_scan_of_more_channels_than_its_counts_hold(lib):
    par, nl = np.array([-1], np.int32), np.array([1], np.int32)
    info, plan = tam.PlanInfo(), tam.PlanT()
    assert lib.tree_plan_query(par.ctypes.data, nl.ctypes.data, 1, ctypes.byref(info)) == 0
    assert lib.tree_plan_bind(ctypes.byref(info), ctypes.c_void_p(1 << 20), ctypes.byref(plan)) == 0
    A = 1 << 30
    for C in (2 ** 28 + 8, 2 ** 30, 2 ** 31 - 8):
        assert lib.tree_scan_fwd(ctypes.byref(plan), A, A, A, A, None, C, 0, 0, A, A, A, None, None) == SHAPE
        assert lib.tree_scan_bwd(ctypes.byref(plan), A, A, A, A, None, A, A, None, C, 0, 0, A, A, A, None, None, None) == SHAPE


def test_rope_axes_buffers_that_overlap(lib):
    """An output overlaps nothing but its own input as a whole (that is let through to the check of the device)."""
    par, nl = np.array([-1, 0], np.int32), np.array([100, 60], np.int32)
    info, plan = tam.PlanInfo(), tam.PlanT()
    assert lib.tree_plan_query(par.ctypes.data, nl.ctypes.data, 2, ctypes.byref(info)) == 0
    assert lib.tree_plan_bind(ctypes.byref(info), ctypes.c_void_p(1 << 20), ctypes.byref(plan)) == 0
    N, Hq, Hkv, d, M = 160, 4, 2, 64, 1 << 24
    size = dict(pos=N * 3 * 4, q=N * Hq * d * 2, k=N * Hkv * d * 2, qr=N * Hq * d * 2, kr=N * Hkv * d * 2)
    at = {n: (1 << 30) + i * M for i, n in enumerate(size)}
    sec = (ctypes.c_int32 * 3)(12, 10, 10)

    for fn in (lib.tree_rope_axes_fwd, lib.tree_rope_axes_bwd):
        def call(**kw):
            a = {**at, **kw}
            return fn(ctypes.byref(plan), a["pos"], sec, 3, 0, a["q"], a["k"], a["qr"], a["kr"], Hq, Hkv, d, 1e4, None)

        for out, own in (("qr", "q"), ("kr", "k")):
            for other in ("pos", "q", "k", "qr", "kr"):
                if other == out:
                    continue
                for off in (0, 16, size[other] - 16, 16 - size[out]):
                    if not (other == own and off == 0):
                        assert call(**{out: at[other] + off}) == ARG, (out, other, off)
        assert call(qr=at["k"], kr=at["q"]) == ARG and call(q=at["k"], qr=at["k"]) == ARG
        if not torch.cuda.is_available():              # what is allowed gets as far as the device, of which there is none
            for good in (call(), call(qr=at["q"]), call(kr=at["k"]), call(qr=at["q"], kr=at["k"]), call(q=at["k"]),
                         call(qr=at["k"] + size["k"]), call(kr=at["q"] - size["kr"])):
                assert good not in (0, ARG, SHAPE)


def test_workspace_and_norm_that_overlap(lib):
    """Neither lies in a gradient, a target or the other one."""
    A, M = 1 << 30, 1 << 20
    c = (tam.GradT * 3)()
    for i, (numel, dtype) in enumerate(((1000, 0), (0, 1), (500, 1))):
        c[i] = tam.GradT(A + 2 * i * M, A + (2 * i + 1) * M, numel, dtype, 0)
    ws, norm, size = A + 10 * M, A + 11 * M, lib.tree_grad_workspace(3)
    spots = [A, A + 1984, A + 4 * M, A + 4 * M + 1996]
    targets = [p + M for p in spots]

    def run(name, ws=ws, norm=norm):
        return lib.tree_grad_norm(c, 3, ws, norm, None) if name == "norm" else lib.tree_grad_clip(c, 3, 1.0, ws, norm, None)

    for name in ("norm", "clip"):
        for p in spots + (targets if name == "clip" else []):
            assert run(name, norm=p) == ARG and run(name, ws=p & ~15) == ARG and run(name, ws=(p & ~15) + 16 - size) == ARG
        assert run(name, norm=ws) == ARG and run(name, norm=ws + size - 4) == ARG
        if not torch.cuda.is_available():
            for good in (run(name), run(name, norm=A + 2 * M), run(name, norm=ws + size), run(name, norm=A + 2000)):
                assert good not in (0, ARG, SHAPE)
