"""Sizes and arguments that the entry points take or refuse, in addition to test_operator_refusals.py; no GPU needed."""
import ctypes
import os

import numpy as np
import pytest

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
