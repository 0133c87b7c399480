"""Sizes and arguments that the entry points take or refuse, in addition to test_operator_refusals.py; no GPU needed."""
import ctypes
import os

import numpy as np
import pytest

import tree_masked_attention_plan_gb300 as tam


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
