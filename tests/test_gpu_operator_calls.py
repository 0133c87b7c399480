"""Calls of the recurrence, the several-axis rotation and the gradient norm that their documentation allows, beside the
ordinary ones: plans of a device without a number."""
import pytest
import torch

import tree_masked_attention_plan_gb300 as tam

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
B, F = torch.bfloat16, torch.float32


def test_a_plan_of_a_device_without_a_number():
    """tree_plan(device="cuda") is the current device's plan: the same bits as that of cuda:0."""
    parent, lens = [-1, 0, 0], [100, 60, 40]
    N, C = sum(lens), 64
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    gate, x, dy, init = r(N, C).to(B), r(N, C).to(B), r(N, C).to(B), r(3, C)
    q, k = r(N, 4, 64).to(B), r(N, 2, 64).to(B)
    pos = torch.arange(N, dtype=torch.int32, device=DEV).repeat(2, 1)
    res = []
    for dev in ("cuda", DEV):
        plan = tam.tree_plan(parent, lens, device=dev)
        tree = tam.tree_arrays(parent, lens, dev)
        assert plan.device == DEV
        y, st = tam.tree_scan_fwd(plan, tree, gate, x, init=init)
        res.append([y, st, *tam.tree_scan_bwd(plan, tree, gate, x, st, dy, init=init),
                    *tam.tree_rope_axes_fwd(plan, pos, q, k, (20, 12)), *tam.tree_rope_axes_bwd(plan, pos, q, k, (20, 12))])
    for a, b in zip(*res):
        assert torch.equal(a, b)
