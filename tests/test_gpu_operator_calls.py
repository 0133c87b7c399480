"""Calls of the recurrence, the several-axis rotation and the gradient norm that their documentation allows, beside the
ordinary ones: plans of a device without a number, lists that are dropped while another stream works on them."""
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


@pytest.mark.parametrize("held", [False, True])
def test_a_gradient_list_that_is_dropped_while_another_stream_works_on_it(held):
    """The partial sums of a call on a side stream are its own until it has ended: blocks of their size that the current
    stream allocates and writes meanwhile are others.  1700 tensors: sums of three launches wait for the last."""
    sizes = [40000 + 17 * (i % 91) for i in range(1700)]
    g = torch.Generator(device=DEV).manual_seed(2)
    flat = torch.randn(sum(sizes), generator=g, device=DEV)
    grads = list(flat.split(sizes))
    before, size = flat.clone(), int(tam._lib().tree_grad_workspace(len(grads)))
    keep = tam.tree_grad_list(grads)
    want = tam.tree_grad_norm(keep).clone()
    max_norm = want.item() / 3
    side, big = torch.cuda.Stream(DEV), torch.zeros(1 << 28, device=DEV)
    for clip in (False, True):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(4):
                big.add_(1.0)                          # (the calls' kernels wait behind these)
        gl = tam.tree_grad_list(grads) if held else grads
        norm = tam.tree_grad_clip(gl, max_norm, stream=side) if clip else tam.tree_grad_norm(gl, stream=side)
        gl = None
        done = side.record_event()
        others = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(16)]
        while not done.query():
            for b in others:
                b.fill_(0x55)                          # as fp64: 1e103
        torch.cuda.synchronize()
        assert torch.equal(norm, want)
    assert ((flat.double() - before.double() / 3).abs() <= 2.0 ** -20 * before.abs()).all()
