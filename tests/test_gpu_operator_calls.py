"""Calls of the recurrence, the several-axis rotation and the gradient norm that their documentation allows, beside the
ordinary ones: plans of a device without a number, lists that are dropped while another stream works on them, steps of
sequences one of which is long, waits that run out, very
wide layers."""
import numpy as np
import pytest
import torch

import tree_masked_attention_plan_gb300 as tam
from oracle import scan as osc

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


def _forward(lens, C=64, seed=3):
    """Nodes that are sequences of their own through the recurrence, against its oracle (24 units of 2^-24 a token, as the
    recurrence's own tests count them); whether it left the workspace as it was."""
    N, n = sum(lens), len(lens)
    g = torch.Generator().manual_seed(seed)
    gate, x, init = torch.randn(N, C, generator=g) + 2, torch.randn(N, C, generator=g), torch.randn(n, C, generator=g)
    plan, tree = tam.tree_plan([-1] * n, lens, device=DEV), tam.tree_arrays([-1] * n, lens, DEV)
    ws = torch.full((tam.tree_scan_workspace(plan, C),), 0xA5, dtype=torch.uint8, device=DEV)
    y, st = tam.tree_scan_fwd(plan, tree, gate.to(DEV), x.to(DEV), init=init.to(DEV), workspace=ws)
    ref = osc.scan([-1] * n, lens, gate.double().numpy(), x.double().numpy(), "sigmoid", init=init.double().numpy())
    for got, name in ((y, "y"), (st[:n], "final")):
        err = np.abs(got.double().cpu().numpy() - ref[name])
        assert (err <= 24 * 2.0 ** -24 * ref["e_" + name] + 2.0 ** -24 * np.abs(ref[name]) + 1e-37).all()
    return bool((ws == 0xA5).all())


@pytest.mark.parametrize("lens", [[0] * 3000 + [20000] + [0] * 17000, [1] * 700 + [0] * 5000 + [4000, 3] + [1] * 200])
def test_one_long_sequence_among_many_empty_ones(lens):
    """No more tokens than nodes, yet one sequence of many: a matter for the kernels that work along a sequence in
    parallel, which keep what its tiles hand on in the workspace."""
    assert sum(lens) <= len(lens)
    assert not _forward(lens)


@pytest.mark.parametrize("lens", [[1] * 600 + [3, 0, 0, 0, 2], [1] * 100 + [0] * 400 + [128] + [1] * 90 + [100, 77],
                                  [0] * 500 + [1, 128, 128, 2, 126, 1]])
def test_a_step_with_some_sequences_of_more_tokens(lens):
    """One launch and nothing in the workspace; sequences that go on behind the 128 tokens of a block."""
    assert 256 < sum(lens) <= len(lens) and max(lens) <= 128
    assert _forward(lens)


def test_waits_that_run_out():
    """A path through 469 tiles under the shortest limit: some of the tiles that are worked on at once wait longer than 0.1
    ms for the state before them.  The status word says so, the call ends, and the next one with the same buffers is right."""
    parent, lens, trunk = [-1], [256], 0
    while sum(lens) < 60000:                           # a trunk's segment, the leaf that follows it, then the trunk's next
        parent += [trunk, len(lens)]
        lens += [64, 16]
        trunk = len(lens) - 2
    N, n, C = sum(lens), len(lens), 64
    g = torch.Generator(device=DEV).manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    gate, x, dy = r(N, C) + 2, r(N, C), r(N, C)
    plan, tree = tam.tree_plan(parent, lens, device=DEV), tam.tree_arrays(parent, lens, DEV)
    ws = torch.empty(tam.tree_scan_workspace(plan, C), dtype=torch.uint8, device=DEV)
    status = tam.new_status(DEV)

    def forward():
        return tam.tree_scan_fwd(plan, tree, gate, x, workspace=ws, status=status)

    def backward(states):
        return tam.tree_scan_bwd(plan, tree, gate, x, states, dy, workspace=ws, status=status)[:2]

    want = forward()
    want += backward(want[1])
    tam.check_status(status, "scan")
    for call in (forward, lambda: backward(want[1])):
        tam.tree_set_wait_limit_ns(100000)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            tam.tree_set_wait_limit_ns(2000000000)
        assert status.item() == -5
        with pytest.raises(tam.TreeError):
            tam.check_status(status, "scan")
        status.zero_()
        got = forward()
        got += backward(got[1])
        tam.check_status(status, "scan")
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("lens", [[2], [1, 3, 2]])
def test_a_layer_wider_than_a_grid_goes(lens):
    """2^26 + 2^20 channels of a few tokens: more slabs and more shares of 1024 channels than 65535.  The sampled channels
    hold their own values, the others zeros."""
    N, n, C = sum(lens), len(lens), (1 << 26) + (1 << 20)
    at = torch.tensor([0, 1, 63, 64, 1 << 20, (1 << 26) - 1, 1 << 26, C - 1], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(6)
    gate, x, dy = (torch.randn(N, 8, generator=g, device=DEV).to(B) for _ in range(3))

    def wide(v):
        w = torch.zeros(N, C, dtype=B, device=DEV)
        w[:, at] = v
        return w

    parent = list(range(-1, n - 1))
    plan, tree = tam.tree_plan(parent, lens, device=DEV), tam.tree_arrays(parent, lens, DEV)
    status = tam.new_status(DEV)
    narrow = tam.tree_scan_fwd(plan, tree, gate, x)
    narrow += tam.tree_scan_bwd(plan, tree, gate, x, narrow[1], dy)[:2]
    g, v, d = wide(gate), wide(x), wide(dy)
    got = tam.tree_scan_fwd(plan, tree, g, v, status=status)
    got += tam.tree_scan_bwd(plan, tree, g, v, got[1], d, status=status)[:2]
    tam.check_status(status, "scan")
    for i, (a, b) in enumerate(zip(got, narrow)):
        assert torch.equal(a[:, at], b), i
        assert int((a != 0).sum()) <= a.shape[0] * 8
