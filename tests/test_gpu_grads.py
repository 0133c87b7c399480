"""The global gradient norm and clipping against fp64.

Tolerances: a vector's squares are summed in fp32 (8 products and sums: 9 units of 2^-24 of the sum at most),
everything else in fp64, and the root halves a relative error: 5 units, with the result's own rounding 6.
Clipped values: one product in fp32 with a coefficient off by 6 + 2 units and one rounding, half a step."""
import numpy as np
import pytest
import torch

import tree_masked_attention_plan_gb300 as tam

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
NORM = 6 * 2.0 ** -24


def _norm(grads):
    return float(np.sqrt(sum((g.double() ** 2).sum().item() for g in grads)))


def _make(sizes, dtypes, scale=1.0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(scale * torch.randn(*([n] if isinstance(n, int) else n), generator=g, device=DEV)).to(t) for n, t in zip(sizes, dtypes)]


def _check_clip(grads, max_norm, out=None):
    before = [g.double() for g in grads]
    norm = _norm(grads)
    got = tam.tree_grad_clip(tam.tree_grad_list(grads, out=out), max_norm)
    assert abs(got.item() - norm) <= NORM * norm
    c = max_norm / norm if norm > max_norm else 1.0
    for b, o in zip(before, out or grads):
        if c == 1.0:
            assert torch.equal(o.double(), b)
        else:
            assert ((o.double() - c * b).abs() <= (HALF[o.dtype] + 10 * 2.0 ** -24) * (c * b).abs() + 1e-40).all()


B, F = torch.bfloat16, torch.float32
LISTS = [([1], [F]), ([1], [B]), ([7, 0, 16384, 16385, 3], [B, F, F, B, B]), ([(33, 65), (5, 3, 9), 100003], [F, B, B]),
         ([5000 + 13 * i for i in range(90)], [(B, F)[i % 2] for i in range(90)]), ([1 + i % 7 for i in range(2000)], [B] * 2000),
         ([20_000_001, 4_000_003], [B, F])]


@pytest.mark.parametrize("sizes,dtypes", LISTS, ids=range(len(LISTS)))
def test_norm_and_clip(sizes, dtypes):
    grads = _make(sizes, dtypes)
    norm = _norm(grads)
    got = tam.tree_grad_norm(grads)
    assert abs(got.item() - norm) <= NORM * norm
    assert torch.equal(got, tam.tree_grad_norm(grads))
    _check_clip(grads, 2 * norm)
    out = [torch.full_like(g, 7) for g in grads]
    keep = [g.clone() for g in grads]
    _check_clip(grads, 2 * norm, out)
    _check_clip(grads, norm / 3, out)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    _check_clip(grads, norm / 3)


def test_views_at_odd_places():
    """Gradients and targets that start anywhere in a buffer, alike and unlike within 16 bytes; what lies between stays."""
    for dt in (B, F):
        src = torch.randn(40000, device=DEV).to(dt)
        for a, b, n in ((1, 1, 3000), (3, 11, 17001), (5, 6, 2999), (0, 7, 1), (2, 3, 9)):
            dst = torch.full((40000,), 3.0, device=DEV, dtype=dt)
            _check_clip([src[a:a + n]], 0.01, [dst[b:b + n]])
            assert (dst[:b] == 3).all() and (dst[b + n:] == 3).all()


@pytest.mark.parametrize("scale", [1e25, 1e-25, 1e-40, 3e18])
def test_squares_that_leave_fp32(scale):
    grads = _make([5000, 33], [F, F], 1.0, 3)
    grads = [(g.double() * scale).float() for g in grads]
    norm = _norm(grads)
    assert abs(tam.tree_grad_norm(grads).item() - norm) <= NORM * norm + 2.0 ** -149
    mixed = _make([1000], [F]) + grads
    assert abs(tam.tree_grad_norm(mixed).item() - _norm(mixed)) <= NORM * _norm(mixed)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("at", [0, 777, 4999])
def test_a_norm_that_is_no_number_leaves_the_gradients(bad, at):
    grads = _make([5000, 300], [B, F])
    grads[0][at] = bad
    keep, out = [g.clone() for g in grads], [torch.empty_like(g) for g in grads]
    for gl in (tam.tree_grad_list(grads, out=out), tam.tree_grad_list(grads)):
        norm = tam.tree_grad_clip(gl, 0.5)
        assert (torch.isnan(norm) if bad != bad else torch.isinf(norm)).all()
        for o, k in zip(gl.out, keep):
            assert torch.equal(o.view(torch.uint8), k.view(torch.uint8))


def test_zeros_and_the_ends_of_max_norm():
    z = [torch.zeros(1000, device=DEV), torch.zeros(3, device=DEV, dtype=B)]
    assert tam.tree_grad_clip(z, 0.0).item() == 0 and all((t == 0).all() for t in z)
    g = _make([1000], [F])
    keep = g[0].clone()
    tam.tree_grad_clip(g, float("inf"))
    assert torch.equal(g[0], keep)
    tam.tree_grad_clip(g, 0.0)
    assert (g[0] == 0).all()


def test_captured_replayed_and_on_another_stream():
    grads = _make([70001, 500, 12], [B, F, B])
    out = [torch.empty_like(g) for g in grads]
    gl = tam.tree_grad_list(grads, out=out)
    want = tam.tree_grad_clip(gl, 1.0).clone(), [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    norm = torch.empty(1, device=DEV)
    with torch.cuda.graph(graph):
        tam.tree_grad_clip(gl, 1.0, norm=norm)
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, want[0]) and all(torch.equal(a, b) for a, b in zip(out, want[1]))
    for g in grads:
        g.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, 2 * want[0])
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    other = tam.tree_grad_norm(gl, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, norm)


def test_the_gradients_of_a_hybrid_layers_step():
    """The recurrence after the causal convolution on one tree, rotary positions beside it, the loss at the end: their
    parameter gradients under one norm, as a training step clips them."""
    from workloads import random_tree
    parent, node_len = random_tree(77, 20, max_len=60, n_roots=2)
    N, C, V = int(node_len.sum()), 256, 1000
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)
    plan, tree = tam.tree_plan(parent, node_len, device=DEV), tam.tree_arrays(parent, node_len, DEV)
    x, gate, w, b = r(N, C).to(B), (r(N, C) + 2).to(B), r(4, C) / 2, r(C)
    W = (r(V, C) / 16).to(B)
    labels = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).to(DEV)
    status = tam.new_status(DEV)
    c = tam.tree_conv1d_fwd(plan, tree, x, w, b, status=status)
    h, states = tam.tree_scan_fwd(plan, tree, gate, c, status=status)
    loss, _, dh, dW = tam.tree_ce_fwd_bwd(plan, tree, h, W, labels, chunk=256, status=status)
    dgate, dc, _ = tam.tree_scan_bwd(plan, tree, gate, c, states, dh, status=status)
    dx, dw, db = tam.tree_conv1d_bwd(plan, tree, x, w, dc, with_bias=True, status=status)
    grads = [dW, dw, db]
    norm = _norm(grads)
    assert norm > 0
    _check_clip(grads, norm / 10)
    assert abs(_norm(grads) - norm / 10) <= 1e-5 * norm
    tam.check_status(status)
    # the same step in fp64 from the layer's own bf16 values: convolution, recurrence and loss by torch's autograd
    import oracle
    from oracle import scan as osc
    p = oracle.plan(parent, node_len)
    prev = osc.token_prev(parent, node_len, p)
    f = [t.double().cpu().requires_grad_() for t in (x, gate, w, b)]
    rows, hs, cs = torch.cat([f[0], torch.zeros(1, C, dtype=torch.float64)]), [], []
    for t in range(N):
        at, acc = t, f[3]
        for k in range(4):
            acc = acc + f[2][k] * rows[at]
            at = prev[at] if at >= 0 else -1
            if at < 0:
                break
        a = torch.sigmoid(f[1][t])
        hs.append((1 - a) * acc + (a * hs[prev[t]] if prev[t] >= 0 else 0))
    logits = torch.stack(hs) @ W.double().cpu().T
    pair = [(t, prev[t]) for t in range(N) if prev[t] >= 0]
    wgt = torch.tensor(p["g"] / p["n_paths"])
    ref = sum(wgt[t] * torch.nn.functional.cross_entropy(logits[s][None], labels[t:t + 1].long().cpu()) for t, s in pair)
    ref.backward()
    assert abs(loss.item() - ref.item()) <= 2e-2 * abs(ref.item())
    for got, leaf in ((dx, f[0]), (dgate, f[1]), (dw * 10, f[2]), (db * 10, f[3])):
        assert (got.double().cpu() - leaf.grad).norm() <= 3e-2 * leaf.grad.norm()
