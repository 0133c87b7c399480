"""Rotary positions with several axes against fp64, forward and backward.

Tolerances: the angle is exact to 2^-24 turns (2^-25 from the float, as much from the table), that is 2 pi
2^-24 < 2^-21 of the pair's length, sine and cosine add 2 units of 2^-24 and the two products and the sum 3,
all below 2^-20 of |x| + |y|; the result is rounded to bf16 once, half a step: 2^-8 of the value."""
import numpy as np
import pytest
import torch

import tree_masked_attention_plan_gb300 as tam
from workloads import random_tree

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def axis_of(sections, interleaved, half):
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    axis = np.zeros(half, dtype=int)
    for i in range(1, len(sections)):
        axis[i + len(sections) * np.arange(sections[i])] = i
    return axis


def rotate(x, pos, sections, theta, interleaved, sign):
    half = x.shape[-1] // 2
    freq = float(np.float32(theta)) ** (-np.arange(half) / half)
    ang = sign * (pos[axis_of(sections, interleaved, half)].T.astype(np.float64) * freq)[:, None, :]
    a, b = x[..., :half], x[..., half:]
    ref = np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], -1)
    size = np.abs(a) + np.abs(b)
    return ref, np.concatenate([size, size], -1)


def _close(got, x, pos, sections, theta, interleaved, sign):
    ref, size = rotate(x.double().numpy(), pos, sections, theta, interleaved, sign)
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size
    assert (err <= tol).all(), (np.argwhere(err > tol)[:4], err.max())


CASES = [(1, 1, 1, 64, (32,), False, 0), (48, 32, 8, 128, (16, 24, 24), False, 70000), (333, 16, 16, 64, (12, 10, 10), True, 0),
         (2500, 6, 2, 128, (22, 21, 21), True, 10 ** 6), (77, 5, 5, 64, (0, 16, 16), False, 0),
         (130, 3, 1, 128, (16, 16, 16, 16), True, -5000), (65, 40, 8, 64, (20, 12), False, 2 ** 31 - 200)]


@pytest.mark.parametrize("N,Hq,Hkv,d,sections,interleaved,start", CASES)
def test_forward_and_backward(N, Hq, Hkv, d, sections, interleaved, start):
    rng = np.random.default_rng(N)
    pos = (start + rng.integers(0, 150, (len(sections), N))).astype(np.int32)
    g = torch.Generator().manual_seed(N)
    q, k = (torch.randn(N, h, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv))
    plan = tam.tree_plan([-1], [N], device=DEV)
    p = torch.from_numpy(pos).to(DEV)
    theta = 10000.0 if N % 2 else 500000.0
    for fn, sign in ((tam.tree_rope_axes_fwd, 1), (tam.tree_rope_axes_bwd, -1)):
        oq, ok = fn(plan, p, q.to(DEV), k.to(DEV), sections, theta=theta, interleaved=interleaved)
        _close(oq, q, pos, sections, theta, interleaved, sign)
        _close(ok, k, pos, sections, theta, interleaved, sign)


def test_one_axis_is_the_plans_own_rotation_and_in_place_is_the_same():
    parent, node_len = random_tree(21, 20, max_len=40, n_roots=2)
    plan = tam.tree_plan(parent, node_len, device=DEV)
    N = plan.n_tokens
    q, k = (torch.randn(N, h, 128, device=DEV).to(torch.bfloat16) for h in (8, 2))
    pos = plan.arrays()["pos"][:N].reshape(1, N).contiguous()
    a = tam.tree_rope_axes_fwd(plan, pos, q, k, [64])
    b = tam.tree_rope_fwd(plan, q, k)
    for x, y in zip(a, b):                             # two roundings of nearly the same value: a step apart at most
        assert ((x.float() - y.float()).abs() <= 2.0 ** -7 * y.float().abs() + 1e-4).all()
    qi, ki = q.clone(), k.clone()
    tam.tree_rope_axes_fwd(plan, pos, qi, ki, [64], qr=qi, kr=ki)
    assert torch.equal(qi, a[0]) and torch.equal(ki, a[1])


def test_attention_of_a_tree_with_image_patches():
    """Text, an image and an answer on two branches: positions from the host helper, rotation, attention, its backward and
    the rotation's; the gradients against torch's through the same steps in fp64."""
    parent, lens = [-1, 0, 1, 0], [20, 16, 9, 30]       # node 1 is a 4 x 4 image
    N, Hq, Hkv, d, sections = sum(lens), 4, 2, 64, [8, 12, 12]
    local = np.concatenate([np.tile(np.arange(20), (3, 1)), np.stack([np.zeros(16, int), np.arange(16) // 4, np.arange(16) % 4]),
                            np.tile(np.arange(9), (3, 1)), np.tile(np.arange(30), (3, 1))], 1)
    pos = tam.tree_axis_positions(parent, lens, [20, 4, 9, 30], local)
    assert pos[0, 36] == 24 and pos[2, 35] == 23 and pos[1, 45] == 20
    g = torch.Generator().manual_seed(3)
    q, k, v, u = (torch.randn(N, h, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv, Hq))
    plan = tam.tree_plan(parent, lens, device=DEV)
    p = torch.from_numpy(pos).to(DEV)
    status = tam.new_status(DEV)
    qr, kr = tam.tree_rope_axes_fwd(plan, p, q.to(DEV), k.to(DEV), sections)
    o, lse = tam.tree_attn_fwd(plan, qr, kr, v.to(DEV), status=status)
    dqr, dkr, dv = tam.tree_attn_bwd(plan, qr, kr, v.to(DEV), o, lse, u.to(DEV), rope_theta=0.0, status=status)
    dq, dk = tam.tree_rope_axes_bwd(plan, p, dqr, dkr, sections)
    torch.cuda.synchronize()
    tam.check_status(status)
    leaf = [t.double().requires_grad_() for t in (q, k, v)]
    ang = torch.from_numpy(pos[axis_of(sections, False, 32)].T.astype(np.float64) * 10000.0 ** (-np.arange(32) / 32))[:, None]

    def rot(x):
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    node = np.repeat(np.arange(4), lens)
    up = {0: {0}, 1: {0, 1}, 2: {0, 1, 2}, 3: {0, 3}}
    see = torch.tensor([[j <= i and node[j] in up[node[i]] for j in range(N)] for i in range(N)])
    kk, vv = (t.repeat_interleave(2, 1) for t in (rot(leaf[1]), leaf[2]))
    s = torch.einsum("ihd,jhd->hij", rot(leaf[0]), kk) / 8
    want = torch.einsum("hij,jhd->ihd", s.masked_fill(~see, -np.inf).softmax(-1), vv)
    (want * u.double()).sum().backward()
    assert (o.double().cpu() - want).abs().max() <= 2e-2
    for got, ref in ((dq, leaf[0].grad), (dk, leaf[1].grad), (dv, leaf[2].grad)):
        assert (got.double().cpu() - ref).abs().max() <= 5e-2 * ref.abs().max()
