"""How near the operators come to their definition at values where fewer bits would show.  Rounding units are 2^-24."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import tree_masked_attention_plan_gb300 as tam

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("n,tail", [(200, 0), (700, 0), (700, 300)])
def test_the_weight_of_the_input_at_strong_sigmoid_gates(n, tail):
    """One token a sequence, no state before it: y = (1 - a) x, and with x = 0 from a state of one y = a.  1 - a = e / (1 + e),
    a = 1 / (1 + e), e = e^-g: the power 2^t is right to 2^-22 (4 units), what its argument lost is put back but for the
    error of ln 2 in fp32 (0.05 units for each unit of g: 4.4 at 87) and one rounding; 1 + e and the reciprocal (2^-23)
    take 1 + 2, two products 1: 13 units at most."""
    C, lens = 8, [1] * n + [tail] * (tail > 0)         # (with the tail: the kernels for many tokens)
    g = torch.linspace(-86.5, 86.5, n * C).reshape(n, C)
    x = torch.rand(n, C, generator=torch.Generator().manual_seed(1)) + 1
    plan, tree = tam.tree_plan([-1] * len(lens), lens, device=DEV), tam.tree_arrays([-1] * len(lens), lens, DEV)
    long = lambda t: torch.cat([t, torch.zeros(tail, C)]).to(DEV)
    y, _ = tam.tree_scan_fwd(plan, tree, long(g), long(x))
    a, _ = tam.tree_scan_fwd(plan, tree, long(g), long(0 * x), init=torch.ones(len(lens), C, device=DEV))
    gd = g.double().numpy()
    for got, ref in ((y, x.double().numpy() / (1 + np.exp(gd))), (a, 1 / (1 + np.exp(-gd)))):
        off = np.abs(got[:n].double().cpu().numpy() - ref) / ref * 2.0 ** 24
        assert off.max() <= 13, (off.max(), gd.flat[off.argmax()])


@pytest.mark.parametrize("rate", [1e-7, 2e-8, 1e-5])
@pytest.mark.parametrize("n", [200, 5000])
def test_decays_next_to_one(n, rate):
    """A state of one that only decays, by 1 - a = `rate` a token: decay and step are rounded by 2^-25 each, where tiles are
    joined a map's product and the sum behind it again (twice a tile of 128): 1.1 units of 2^-24 a token."""
    C = 8
    plan, tree = tam.tree_plan([-1], [n], device=DEV), tam.tree_arrays([-1], [n], DEV)
    g = torch.full((n, C), -rate, device=DEV)
    y, _ = tam.tree_scan_fwd(plan, tree, g, torch.zeros(n, C, device=DEV), init=torch.ones(1, C, device=DEV), gate_kind="log")
    t = np.arange(1, n + 1)
    off = np.abs(y.double().cpu().numpy() - np.exp(t * float(np.float32(-rate)))[:, None])
    assert (off <= 1.1 * 2.0 ** -24 * t[:, None]).all()


@pytest.mark.parametrize("n", [3, 5, 50000])
def test_the_coefficient_of_clipping(n):
    """max_norm is taken as it is given: the coefficient max_norm / norm is rounded once, half a step of fp32, one unit at
    most.  Equal elements of 2 have exact squares and sums, and their product with the coefficient is exact."""
    for max_norm in np.random.default_rng(n).uniform(0.1, 0.9, 40):
        grads = [torch.full((n,), 2.0, device=DEV)]
        norm = 2.0 * np.sqrt(np.float64(n))
        tam.tree_grad_clip(grads, float(max_norm))
        off = abs(grads[0][0].item() / (2.0 * max_norm / norm) - 1) * 2.0 ** 24
        assert off <= 1 + 1e-6 and (grads[0] == grads[0][0]).all(), (max_norm, off)


@pytest.mark.parametrize("theta", [1.0, 1.25, 2.0, 10000.0, 1e12, 0.5, 0.01, 1e-4, 2.0 ** -40])
@pytest.mark.parametrize("d", [64, 128])
def test_angles_at_the_ends_of_the_positions(theta, d):
    """The rotation of a pair (1, 0) is (cos, sin) of its angle, which is right to 2^-25 turns at every position for every
    theta of 2^-40 and more; sine and cosine add 2 units of 2^-24, the result is rounded to bf16, half a step.  Most of the
    4000 positions are far out, so that some cosines and sines lie at zero and at borders of rounding, where the angle shows."""
    half = d // 2
    ps = [0, 1, -1, 12345, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 2 ** 31 - 54321]
    ps += [int(v) for v in np.random.default_rng(d).integers(-2 ** 31, 2 ** 31, 4000)]
    N = len(ps)
    q = torch.zeros(N, 1, d, dtype=torch.bfloat16, device=DEV)
    q[..., :half] = 1
    plan = tam.tree_plan([-1], [N], device=DEV)
    pos = torch.tensor([ps], dtype=torch.int64).to(torch.int32).to(DEV)
    out, _ = tam.tree_rope_axes_fwd(plan, pos, q, q.clone(), (half,), theta=theta)
    out = out[:, 0].double().cpu().numpy()
    # turns of position and frequency, modulo one, in whole numbers: frequencies as fractions of 2^160
    getcontext().prec = 90
    th, pi = Decimal(float(np.float32(theta))), Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    turn = np.empty((N, half))
    for c in range(half):
        f = int((-th.ln() * c / half).exp() / (2 * pi) * 2 ** 160)
        turn[:, c] = [((p * f) % 2 ** 160) / 2 ** 160 for p in ps]
    ang = 2 * np.pi * turn
    for got, ref in ((out[:, :half], np.cos(ang)), (out[:, half:], np.sin(ang))):
        tol = 2.0 ** -8 * np.abs(ref) + 2 * np.pi * 2.0 ** -25 + 2.0 ** -23
        assert (np.abs(got - ref) <= tol).all()
