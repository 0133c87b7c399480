"""The gated linear recurrence against its fp64 oracle, forward and backward.

Tolerances: the oracle carries, next to every value, how many fp32 roundings of what magnitude reach it
(one unit a token, counted in units of 2^-24).  A token costs, forward: e = exp(-g) as 2^t, t = -g log2(e):
the constant (0.3 |g|) and the product (half a unit in the last place of t, 5.5 for |g| <= 11 after the
factor ln 2) and the power (2 ulp: 4); 1 - a = e a adds the reciprocal (2) and a product (1), less where e is
large, and e's own part of it is e's weight 1 / (1 + e) there and e / (1 + e) in a: together at most 15 of the
larger of the two; times x 1, the step 1, and where the sequence is cut into tiles their products and sums
(2 per joined map, 4 a tile of 128: below 1).  Backward: p's exponential carries what its argument lost
(2 ulp and 1), a reciprocal and a product (3), the step 2, once more for h, which is computed again: 16.  24
units cover both.  Results in bf16 add half a step, 2^-8 of the value; fp32 results 2^-24."""
import numpy as np
import pytest
import torch

import oracle
import tree_masked_attention_plan_gb300 as tam
from oracle import scan as osc
from workloads import caterpillar_tree, random_tree

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
UNITS = 24 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(N, n, C, kind, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    gate = 2 * r(N, C) + 2 if kind == "sigmoid" else -torch.exp(1.5 * r(N, C) - 2)
    return gate.to(dtype), r(N, C).to(dtype), r(n, C), r(N, C).to(dtype), r(n, C)


def _close(name, got, ref, err, dtype):
    got = _f64(got)
    tol = HALF[dtype] * np.abs(ref) + UNITS * err + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (name, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])


def run_gpu(parent, node_len, gate, x, kind, init, dy=None, d_final=None):
    plan = tam.tree_plan(parent, node_len, device=DEV)
    tree = tam.tree_arrays(parent, node_len, DEV)
    d = lambda t: None if t is None else t.to(DEV)
    status = tam.new_status(DEV)
    y, states = tam.tree_scan_fwd(plan, tree, d(gate), d(x), init=d(init), gate_kind=kind, status=status)
    out = dict(y=y, final=states[:len(node_len)])
    if dy is not None:
        out["dgate"], out["dx"], out["d_init"] = tam.tree_scan_bwd(
            plan, tree, d(gate), d(x), states, d(dy), init=d(init), d_final=d(d_final), gate_kind=kind, status=status)
    torch.cuda.synchronize()
    tam.check_status(status, "scan")
    return out


def check(parent, node_len, C, kind="sigmoid", dtype=torch.bfloat16, seed=0, ends=True, channels=None):
    node_len = np.asarray(node_len)
    N, n = int(node_len.sum()), len(node_len)
    gate, x, init, dy, dfin = _inputs(N, n, C, kind, dtype, seed)
    if not ends:
        init = dfin = None
    got = run_gpu(parent, node_len, gate, x, kind, init, dy, dfin)
    ch = np.arange(C) if channels is None else channels
    sub = lambda t: None if t is None else _f64(t)[:, ch]
    ref = osc.scan(parent, node_len, sub(gate), sub(x), kind, init=sub(init), dy=sub(dy), d_final=sub(dfin))
    for name, dt in (("y", dtype), ("final", torch.float32), ("dgate", dtype), ("dx", dtype), ("d_init", torch.float32)):
        if got[name] is not None:
            _close(name, got[name][:, ch], ref[name], ref["e_" + name], dt)
    return got


@pytest.mark.parametrize("kind", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("seed,n_nodes,max_len,C", [(0, 12, 90, 64), (1, 60, 40, 72), (2, 200, 6, 8), (3, 7, 700, 136)])
def test_random_trees(kind, dtype, seed, n_nodes, max_len, C):
    parent, node_len = random_tree(400 + seed, n_nodes, max_len=max_len, zero_prob=0.15, n_roots=1 + seed % 3)
    check(parent, node_len, C, kind, dtype, seed, ends=seed % 2 == 0)


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 1500, 6000])
def test_one_sequence(n):
    check([-1], [n], 40, "log" if n % 2 else "sigmoid", torch.float32 if n % 3 == 0 else torch.bfloat16, n)


@pytest.mark.parametrize("n", [1, 5, 64, 300])
def test_one_step_of_many_sequences(n):
    check([-1] * n, [1] * n, 264, "sigmoid", torch.bfloat16, n)


def test_caterpillar():
    parent, node_len = caterpillar_tree()
    check(parent, node_len, 64, "sigmoid", torch.bfloat16, 5)


def test_many_children_of_one_node_and_ends_at_tile_edges():
    """A prompt of exactly two tiles with 70 answers, some exactly a tile long, most of them short."""
    rng = np.random.default_rng(0)
    lens = [256] + [int(v) for v in rng.choice([1, 2, 30, 128, 129], 70)]
    check([-1] + [0] * 70, lens, 72, "log", torch.float32, 9)


def test_star_of_single_tokens_in_one_tile():
    check([-1] + [0] * 100, [1] * 101, 16, "sigmoid", torch.float32, 10)


def test_children_in_the_tile_of_their_parent_and_far_behind_it():
    """Siblings whose subtrees span many tiles, with short nodes on both sides of the edges."""
    parent = [-1, 0, 1, 1, 0, 4, 4, 0]
    check(parent, [100, 20, 700, 3, 5, 900, 129, 1], 64, "sigmoid", torch.bfloat16, 11)


def test_chain_of_single_tokens_through_empty_nodes():
    n = 400
    check(np.arange(-1, n - 1), np.where(np.arange(n) % 3 == 1, 0, 1), 8, "log", torch.float32, 12)


def test_wide_layer_on_sampled_channels():
    parent, node_len = random_tree(420, 40, max_len=300, n_roots=2)
    check(parent, node_len, 4104, "sigmoid", torch.bfloat16, 13, channels=np.r_[0:4, 2040:2056, 4096:4104])


@pytest.mark.parametrize("kind", ["sigmoid", "log"])
def test_gates_at_their_ends(kind):
    """Decays of exactly zero and one, and gates that no decay below one belongs to."""
    N, C = 700, 8
    gate, x, init, dy, dfin = _inputs(N, 2, C, kind, torch.float32, 3)
    inf = float("inf")
    gate[::7] = -inf
    gate[3::11] = 100.0 if kind == "sigmoid" else 0.0
    gate[5::13] = -100.0
    gate[6::17] = inf if kind == "sigmoid" else 5.0
    gate[8::19] = 0.0
    got = run_gpu([-1, 0], [650, 50], gate, x, kind, init, dy, dfin)
    ref = osc.scan([-1, 0], [650, 50], _f64(gate), _f64(x), kind, init=_f64(init), dy=_f64(dy), d_final=_f64(dfin))
    for name in ("y", "final", "dgate", "dx", "d_init"):
        _close(name, got[name], ref[name], ref["e_" + name], torch.float32)


def test_what_is_not_a_number_stays_on_its_paths():
    """A NaN and an infinity in one branch reach its tokens, and going back its ancestors' gradients; not the other branches."""
    parent, lens = [-1, 0, 0, 2, -1], [150, 200, 60, 300, 90]
    N, C = sum(lens), 8
    gate, x, init, dy, dfin = _inputs(N, 5, C, "sigmoid", torch.float32, 4)
    clean = run_gpu(parent, lens, gate, x, "sigmoid", init, dy, dfin)
    bad_x, bad_dy = x.clone(), dy.clone()
    bad_x[160, 0] = float("nan")
    bad_x[200, 1] = float("inf")
    bad_dy[300, 2] = float("nan")
    got = run_gpu(parent, lens, gate, bad_x, "sigmoid", init, bad_dy, dfin)
    y, c = got["y"].cpu(), clean["y"].cpu()
    assert not torch.isfinite(y[160:350, 0]).any() and not torch.isfinite(y[200:350, 1]).any()
    y[160:350, 0] = c[160:350, 0]
    y[200:350, 1] = c[200:350, 1]
    assert torch.equal(y, c)
    dx, c = got["dx"].cpu(), clean["dx"].cpu()
    assert not torch.isfinite(dx[:301, 2]).any()
    dx[:301, 2] = c[:301, 2]
    assert torch.equal(dx, c)
    assert torch.equal(got["final"][2:].cpu(), clean["final"][2:].cpu())


def test_the_same_bits_every_time_on_another_stream_and_from_a_graph():
    parent, node_len = random_tree(430, 50, max_len=200, n_roots=2)
    N, n, C = int(node_len.sum()), 50, 520
    gate, x, init, dy, dfin = (t.to(DEV) for t in _inputs(N, n, C, "log", torch.bfloat16, 6))
    plan, tree = tam.tree_plan(parent, node_len, device=DEV), tam.tree_arrays(parent, node_len, DEV)
    ws = torch.empty(tam.tree_scan_workspace(plan, C), dtype=torch.uint8, device=DEV)

    def call(ws, stream=None):
        y, st = tam.tree_scan_fwd(plan, tree, gate, x, init=init, gate_kind="log", workspace=ws, stream=stream)
        return (y, st) + tam.tree_scan_bwd(plan, tree, gate, x, st, dy, init=init, d_final=dfin, gate_kind="log",
                                           workspace=ws, stream=stream)

    first = call(ws)
    torch.cuda.synchronize()
    ws.fill_(0xA5)                                     # the workspace holds nothing between calls
    for _ in range(3):
        for a, b in zip(first, call(ws)):
            assert torch.equal(a, b)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    other = call(None, side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call(ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, captured):
        assert torch.equal(a, b)
    keep = x.clone()
    x.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(first[0], captured[0])
    x.copy_(keep)


def test_states_continue_across_a_cut():
    """A child partition that starts from its gateway's final state gives the whole tree's rows, and its d_init is what the
    parent partition needs as d_final."""
    parent, lens = [-1, 0, 1, 0], [200, 150, 90, 70]
    N, C = sum(lens), 64
    gate, x, _, dy, _ = _inputs(N, 4, C, "sigmoid", torch.float32, 8)
    whole = run_gpu(parent, lens, gate, x, "sigmoid", None, dy)
    cut = slice(200, 440)                              # nodes 1 and 2
    top = np.r_[0:200, 440:510]
    up = run_gpu([-1, 0], [200, 70], gate[top], x[top], "sigmoid", None)
    init = torch.zeros(2, C)
    init[0] = up["final"][0].cpu()
    low = run_gpu([-1, 0], [150, 90], gate[cut], x[cut], "sigmoid", init, dy[cut])
    d_final = torch.zeros(2, C)
    d_final[0] = low["d_init"][0].cpu()
    up = run_gpu([-1, 0], [200, 70], gate[top], x[top], "sigmoid", None, dy[top], d_final)
    ref = osc.scan(parent, lens, _f64(gate), _f64(x), "sigmoid", dy=_f64(dy))
    for name in ("y", "dgate", "dx"):
        for part, rows in ((low, cut), (up, top)):
            _close(name, part[name], ref[name][rows], ref["e_" + name][rows], torch.float32)
    del whole


def test_guards_around_every_buffer():
    """Nothing is written outside the outputs and the workspace: canaries on both sides stay."""
    parent, node_len = random_tree(440, 30, max_len=50, zero_prob=0.2, n_roots=2)
    N, n, C = int(node_len.sum()), 30, 72
    gate, x, init, dy, dfin = (t.to(DEV) for t in _inputs(N, n, C, "sigmoid", torch.bfloat16, 7))
    plan, tree = tam.tree_plan(parent, node_len, device=DEV), tam.tree_arrays(parent, node_len, DEV)
    raws = []

    def guarded(shape, dtype):
        b = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
        raw = torch.full((8192 + b,), 0xA5, dtype=torch.uint8, device=DEV)
        raws.append((raw, b))
        return raw[4096:4096 + b].view(dtype).view(*shape)

    ws = guarded((tam.tree_scan_workspace(plan, C),), torch.uint8)
    y, st = guarded((N, C), torch.bfloat16), guarded((tam.tree_scan_rows(plan), C), torch.float32)
    dg, dx, di = guarded((N, C), torch.bfloat16), guarded((N, C), torch.bfloat16), guarded((n, C), torch.float32)
    tam.tree_scan_fwd(plan, tree, gate, x, init=init, workspace=ws, y=y, states=st)
    tam.tree_scan_bwd(plan, tree, gate, x, st, dy, init=init, d_final=dfin, workspace=ws, dgate=dg, dx=dx, d_init=di)
    torch.cuda.synchronize()
    for raw, b in raws:
        assert bool((raw[:4096] == 0xA5).all()) and bool((raw[4096 + b:] == 0xA5).all())
    for t in (st, di):
        assert torch.isfinite(t).all() and t.abs().max() < 1e3


@pytest.mark.parametrize("kind,dtype", [("sigmoid", torch.bfloat16), ("log", torch.float32)])
@pytest.mark.parametrize("seed,n_nodes,max_len,zero,C", [(0, 5, 40, 0, 8), (1, 20, 6, 0.2, 72), (2, 60, 2, 0.3, 136),
                                                         (3, 128, 1, 0, 40), (4, 700, 1, 0.9, 64)])
def test_few_tokens(kind, dtype, seed, n_nodes, max_len, zero, C):
    """At most 128 tokens: chains, paths that part within a few tokens, many trees, many nodes without tokens."""
    parent, node_len = random_tree(450 + seed, n_nodes, max_len=max_len, zero_prob=zero, n_roots=1 + 3 * seed)
    assert 1 <= node_len.sum() <= 128
    check(parent, node_len, C, kind, dtype, seed, ends=seed % 2 == 1)


def test_few_and_many_tokens_agree():
    """A sequence of 128 tokens and the first 128 of a longer one; the states row between tiles is the state there."""
    C = 64
    gate, x, _, _, _ = _inputs(300, 1, C, "sigmoid", torch.float32, 14)
    d = lambda t: t.to(DEV)
    res = []
    for n in (128, 300):
        plan, tree = tam.tree_plan([-1], [n], device=DEV), tam.tree_arrays([-1], [n], DEV)
        res.append(tam.tree_scan_fwd(plan, tree, d(gate[:n].contiguous()), d(x[:n].contiguous())))
    ref = osc.scan([-1], [128], _f64(gate[:128]), _f64(x[:128]), "sigmoid")
    for y, _ in res:
        _close("y", y[:128], ref["y"], ref["e_y"], torch.float32)
    assert torch.equal(res[0][1][1], res[0][1][0]) and torch.equal(res[0][1][0], res[0][0][127])
    _close("between", res[1][1][1:2], ref["y"][127:], ref["e_y"][127:], torch.float32)


def test_many_calls_of_a_tree_of_short_nodes():
    """Many slabs of tiles full of breaks, again and again: every wait ends and no bit changes."""
    parent, node_len = random_tree(460, 300, max_len=30, zero_prob=0.1, n_roots=9)
    N, n, C = int(node_len.sum()), 300, 1000
    gate, x, init, dy, dfin = (t.to(DEV) for t in _inputs(N, n, C, "log", torch.float32, 15))
    plan, tree = tam.tree_plan(parent, node_len, device=DEV), tam.tree_arrays(parent, node_len, DEV)
    ws = torch.empty(tam.tree_scan_workspace(plan, C), dtype=torch.uint8, device=DEV)
    status = tam.new_status(DEV)
    first = None
    for i in range(60):
        y, st = tam.tree_scan_fwd(plan, tree, gate, x, init=init, gate_kind="log", workspace=ws, status=status)
        now = (y, st) + tam.tree_scan_bwd(plan, tree, gate, x, st, dy, init=init, d_final=dfin, gate_kind="log",
                                          workspace=ws, status=status)
        first = first or now
        if i % 20 == 19:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
    torch.cuda.synchronize()
    tam.check_status(status, "scan")


def test_two_streams_at_once_and_two_graphs_of_one_workspace():
    parent, node_len = random_tree(470, 60, max_len=150, n_roots=2)
    N, n, C = int(node_len.sum()), 60, 2056
    plan, tree = tam.tree_plan(parent, node_len, device=DEV), tam.tree_arrays(parent, node_len, DEV)
    ins = [[t.to(DEV) for t in _inputs(N, n, C, "sigmoid", torch.bfloat16, 16 + i)] for i in range(2)]
    status = tam.new_status(DEV)

    def call(i, ws, stream=None):
        gate, x, init, dy, dfin = ins[i]
        y, st = tam.tree_scan_fwd(plan, tree, gate, x, init=init, workspace=ws, status=status, stream=stream)
        return (y, st) + tam.tree_scan_bwd(plan, tree, gate, x, st, dy, init=init, d_final=dfin, workspace=ws,
                                           status=status, stream=stream)

    own = [torch.empty(tam.tree_scan_workspace(plan, C), dtype=torch.uint8, device=DEV) for _ in range(2)]
    alone = [call(i, own[i]) for i in range(2)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(DEV) for _ in range(2)]
    both = [[call(i, own[i], side[i]) for i in range(2)] for _ in range(4)]      # blocks of both calls share the GPU
    torch.cuda.synchronize()
    for pair in both:
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(alone[i], pair[i]))
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], [None, None]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            got[i] = call(i, own[0])
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(alone[i], got[i]))
    tam.check_status(status, "scan")


def test_offsets_beyond_32_bits():
    """More than 2^32 elements: the last channels of a sequence whose every tensor is 8.6 GB."""
    N, C = 131072, 32776
    free, _ = torch.cuda.mem_get_info(DEV)
    if free < 100e9:
        pytest.skip("needs 100 GB of device memory")
    plan, tree = tam.tree_plan([-1], [N], device=DEV), tam.tree_arrays([-1], [N], DEV)
    ch = np.r_[0:2, C - 4:C]
    # the same six channels' values everywhere but at the sampled ones, which are their own
    gate, x, _, dy, _ = _inputs(N, 1, len(ch), "sigmoid", torch.bfloat16, 17)

    def wide(t):
        w = torch.zeros(N, C, dtype=t.dtype, device=DEV)
        w[:, torch.as_tensor(ch, device=DEV)] = t.to(DEV)
        return w

    g, v, d = wide(gate), wide(x), wide(dy)
    y, st = tam.tree_scan_fwd(plan, tree, g, v)
    dg, dx, _ = tam.tree_scan_bwd(plan, tree, g, v, st, d)
    ref = osc.scan([-1], [N], _f64(gate), _f64(x), "sigmoid", dy=_f64(dy))
    idx = torch.as_tensor(ch, device=DEV)
    for name, got in (("y", y), ("dgate", dg), ("dx", dx)):
        _close(name, got[:, idx], ref[name], ref["e_" + name], torch.bfloat16)
    _close("final", st[:1, idx], ref["final"], ref["e_final"], torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_nodes,max_len", [(20, 6), (50, 60)])
def test_outputs_in_the_place_of_inputs(dtype, n_nodes, max_len):
    """y in x, then dgate in gate and dx in dy, as a whole: the same bits as in buffers of their own."""
    parent, node_len = random_tree(480 + n_nodes, n_nodes, max_len=max_len, n_roots=2)
    N, C = int(node_len.sum()), 200
    gate, x, init, dy, dfin = (t.to(DEV) for t in _inputs(N, n_nodes, C, "sigmoid", dtype, 18))
    plan, tree = tam.tree_plan(parent, node_len, device=DEV), tam.tree_arrays(parent, node_len, DEV)
    y, st = tam.tree_scan_fwd(plan, tree, gate, x, init=init)
    dg, dx, di = tam.tree_scan_bwd(plan, tree, gate, x, st, dy, init=init, d_final=dfin)
    for keep in (x.clone(), gate.clone()):
        other = gate if torch.equal(keep, x) else x
        y2, st2 = (tam.tree_scan_fwd(plan, tree, other, keep, init=init, y=keep) if other is gate
                   else tam.tree_scan_fwd(plan, tree, keep, other, init=init, y=keep))
        assert torch.equal(y, y2) and torch.equal(st, st2)
    g2, d2 = gate.clone(), dy.clone()
    _, _, di2 = tam.tree_scan_bwd(plan, tree, g2, x, st, d2, init=init, d_final=dfin, dgate=g2, dx=d2)
    assert torch.equal(dg, g2) and torch.equal(dx, d2) and torch.equal(di, di2)
    with pytest.raises(tam.TreeError):
        tam.tree_scan_fwd(plan, tree, gate, x, init=st[:n_nodes], states=st)


@pytest.mark.parametrize("kind,dtype", [("sigmoid", torch.float32), ("log", torch.bfloat16)])
@pytest.mark.parametrize("parent,lens", [
    ([-1, 0, 0, 2], [100, 60, 40, 56]),                # 256 tokens, a path across the tile's edge
    ([-1, 0], [128, 128]), ([-1, -1], [128, 100]),     # it goes on there, and it does not
    ([-1] * 200, [1] * 200), ([-1, 0, 1, 0], [127, 0, 1, 1]),
    ([-1] + [0] * 99, [30] + [1] * 99)], ids=range(6))
def test_two_tiles_of_tokens(kind, dtype, parent, lens):
    """The states row between the two, which the backward starts from."""
    check(parent, lens, 72, kind, dtype, 21, ends=len(lens) % 2 == 0)


@pytest.mark.parametrize("kind,dtype", [("sigmoid", torch.bfloat16), ("log", torch.float32)])
@pytest.mark.parametrize("lens", [[1] * 700, [0, 2] * 200, [0] * 450 + [150, 300] + [1] * 200, [1] * 127 + [0] * 400 + [300]],
                         ids=range(4))
def test_a_step_of_many_sequences(kind, dtype, lens):
    """Nodes that are sequences of their own, no more tokens than nodes: most have one token, some go across tiles."""
    assert 256 < sum(lens) <= len(lens)
    check([-1] * len(lens), lens, 136, kind, dtype, 22, ends=len(lens) != 700 or kind == "log")
