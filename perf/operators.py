"""The operators that a training step of a hybrid (attention + recurrence) layer on a packed prefix tree uses around
attention, as cases to be measured: the gated linear recurrence along root paths (forward, and forward with its backward),
rotary positions with several axes (forward and backward), and the global gradient norm with clipping.

`run` computes a case in its plain form, out of elementary torch operations, or with `own` set by the library's calls.
`exact` gives the same from the definition in 64 bits."""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of 64 sequences: one-token trees that start from given states; latency is all of it
        dict(name="scan step 64x4096", op="scan", tree="steps", tokens=64, tree_seed=0, channels=4096, dtype="bf16",
             gate="sigmoid", init=True, train=False),
        # a vision-language-action episode: a trunk with a short action leaf at every step, inference
        dict(name="scan caterpillar 3456x4096", op="scan", tree="caterpillar", tokens=3456, tree_seed=0, channels=4096,
             dtype="bf16", gate="sigmoid", init=False, train=False),
        # a packed rollout tree through a wide hybrid layer, forward only (log-probabilities of rollouts)
        dict(name="scan rollout 32768x8192", op="scan", tree="rollout", tokens=32768, tree_seed=0, channels=8192,
             dtype="bf16", gate="sigmoid", init=False, train=False),
        # one long sequence through a narrow layer: all of the parallelism is along the sequence
        dict(name="scan chain 131072x2048", op="scan", tree="chain", tokens=131072, tree_seed=0, channels=2048,
             dtype="bf16", gate="log", init=False, train=False),
        # the training step of the rollout tree
        dict(name="scan train rollout 32768x8192", op="scan", tree="rollout", tokens=32768, tree_seed=0, channels=8192,
             dtype="bf16", gate="sigmoid", init=False, train=True),
        # ragged: several roots, empty nodes, short nodes, an odd token count, a partial channel slab, 32-bit values,
        # the roots' states given and their gradients wanted (a partition below a cut)
        dict(name="scan train forest 20011x1000", op="scan", tree="forest", tokens=20011, tree_seed=1, channels=1000,
             dtype="fp32", gate="log", init=True, train=True),
        # positions of a few new tokens: latency
        dict(name="rope axes 48 tokens", op="rope", tokens=48, hq=32, hkv=8, d=128, sections="16,24,24",
             interleaved=False, backward=False, start=70000),
        # queries and keys of the packed rollout tree with image patches in it
        dict(name="rope axes 32768 tokens", op="rope", tokens=32768, hq=32, hkv=8, d=128, sections="16,24,24",
             interleaved=False, backward=False, start=0),
        # its gradients back through the rotation: small heads, axes interleaved over the frequencies, an odd length
        dict(name="rope axes backward 9973 tokens", op="rope", tokens=9973, hq=16, hkv=16, d=64, sections="12,10,10",
             interleaved=True, backward=True, start=0),
        # the norm of a whole model's small gradients (norm weights, biases, taps): many tensors, little data
        dict(name="grad norm 291 tensors", op="norm", tensors=291, elements=2000003, dtype="mixed", tensor_seed=0),
        # a layer's gradients, clipped into the flat buffer that an optimizer reads
        dict(name="grad clip 12 tensors 218M bf16", op="clip", tensors=12, elements=218112003, dtype="bf16",
             tensor_seed=1, factor=0.3),
        # with the 32-bit gradient of a 128256 x 4096 vocabulary matrix
        dict(name="grad clip 5 tensors 528M fp32", op="clip", tensors=5, elements=528482304, dtype="fp32",
             tensor_seed=2, factor=0.7),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], uniform over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "rope", "norm", "clip"])
    if op == "scan":
        channels = 8 * _between(rng, 1, 1024)
        tokens = _between(rng, 1, min(131072, (32768 * 8192) // channels))
        tree = rng.choice(["steps", "caterpillar", "rollout", "chain", "forest"])
        if tree == "steps":
            tokens = min(tokens, 4096)
        return dict(op="scan", tree=tree, tokens=tokens, tree_seed=rng.randrange(1000), channels=channels,
                    dtype=rng.choice(["bf16", "fp32"]), gate=rng.choice(["sigmoid", "log"]), init=rng.random() < 0.5,
                    train=rng.random() < 0.5)
    if op == "rope":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 16])
        hq = hkv * rng.choice([1, 2, 4])
        tokens = _between(rng, 1, min(131072, (32768 * 40 * 128) // ((hq + hkv) * d)))
        a = rng.randrange(1, d // 6)
        sections = rng.choice([(d // 2 - 2 * a, a, a), (d // 2 - a, a), (d // 2,)])
        return dict(op="rope", tokens=tokens, hq=hq, hkv=hkv, d=d, sections=",".join(str(s) for s in sections),
                    interleaved=rng.random() < 0.5, backward=rng.random() < 0.5,
                    start=rng.choice([0, rng.randrange(1000000)]))
    tensors = _between(rng, 1, 300)
    elements = max(tensors, _between(rng, 100, 200000000))
    case = dict(op=op, tensors=tensors, elements=elements, dtype=rng.choice(["bf16", "fp32", "mixed"]),
                tensor_seed=rng.randrange(1000))
    return dict(case, factor=rng.choice([0.1, 0.6, 2.0])) if op == "clip" else case


# ------------------------------------------------------------------------------------------------------ trees

def _tree(case):
    """parent and node_len of a case's tree; every parent has a smaller id than its children."""
    n, r = case["tokens"], np.random.RandomState(case["tree_seed"])
    kind = case["tree"]
    if kind == "chain":
        return [-1], [n]
    if kind == "steps":
        return [-1] * n, [1] * n
    parent, lens, left = [-1], [], n
    if kind == "caterpillar":
        lens.append(min(left, 256))
        left -= lens[0]
        trunk = 0
        while left > 0:
            parent.append(trunk)
            lens.append(min(left, 64))
            left -= lens[-1]
            trunk = len(lens) - 1
            if left > 0:
                parent.append(trunk)
                lens.append(min(left, 16))
                left -= lens[-1]
        return parent, lens
    forest = kind == "forest"
    depth = [0]
    lens.append(min(left, max(1, n // 16)))
    left -= lens[0]
    while left > 0:
        p = -1 if forest and r.rand() < 0.08 else int(r.randint(max(0, len(lens) - 24), len(lens)))
        if p >= 0 and depth[p] >= 8:
            p = 0
        size = 0 if forest and r.rand() < 0.1 else int(np.clip((40 if forest else 256) * math.exp(0.8 * r.randn()), 1, 4096))
        if len(lens) > 3000:
            size = left
        parent.append(p)
        depth.append(0 if p < 0 else depth[p] + 1)
        lens.append(min(left, size))
        left -= lens[-1]
    return parent, lens


def _pack(parent, lens):
    """The depth-first packing (children by ascending id): per token, the token before it on its root path (-1 before a
    root) and its depth; per node, its last token (-1: it has none); the nodes that start from nothing, each with its first
    token."""
    m = len(parent)
    kids = [[] for _ in range(m)]
    roots = []
    for v in range(m):
        (roots if parent[v] < 0 else kids[parent[v]]).append(v)
    prev = np.arange(-1, sum(lens) - 1)
    depth = np.zeros(sum(lens), np.int64)
    last, state, base, starts, at = [-1] * m, [-1] * m, [0] * m, [], 0
    stack = roots[::-1]
    while stack:
        v = stack.pop()
        above = state[parent[v]] if parent[v] >= 0 else -1
        base[v] = base[parent[v]] + lens[parent[v]] if parent[v] >= 0 else 0
        state[v] = above
        if lens[v]:
            prev[at] = above
            if above < 0:
                starts.append((v, at))
            depth[at:at + lens[v]] = base[v] + np.arange(lens[v])
            at += lens[v]
            last[v] = state[v] = at - 1
        stack.extend(kids[v][::-1])
    return prev, depth, np.array(last), starts


def _tensor_sizes(case):
    """Element counts of a case's gradients: shares of the whole, odd ones among them."""
    r = np.random.RandomState(case["tensor_seed"])
    n, k = case["elements"], case["tensors"]
    share = np.exp(1.2 * r.randn(k)) if k > 5 else np.array([300.0, 2, 1, 1, 1][:k])
    sizes = np.maximum(1, (share / share.sum() * (n - k)).astype(np.int64))
    sizes[0] += n - sizes.sum()
    kinds = [case["dtype"] if case["dtype"] != "mixed" else ("bf16", "fp32")[int(r.randint(2))] for _ in range(k)]
    return [int(s) for s in sizes], kinds


DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------ states

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    if case["op"] == "scan":
        n, c, dt = case["tokens"], case["channels"], DTYPES[case["dtype"]]
        parent, lens = _tree(case)
        prev, depth, last, starts = _pack(parent, lens)
        s = dict(case=case, n=n, last=torch.from_numpy(last).to(dev))
        s["root_nodes"] = torch.tensor([v for v, _ in starts], device=dev)
        s["root_tokens"] = torch.tensor([t for _, t in starts], device=dev)
        # memories from a few tokens to thousands of them, as trained gates have
        s["gate"] = (1.5 * normal(n, c) + 3.0).to(dt) if case["gate"] == "sigmoid" else (-torch.exp(1.5 * normal(n, c) - 3.0)).to(dt)
        s["x"] = normal(n, c, dtype=dt)
        if case["init"]:
            s["init"] = normal(len(parent), c)
        if case["train"]:
            s["dy"] = normal(n, c, dtype=dt)
            if case["init"]:
                s["d_final"] = normal(len(parent), c)
        if own:
            import tree_masked_attention_plan_gb300 as tam
            s["tam"], s["plan"], s["tree"] = tam, tam.tree_plan(parent, lens, device=dev), tam.tree_arrays(parent, lens, dev)
            s["workspace"] = torch.empty(tam.tree_scan_workspace(s["plan"], c), dtype=torch.uint8, device=dev)
        else:  # the index plan of the plain form: round r adds what lies 2^r tokens further up
            at = torch.from_numpy(np.append(np.where(prev < 0, n, prev), n)).to(dev)
            s["jumps"] = []
            for _ in range(int(depth.max()).bit_length()):
                s["jumps"].append(at)
                at = at[at]
        return s
    if case["op"] == "rope":
        n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        sections = [int(v) for v in case["sections"].split(",")]
        s = dict(case=case, sections=sections, q=normal(n, hq, d, dtype=torch.bfloat16), k=normal(n, hkv, d, dtype=torch.bfloat16))
        # text and 16 x 16 image patches in turn; an image's patches share a time and differ in height and width
        t = torch.arange(n, device=dev)
        start = case["start"] + int(torch.randint(0, 100, (1,), generator=gen, device=dev))
        block, within = t // 256, t % 256
        image = block % 2 == 1
        base = start + (block // 2) * (256 + 16) + torch.where(image, 256, 0)
        axes = [torch.where(image, base, base + within), torch.where(image, base + within // 16, base + within),
                torch.where(image, base + within % 16, base + within)]
        s["pos"] = torch.stack(axes[:len(sections)]).to(torch.int32).contiguous()
        if own:
            import tree_masked_attention_plan_gb300 as tam
            s["tam"], s["plan"] = tam, tam.tree_plan([-1], [n], device=dev)
        return s
    sizes, kinds = _tensor_sizes(case)
    s = dict(case=case, grads=[normal(k, dtype=DTYPES[t]).mul_(0.01) for k, t in zip(sizes, kinds)])
    if case["op"] == "clip":
        s["max_norm"] = case["factor"] * 0.01 * math.sqrt(case["elements"])
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        if len(sizes) > 48:  # views of one flat buffer for each type
            s["flat"] = {t: torch.empty(sum(-(-k // 8) * 8 for k, u in zip(sizes, kinds) if u == t), dtype=DTYPES[t], device=dev).zero_() for t in sorted(set(kinds))}
            at = dict.fromkeys(s["flat"], 0)
            s["out"] = []
            for k, t in zip(sizes, kinds):
                s["out"].append(s["flat"][t][at[t]:at[t] + k])
                at[t] += -(-k // 8) * 8
    if own:
        import tree_masked_attention_plan_gb300 as tam
        s["tam"] = tam
        s["list"] = tam.tree_grad_list(s["grads"], out=s.get("out"))
    return s


# ------------------------------------------------------------------------------------------------------ plain forms

def _decay(s):
    """The decay a, what it lacks to one (accurate where a is close to one), and the weight of the input."""
    g = s["gate"].float()
    if s["case"]["gate"] == "sigmoid":
        lack = 1.0 / (1.0 + torch.exp(g))
        return 1.0 / (1.0 + torch.exp(-g)), lack, lack
    lack = -torch.special.expm1(torch.clamp(g, max=0.0))
    return 1.0 - lack, lack, None


def _plain_scan(s):
    case, n = s["case"], s["n"]
    x = s["x"].float()
    a, lack, weight = _decay(s)
    one = torch.zeros(1, x.shape[1], device=x.device)
    b = torch.cat([x if weight is None else weight * x, one])
    if case["init"]:
        b[s["root_tokens"]] += a[s["root_tokens"]] * s["init"][s["root_nodes"]]
    A, factors = torch.cat([a, one]), []
    for at in s["jumps"]:
        factors.append(A)
        b = b + A * b[at]
        A = A * A[at]
    h = b[:n]
    final = torch.cat([h, one])[s["last"]]  # zeros for nodes without tokens: -1 is the row of zeros
    out = dict(y=h.to(s["x"].dtype), final=final)
    if not case["train"]:
        return out
    lam = torch.cat([s["dy"].float(), one])
    if case["init"]:
        lam.index_add_(0, torch.where(s["last"] < 0, n, s["last"]), s["d_final"])
        lam[n] = 0
    for at, A in zip(s["jumps"][::-1], factors[::-1]):
        lam = lam.index_add(0, at, A * lam)
        lam[n] = 0
    lam = lam[:n]
    before = b[s["jumps"][0][:n]] if s["jumps"] else torch.zeros_like(h)
    if case["init"]:
        before[s["root_tokens"]] = s["init"][s["root_nodes"]]
        d_init = torch.zeros_like(s["init"])
        d_init[s["root_nodes"]] = a[s["root_tokens"]] * lam[s["root_tokens"]]
        out["d_init"] = d_init
    if weight is None:
        dgate, dx = lam * before * a * (s["gate"] <= 0), lam
    else:
        dgate, dx = lam * (before - x) * a * lack, lam * lack
    return dict(out, dgate=dgate.to(s["x"].dtype), dx=dx.to(s["x"].dtype))


def _axis_of(sections, interleaved, half):
    """The axis of each frequency: in runs, or dealt in turn (axis i takes i, i + n, ... until it has its share; what is
    left goes to the first)."""
    if not interleaved:
        return [i for i, k in enumerate(sections) for _ in range(k)]
    axis, m = [0] * half, len(sections)
    for i in range(1, m):
        for j in range(sections[i]):
            axis[i + m * j] = i
    return axis


def _angles(s):
    half = s["case"]["d"] // 2
    axis = torch.tensor(_axis_of(s["sections"], s["case"]["interleaved"], half), device=s["pos"].device)
    freq = 10000.0 ** (-torch.arange(half, device=axis.device, dtype=torch.float64) / half)
    angle = s["pos"][axis].t().to(torch.float64) * freq  # 64 bits: far positions
    return -angle if s["case"]["backward"] else angle


def _plain_rope(s):
    angle = _angles(s)[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    half, out = s["case"]["d"] // 2, []
    for v in (s["q"], s["k"]):
        x, y = v[..., :half].float(), v[..., half:].float()
        out.append(torch.cat([x * cos - y * sin, y * cos + x * sin], -1).to(v.dtype))
    return out


def _plain_norm(s):
    """The norm over all tensors; sums of squares in 64 bits, in pieces that fit."""
    total = torch.zeros((), dtype=torch.float64, device=s["grads"][0].device)
    for g in s["grads"]:
        for p in g.split(1 << 26):
            v = p.double()
            total = total + (v * v).sum()
    return torch.sqrt(total)


def _plain_clip(s):
    norm = _plain_norm(s)
    scale = torch.where((norm > s["max_norm"]) & torch.isfinite(norm), s["max_norm"] / norm, 1.0).float()
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * scale)
    return norm.float().reshape(1), s.get("flat") or s["out"]


def run(s):
    case = s["case"]
    if case["op"] == "scan":
        if not own:
            return _plain_scan(s)
        tam, plan, tree = s["tam"], s["plan"], s["tree"]
        y, states = tam.tree_scan_fwd(plan, tree, s["gate"], s["x"], init=s.get("init"), gate_kind=case["gate"],
                                      workspace=s["workspace"])
        out = dict(y=y, final=states[:plan.info.n_nodes])
        if case["train"]:
            out["dgate"], out["dx"], d_init = tam.tree_scan_bwd(
                plan, tree, s["gate"], s["x"], states, s["dy"], init=s.get("init"), d_final=s.get("d_final"),
                gate_kind=case["gate"], workspace=s["workspace"])
            if case["init"]:
                out["d_init"] = d_init
        return out
    if case["op"] == "rope":
        if not own:
            return _plain_rope(s)
        call = s["tam"].tree_rope_axes_bwd if case["backward"] else s["tam"].tree_rope_axes_fwd
        return list(call(s["plan"], s["pos"], s["q"], s["k"], s["sections"], theta=10000.0, interleaved=case["interleaved"]))
    if case["op"] == "norm":
        return s["tam"].tree_grad_norm(s["list"]) if own else _plain_norm(s).float().reshape(1)
    if not own:
        return _plain_clip(s)
    return s["tam"].tree_grad_clip(s["list"], s["max_norm"]), s.get("flat") or s["out"]


# ------------------------------------------------------------------------------------------------------ work

def work(case):
    if case["op"] == "scan":
        per = 2 if case["dtype"] == "bf16" else 4
        elements, states = case["tokens"] * case["channels"], len(_tree(case)[0]) * case["channels"] * 4
        states *= 1 + case["init"] + 2 * (case["init"] and case["train"])
        return {"bytes": elements * per * (6 if case["train"] else 3) + states, "flops": elements * (24 if case["train"] else 8)}
    if case["op"] == "rope":
        elements = case["tokens"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": 4 * elements + 4 * case["tokens"] * len(case["sections"].split(",")), "flops": 3 * elements}
    sizes, kinds = _tensor_sizes(case)
    read = sum(k * (2 if t == "bf16" else 4) for k, t in zip(sizes, kinds))
    return {"bytes": read * (2 if case["op"] == "clip" else 1) + 4, "flops": (3 if case["op"] == "clip" else 2) * sum(sizes)}


# ------------------------------------------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "scan":
        return _exact_scan(s)
    if case["op"] == "rope":
        return _exact_rope(s)
    squares = [float(sum((p.double() ** 2).sum().item() for p in g.split(1 << 24))) for g in s["grads"]]
    norm = math.sqrt(math.fsum(squares))
    if case["op"] == "norm":
        return torch.tensor([norm], dtype=torch.float64)
    scale = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
    if "flat" not in s:
        return torch.tensor([norm], dtype=torch.float64), [g.double() * scale for g in s["grads"]]
    flat = {t: torch.zeros(f.shape, dtype=torch.float64, device=f.device) for t, f in s["flat"].items()}
    for g, o in zip(s["grads"], s["out"]):
        f = flat["bf16" if g.dtype == torch.bfloat16 else "fp32"]
        at = o.storage_offset()
        f[at:at + o.numel()] = g.double() * scale
    return torch.tensor([norm], dtype=torch.float64), flat


def _exact_rope(s):
    case, half = s["case"], s["case"]["d"] // 2
    pos, axis = s["pos"].cpu().numpy().astype(np.float64), _axis_of(s["sections"], case["interleaved"], half)
    angle = np.stack([pos[axis[c]] * math.exp(-math.log(10000.0) * c / half) for c in range(half)], 1)
    turn = np.exp((-1j if case["backward"] else 1j) * angle)[:, None, :]
    out = []
    for v in (s["q"], s["k"]):
        w = torch.from_numpy(np.ascontiguousarray(turn)).to(v.device)
        z = torch.complex(v[..., :half].double(), v[..., half:].double()) * w
        out.append(torch.cat([z.real, z.imag], -1))
    return out


def _exact_scan(s):
    """The recurrence token by token in 64 bits: all tokens at one distance from their roots at a time."""
    case, n = s["case"], s["n"]
    parent, lens = _tree(case)
    prev, depth, last, starts = _pack(parent, lens)
    dev = s["x"].device
    x, g = s["x"].double(), s["gate"].double()
    if case["gate"] == "sigmoid":
        a, b = torch.sigmoid(g), torch.sigmoid(-g) * x
    else:
        a, b = torch.exp(torch.clamp(g, max=0.0)), x.clone()
    order = np.argsort(depth, kind="stable")
    cuts = np.searchsorted(depth[order], np.arange(int(depth.max()) + 2))
    order_t, up = torch.from_numpy(order).to(dev), torch.from_numpy(np.where(prev < 0, n, prev)[order]).to(dev)
    h = torch.zeros(n + 1, x.shape[1], dtype=torch.float64, device=dev)
    before = torch.zeros_like(x)
    h0 = torch.zeros_like(h)
    if case["init"]:
        for v, t in starts:
            h0[t] = s["init"][v].double()
    for i in range(len(cuts) - 1):
        rows, above = order_t[cuts[i]:cuts[i + 1]], up[cuts[i]:cuts[i + 1]]
        if i == 0:
            before[rows] = h0[rows]
        else:
            before[rows] = h[above]
        h[rows] = a[rows] * before[rows] + b[rows]
    lt = torch.from_numpy(np.where(last < 0, n, last)).to(dev)
    final = h[lt]
    out = dict(y=h[:n], final=final)
    if not case["train"]:
        return out
    lam = torch.cat([s["dy"].double(), torch.zeros(1, x.shape[1], dtype=torch.float64, device=dev)])
    if case["init"]:
        lam.index_add_(0, lt, s["d_final"].double())  # row n takes those of nodes without tokens
    for i in range(len(cuts) - 2, 0, -1):
        rows, above = order_t[cuts[i]:cuts[i + 1]], up[cuts[i]:cuts[i + 1]]
        lam.index_add_(0, above, a[rows] * lam[rows])
    lam = lam[:n]
    if case["init"]:
        d_init = torch.zeros_like(s["init"], dtype=torch.float64)
        for v, t in starts:
            d_init[v] = a[t] * lam[t]
        out["d_init"] = d_init
    if case["gate"] == "sigmoid":
        return dict(out, dgate=lam * (before - x) * a * (1 - a), dx=lam * torch.sigmoid(-g))
    return dict(out, dgate=lam * before * a * (g <= 0), dx=lam)
