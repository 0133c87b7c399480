"""Oracle for the gated linear recurrence on a tree (TEST INFRASTRUCTURE ONLY): the recurrent layer of
"Tree Training 技术详解" section 9.1, h_t = a_t h_prev(t) + b_t along every root-to-leaf path, token by
token in fp64, and the gradients of L = sum_t <dy_t, y_t> + sum_v <d_final_v, final_v>.

Next to each result stands its `e_*`: how far the same recurrence in 32 bits may be off, in units of one
rounding.  Every token adds one unit of the magnitudes it handles and passes on what reached it:
e_t = a_t e_prev + m_t with m_t = a_t m_prev + |b_t|, and the same from the leaves up for the gradient."""
from __future__ import annotations

import numpy as np

from .tree import plan as _plan


def token_prev(parent, node_len, p):
    """prev(t) of every packed token, -1 before a root, taken from the tokens of the root-to-leaf paths."""
    prev = np.full(p["n_tokens"], -2, dtype=np.int64)
    for path in p["paths"]:
        toks = np.concatenate([np.arange(p["tok_start"][v], p["tok_start"][v] + node_len[v]) for v in path]).astype(int)
        if len(toks):
            before = np.concatenate([[-1], toks[:-1]])
            seen = prev[toks] != -2
            assert (prev[toks][seen] == before[seen]).all()
            prev[toks] = before
    return prev


def decay_and_input(gate, x, kind):
    """a, 1 - a and b in fp64 (1 - a without cancellation)."""
    gate, x = np.asarray(gate, np.float64), np.asarray(x, np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            a, s = 1 / (1 + np.exp(-gate)), 1 / (1 + np.exp(gate))
        return a, s, s * x
    q = np.where(gate > 0, 0.0, gate)
    return np.exp(q), -np.expm1(q), x


def scan(parent, node_len, gate, x, kind, init=None, dy=None, d_final=None, p=None):
    node_len = np.asarray(node_len, dtype=np.int64)
    p = p if p is not None else _plan(parent, node_len)
    N, n = p["n_tokens"], len(node_len)
    x = np.asarray(x, np.float64)
    C = x.shape[1]
    a, s, b = decay_and_input(gate, x, kind)
    prev = token_prev(parent, node_len, p)
    node = np.asarray(p["tok_node"])[:N]
    h, m, e = (np.zeros((N, C)) for _ in range(3))
    hp, mp, ep = (np.zeros((N, C)) for _ in range(3))
    for t in range(N):
        if prev[t] >= 0:
            hp[t], mp[t], ep[t] = h[prev[t]], m[prev[t]], e[prev[t]]
        elif init is not None:
            hp[t] = init[node[t]]
            mp[t] = np.abs(hp[t])
        h[t] = a[t] * hp[t] + b[t]
        m[t] = a[t] * mp[t] + np.abs(b[t])
        e[t] = a[t] * ep[t] + m[t]
    last = np.where(node_len > 0, np.asarray(p["tok_start"]) + node_len - 1, -1)
    has = last >= 0
    final, e_final = np.zeros((n, C)), np.zeros((n, C))
    final[has], e_final[has] = h[last[has]], e[last[has]]
    out = dict(y=h, e_y=e, final=final, e_final=e_final, prev=prev)
    if dy is None:
        return out
    lam = np.array(dy, dtype=np.float64)
    if d_final is not None:
        lam[last[has]] += np.asarray(d_final, np.float64)[has]
    ml, el = np.abs(np.asarray(dy, np.float64)), np.zeros((N, C))
    if d_final is not None:
        ml[last[has]] += np.abs(np.asarray(d_final, np.float64))[has]
    d_init, e_init = np.zeros((n, C)), np.zeros((n, C))
    for t in range(N - 1, -1, -1):
        el[t] += ml[t]
        if prev[t] >= 0:
            lam[prev[t]] += a[t] * lam[t]
            ml[prev[t]] += a[t] * ml[t]
            el[prev[t]] += a[t] * el[t]
        else:
            d_init[node[t]] = a[t] * lam[t]
            e_init[node[t]] = a[t] * (el[t] + ml[t])
    if kind == "sigmoid":
        dx, e_dx = lam * s, s * (el + ml)
        dg = lam * s * a * (hp - x)
        e_dg = s * a * (np.abs(hp - x) * (el + ml) + np.abs(lam) * (ep + mp + np.abs(x)))
    else:
        dx, e_dx = lam, el + ml
        on = np.asarray(gate, np.float64) <= 0
        dg = np.where(on, lam * a * hp, 0.0)
        e_dg = np.where(on, a * (np.abs(hp) * (el + ml) + np.abs(lam) * (ep + mp)), 0.0)
    out.update(dgate=dg, e_dgate=e_dg, dx=dx, e_dx=e_dx, d_init=d_init, e_d_init=e_init, lam=lam)
    return out
