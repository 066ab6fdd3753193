"""Plain 64-bit definitions of the speculative-decoding operators, on the CPU (test
infrastructure; independent of the library and of perf/operators.py)."""
import math

import numpy as np
import torch


def ancestors(parents, n_nodes):
    """Per node the sorted list of itself and its ancestors, or None where the parents are not a
    tree's (a parent outside [-1, i), or such an ancestor)."""
    out = []
    for i in range(n_nodes):
        p = int(parents[i])
        if p == -1:
            out.append([i])
        elif p < -1 or p >= i or out[p] is None:
            out.append(None)
        else:
            out.append(out[p] + [i])
    return out


def wide_bound(o, a, v, dtype):
    """The same for fp32 q and o over a 16-bit cache.  q and P enter as two parts, each off by at most
    h^2, h = eps / 2: h^2 A from P, and from q, with |q|.|k| scale below 16, weights off by 16 h^2.  S
    sums up to 256 products in fp32: 256 x 2^-24 x 16 = 2^-12; exp2, the sums and the merge 2^-13.  The
    weights' sum moves as well: twice that.  fp16 parts below 2^-14 are multiples of 2^-24 (x 2^-7)."""
    h2 = (torch.finfo(dtype).eps / 2) ** 2
    tiny = 2.0 ** -31 * v.double().abs().amax() * v.shape[2] if dtype == torch.float16 else 1e-30
    return 2.0 ** -24 * o.abs() + (h2 + 2 * (16 * h2 + 2.0 ** -12 + 2.0 ** -13)) * a + tiny


def random_tree(rng, n, kind):
    if kind == "chain":
        return np.arange(n, dtype=np.int32) - 1
    if kind == "star":
        return np.array([-1] + [0] * (n - 1), dtype=np.int32)
    if kind == "forest":
        return np.array([-1 if i == 0 or rng.random() < 0.3 else rng.integers(0, i) for i in range(n)],
                        dtype=np.int32)
    return np.array([-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n)], dtype=np.int32)


def attention_rows(q, k, v, parents, n_nodes, lens, scale):
    """o and A = sum_j p_j |v_j| in float64, [B, n, hq, d]; NaN rows where nothing is written."""
    q, k, v = q.double(), k.double(), v.double()
    B, n, hq, d = q.shape
    hkv, S = k.shape[1], k.shape[2]
    o = torch.full((B, n, hq, d), math.nan, dtype=torch.float64)
    a = torch.zeros((B, n, hq, d), dtype=torch.float64)
    for b in range(B):
        ln = min(max(int(lens[b]), 0), S)
        nn = min(min(max(int(n_nodes[b]), 0), n) if n_nodes is not None else n, S - ln)
        anc = ancestors(parents[b], nn)
        for i in range(nn):
            if anc[i] is None:
                o[b, i] = 0
                continue
            rows = torch.tensor(list(range(ln)) + [ln + x for x in anc[i]])
            for h in range(hq):
                kk, vv = k[b, h // (hq // hkv), rows], v[b, h // (hq // hkv), rows]
                p = torch.softmax(kk @ q[b, i, h] * scale, 0)
                o[b, i, h] = p @ vv
                a[b, i, h] = p @ vv.abs()
    return o, a


def attention_bound(o, a, v, dtype):
    """|error| allowed, value by value.  Roundings, each at most half a step h = eps / 2 relative:
    the output's (h |o|) and P's (h per weight: h A, A = sum p |v|).  fp32 work: S sums d <= 128
    products in fp32 steps; with |q|.|k| scale below 16 each weight moves by at most 128 x 16 x
    2^-23 < 2^-11 relative, and exp2, the sums over keys and the merge stay below 2^-13 together;
    (2^-11 + 2^-13) A, doubled since the sum of the weights moves as well.  fp16 weights below
    2^-14 x 2^-7 are rounded to multiples of 2^-24 x 2^-7 of the largest: 2^-32 |v| each."""
    h = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -32 * v.double().abs().amax() * v.shape[2] + 2.0 ** -25 if dtype == torch.float16 else 1e-30
    return h * (1 + h) * (o.abs() + a) + 2 * (2.0 ** -11 + 2.0 ** -13) * a + tiny


def softmax_long(x, temperature):
    """Softmax of x / temperature in extended precision; temperature 0: one-hot at the largest
    value's lowest index; None where x is no distribution."""
    x = x.astype(np.longdouble)
    if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
        return None
    if temperature == 0:
        return (np.arange(x.size) == int(np.argmax(x))).astype(np.longdouble)
    e = np.exp((x - x.max()) / np.longdouble(temperature))
    return e / e.sum()


def verify_walk(target, draft, tokens, parents, n_nodes, u, r, temperature, draft_temperature):
    """path, next token and the smallest relative distance of any decision to its border, for one
    sequence (numpy arrays)."""
    V = target.shape[1]
    margin = np.inf
    if n_nodes == 0:
        return [], -1, margin
    greedy = temperature == 0
    word = np.arange(V)
    path, cur = [0], 0
    P = softmax_long(target[0], temperature)
    for c in range(1, n_nodes):
        if parents[c] != cur or P is None:
            continue
        x = int(tokens[c])
        if greedy or draft is None:
            q = (word == x).astype(np.longdouble)
        else:
            q = softmax_long(draft[cur], draft_temperature)
        qx, px = (q[x], P[x]) if 0 <= x < V else (np.longdouble(draft is None or greedy), np.longdouble(0))
        a = np.longdouble(0 if greedy else u[c]) * qx
        if max(a, px) > 0:
            margin = min(margin, abs(a - px) / max(a, px))
        if a < px:
            path.append(c)
            cur, P = c, softmax_long(target[c], temperature)
        elif not greedy:
            rest = np.maximum(P - q, 0)
            if rest.sum() > 0:
                P = rest / rest.sum()
    if P is None:
        return path, -1, margin
    cum = np.cumsum(P)
    want = np.longdouble(r) * cum[-1]
    at = int(np.nonzero((cum > want) & (P > 0))[0][0]) if not greedy else int(np.argmax(P))
    if not greedy:
        margin = min(margin, float(abs(cum - want)[P > 0].min()) * V)
    return path, at, margin
