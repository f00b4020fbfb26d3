"""64-bit references of the drafted-token operators, and the inputs of their tests (CPU, torch)."""
from __future__ import annotations

import random

import torch


def trees(counts, shape, seed):
    """Parents of packed trees: "chain", "star" (all behind node 0), "forest" (all behind the slot),
    "random" (any earlier node or the slot)."""
    r = random.Random(seed)
    out = []
    for n in counts:
        for j in range(n):
            out.append({"chain": j - 1, "star": min(j, 1) - 1, "forest": -1,
                        "random": r.randint(-1, j - 1) if j else -1}[shape])
    return out


def node(S, A, k, v, alpha, beta, delta):
    """One token behind state S [heads, dv, dk], with A the sums of its terms' magnitudes."""
    a = alpha[:, None, :] if alpha.dim() == 2 else alpha[:, None, None]
    S, A = S * a, A * a.abs()
    w, W = v, v.abs()
    if delta:
        w = w - (S * k[:, None, :]).sum(-1)
        W = W + (A * k.abs()[:, None, :]).sum(-1)
    w, W = w * beta[:, None], W * beta.abs()[:, None]
    return S + w[..., None] * k[:, None, :], A + W[..., None] * k.abs()[:, None, :]


def _row(x, t, share):
    return x[t].double().repeat_interleave(share, 0)


def tree_ref(pool, slots, fresh, cu, parents, q, k, v, alpha, beta, delta=0):
    """step_tree: (o with NaN rows where none is written, the sums of its terms' magnitudes)."""
    n, heads, dv = q.shape[0], pool.shape[1], pool.shape[2]
    share = heads // q.shape[1]
    o = torch.full((n, heads, dv), float("nan"), dtype=torch.float64)
    mag = torch.zeros_like(o)
    for i, s in enumerate(slots):
        if s < 0:
            continue
        S0 = pool[s].double() * (0.0 if fresh is not None and fresh[i] else 1.0)
        if fresh is not None and fresh[i]:
            S0 = torch.zeros_like(S0)
        states = {-1: (S0, S0.abs())}
        for j in range(cu[i + 1] - cu[i]):
            t = cu[i] + j
            states[j] = node(*states[parents[t]], _row(k, t, share), v[t].double(), alpha[t].double(),
                             beta[t].double(), delta)
            qt = _row(q, t, share)
            o[t] = (states[j][0] * qt[:, None, :]).sum(-1)
            mag[t] = (states[j][1] * qt.abs()[:, None, :]).sum(-1)
    return o, mag


def path_ref(pool, slots, fresh, cu, paths, k, v, alpha, beta, delta=0):
    """accept_path over lists of nodes: (pool, the sums of its terms' magnitudes)."""
    pool = pool.double().clone()
    mag = pool.abs()
    share = pool.shape[1] // k.shape[1]
    for i, s in enumerate(slots):
        if s < 0 or not paths[i]:
            continue
        S, A = pool[s], mag[s]
        if fresh is not None and fresh[i]:
            S, A = torch.zeros_like(S), torch.zeros_like(S)
        for j in paths[i]:
            t = cu[i] + j
            S, A = node(S, A, _row(k, t, share), v[t].double(), alpha[t].double(), beta[t].double(), delta)
        pool[s], mag[s] = S, A
    return pool, mag


def residual(p, q, tried, replacement):
    """What is left of a node's row after the tokens tried, by the definition: the residual
    distribution, normalised after each rejection.  q None: one-hot drafts."""
    p, gone = p.double().clone(), 0.0
    for x in tried:
        if q is None:
            px = float(p[x])
            p[x] = 0.0
            p = p / (1.0 - px) if px < 1.0 else p
            continue
        now = q.double() if replacement else q.double() / (1.0 - gone)
        p = (p - now).clamp(min=0)
        p = p / p.sum() if float(p.sum()) > 0 else p
        gone += float(q[x])
    return p, gone


def verify_ref(target, draft, ids, parents, cu, uniform, uniform_next, replacement, depth):
    """verify_tree over sound trees: (path, lengths, next) as lists, by the definition."""
    V = target.shape[1]
    paths, lengths, tokens = [], [], []
    for i in range(len(cu) - 1):
        a, n = cu[i], cu[i + 1] - cu[i]
        if n == 0:
            paths.append([-1] * depth), lengths.append(0), tokens.append(-1)
            continue
        path, left = [0], None
        while True:
            row, tried, taken = a + path[-1], [], None
            q = None if draft is None else draft[row]
            for j in range(path[-1] + 1, n):
                if len(path) >= depth:
                    break
                x = int(ids[a + j])
                if parents[a + j] != path[-1] or not 0 <= x < V:
                    continue
                p, gone = residual(target[row], q, tried, replacement)
                qx = 1.0 if q is None else float(q[x]) if replacement else float(q[x]) / (1.0 - gone)
                if float(uniform[a + j]) * qx < float(p[x]):
                    taken = j
                    break
                tried.append(x)
            if taken is None:
                left = residual(target[row], q, tried, replacement)[0]
                break
            path.append(taken)
        if float(left.sum()) == 0:
            left = target[row].double()
        cum = left.cumsum(0)
        y = int((cum <= float(uniform_next[i]) * float(cum[-1])).sum())
        tokens.append(min(y, int(torch.nonzero(left > 0)[-1])))
        paths.append(path + [-1] * (depth - len(path)))
        lengths.append(len(path))
    return paths, lengths, tokens
