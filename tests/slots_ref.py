"""64-bit references of the slot operators, and the inputs of their tests (CPU, torch)."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24                       # half a step of fp32, relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tokens(n, heads, qk_heads, dk, dv, dtype, seed, diag=0, slow=False, pad=0):
    """q, k, v, alpha, beta of n tokens.  pad: extra elements behind each token's row of q, k and v
    (a slice of a wider projection), filled with NaN."""
    g = torch.Generator().manual_seed(seed)

    def rows(h, d):
        x = torch.randn((n, h * d), generator=g)
        x = (x.view(n, h, d) / d ** 0.5).reshape(n, h * d).to(dtype)
        if pad:
            wide = torch.full((n, h * d + pad), float("nan"), dtype=dtype)
            wide[:, :h * d] = x
            x = wide
        return x[:, :h * d].unflatten(1, (h, d))

    q, k = rows(qk_heads, dk), rows(qk_heads, dk)
    v = rows(heads, dv)
    shape = (n, heads, dk) if diag else (n, heads)
    alpha = torch.sigmoid(torch.randn(shape, generator=g) + (7.0 if slow else 2.5))
    beta = torch.sigmoid(torch.randn((n, heads), generator=g))
    return q, k, v, alpha, beta


def recur(S, q, k, v, alpha, beta, delta=0):
    """The recurrence of one sequence in 64 bits: S [heads, dv, dk], tokens leading.  Returns
    (o, S, |o|, |S|), the last two with every term taken by its absolute value (delta 0)."""
    S = S.double().clone()
    A = S.abs()
    heads = S.shape[0]
    share = heads // q.shape[1]
    o, ao = [], []
    for t in range(q.shape[0]):
        kt = k[t].double().repeat_interleave(share, 0)
        qt = q[t].double().repeat_interleave(share, 0)
        a = alpha[t].double()
        a = a[:, None, :] if a.dim() == 2 else a[:, None, None]
        S = S * a
        w = v[t].double()
        if delta:
            w = w - (S * kt[:, None, :]).sum(-1)
        w = w * beta[t].double()[:, None]
        S = S + w[..., None] * kt[:, None, :]
        A = A * a + w.abs()[..., None] * kt.abs()[:, None, :]
        o.append((S * qt[:, None, :]).sum(-1))
        ao.append((A * qt.abs()[:, None, :]).sum(-1))
    empty = torch.zeros(0, heads, S.shape[1], dtype=torch.float64)
    return torch.stack(o) if o else empty, S, torch.stack(ao) if ao else empty, A


def batch_ref(pool, slots, fresh, cu, q, k, v, alpha, beta, delta=0):
    """attend over a pool [slots, heads, dv, dk]: (o with NaN rows where none is written, pool,
    |o|, |pool|)."""
    pool = pool.double().clone()
    mag = pool.abs()
    n, heads, dv = q.shape[0], pool.shape[1], pool.shape[2]
    o = torch.full((n, heads, dv), float("nan"), dtype=torch.float64)
    ao = torch.zeros_like(o)
    for i, s in enumerate(slots):
        a, b = cu[i], cu[i + 1]
        if s < 0 or b <= a:
            continue
        S0 = torch.zeros_like(pool[s]) if fresh is not None and fresh[i] else pool[s]
        o[a:b], pool[s], ao[a:b], mag[s] = recur(S0, q[a:b], k[a:b], v[a:b], alpha[a:b], beta[a:b], delta)
    return o, pool, ao, mag


def rel(x, y) -> float:
    """2-norm of the difference over the 2-norm of y."""
    d = (x.double() - y).norm()
    return float(d / y.norm()) if float(y.norm()) else float(d)
