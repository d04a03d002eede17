"""fp64 packed cross attention (queries and keys of different lengths) and its gradient.

Test infrastructure only, never product code.

Segment g: query rows [cu_q[g], cu_q[g+1]) attend to key rows [cu_k[g], cu_k[g] + used[g]); query
head h reads key head h * Hkv // Hq.  A segment without keys gives o = 0 and lse = -inf and takes
no gradient.  Gradient of sum(do * o):
    dv = P^T do,  dP = do v^T,  dS = P * (dP - rowsum(P * dP)),  dq = scale dS k,  dk = scale dS^T q.
"""
from __future__ import annotations

import numpy as np

from .norm import _f64


def _segments(cu_q, cu_k, used):
    for g in range(len(cu_q) - 1):
        b = int(cu_k[g])
        n = int(cu_k[g + 1]) - b if used is None else int(used[g])
        yield slice(int(cu_q[g]), int(cu_q[g + 1])), slice(b, b + n)


def _probabilities(q, k, scale):
    s = scale * (q @ k.T)
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    total = e.sum(1, keepdims=True)
    return e / total, (top + np.log(total))[:, 0]


def cross_attention(q, k, v, cu_q, cu_k, used=None, scale=None):
    """(o [Cq, Hq, D], lse [Hq, Cq]); rows of no segment are NaN."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    _, hq, d = q.shape
    group = hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, lse = np.full(q.shape, np.nan), np.full((hq, q.shape[0]), np.nan)
    for rows, keys in _segments(cu_q, cu_k, used):
        o[rows], lse[:, rows] = 0.0, -np.inf
        if keys.stop == keys.start:
            continue
        for h in range(hq):
            p, lse[h, rows] = _probabilities(q[rows, h], k[keys, h // group], scale)
            o[rows, h] = p @ v[keys, h // group]
    return o, lse


def cross_attention_grad(do, q, k, v, cu_q, cu_k, used=None, scale=None):
    """(dq, dk, dv) for the gradient do of o; rows of no segment are NaN, rows of a segment that
    take no part are 0."""
    do, q, k, v = _f64(do), _f64(q), _f64(k), _f64(v)
    _, hq, d = q.shape
    group = hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = (np.full(x.shape, np.nan) for x in (q, k, v))
    for g in range(len(cu_q) - 1):
        dq[int(cu_q[g]):int(cu_q[g + 1])] = 0.0
        dk[int(cu_k[g]):int(cu_k[g + 1])] = 0.0
        dv[int(cu_k[g]):int(cu_k[g + 1])] = 0.0
    for rows, keys in _segments(cu_q, cu_k, used):
        if keys.stop == keys.start:
            continue
        for h in range(hq):
            kh = h // group
            p, _ = _probabilities(q[rows, h], k[keys, kh], scale)
            dv[keys, kh] += p.T @ do[rows, h]
            dp = do[rows, h] @ v[keys, kh].T
            ds = scale * p * (dp - (p * dp).sum(1, keepdims=True))
            dq[rows, h] = ds @ k[keys, kh]
            dk[keys, kh] += ds.T @ q[rows, h]
    return dq, dk, dv
