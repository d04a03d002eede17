"""fp64 paged key/value cache (bf16, or e4m3 with a power-of-two scale per row) and attention over it.

Test infrastructure only, never product code.

Position j of segment g stands in page table[g][j // page], row j % page.  An e4m3 row holds
round(x / 2^e) to a sign, four exponent bits (bias 7) and three mantissa bits, to nearest even, with the
least integer e for which max |x| <= 448 * 2^e, kept within [-110, 120].
"""
from __future__ import annotations

import numpy as np

from .cross import _probabilities
from .norm import _f64

E4M3_MOST, SCALE_MIN, SCALE_MAX = 448.0, -110, 120


def e4m3_round(x):
    """fp64 values rounded to the nearest e4m3 value, ties to even; past 448 to 448."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)  # eight steps to a binade, 2^-9 below 2^-6
    with np.errstate(invalid="ignore"):
        return np.clip(np.rint(x / step) * step, -E4M3_MOST, E4M3_MOST)


def e4m3_scale(rows):
    """Exponent e of each row [..., D]."""
    most = np.abs(_f64(rows)).max(-1)
    e = np.full(most.shape, SCALE_MIN)
    for k in range(SCALE_MIN, SCALE_MAX):  # the definition, tried out
        e = np.where(most > E4M3_MOST * 2.0 ** k, k + 1, e)
    return e


def e4m3_row_values(rows):
    """What rows [..., D] read back as."""
    unit = np.ldexp(1.0, e4m3_scale(rows))[..., None]
    return e4m3_round(_f64(rows) / unit) * unit


def key_limit(position, used, block):
    """Keys that the token at `position` of `used` sees: all (block 0), or those of its causal block and before."""
    return used if block == 0 else min(used, max(0, (position // block + 1) * block))


def paged_attention(q, k_rows, v_rows, cu_q, used, block=0, scale=None):
    """(o [C, Hq, D], lse [Hq, C]): the rows of segment g are the last of its used[g] tokens, whose keys and
    values k_rows[g], v_rows[g] [used[g], Hkv, D] are.  Rows of no segment are NaN."""
    q = _f64(q)
    _, hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    o, lse = np.full(q.shape, np.nan), np.full((hq, q.shape[0]), np.nan)
    for g in range(len(cu_q) - 1):
        a, b = int(cu_q[g]), int(cu_q[g + 1])
        k, v = _f64(k_rows[g]), _f64(v_rows[g])
        for i in range(a, b):
            o[i], lse[:, i] = 0.0, -np.inf
        # rows with one limit are taken together
        limits = np.array([key_limit(int(used[g]) - (b - a) + i, int(used[g]), block) for i in range(b - a)])
        for n in np.unique(limits):
            if n == 0:
                continue
            rows = a + np.flatnonzero(limits == n)
            for h in range(hq):
                kh = h // (hq // k.shape[1])
                p, lse[h, rows] = _probabilities(q[rows, h], k[:n, kh], scale)
                o[rows, h] = p @ v[:n, kh]
    return o, lse
