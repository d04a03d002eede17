"""fp64 step between two branches of a block (gated residual, modulated norm) and its gradient.

Test infrastructure only, never product code.

For a token of request r, stream row x and branch output y (dim values each):
    u = N_b(y) w_b,  x' = alpha x + gate_r u,  h = N(x') w (1 + scale_r) + shift_r
N(x) is x ("none"), x / sqrt(mean(x^2) + eps) ("rms") or the same of x - mean(x) ("layer").  The gradient
is the chain rule, step by step, with the Jacobian of N applied in closed form.
"""
from __future__ import annotations

import numpy as np

from .norm import _f64


def unit(x, kind, eps):
    """(N(x), its factor) of rows x."""
    if kind == "none":
        return x, np.ones(x.shape[:-1] + (1,))
    c = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    f = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return c * f, f


def unit_grad(g, z, f, kind):
    """Gradient of x for the gradient g of z = N(x) with factor f."""
    if kind == "none":
        return g
    back = g - z * (g * z).mean(-1, keepdims=True)
    return f * (back - g.mean(-1, keepdims=True) if kind == "layer" else back)


def requests_of(n, cu_requests):
    cu = [0, n] if cu_requests is None else list(map(int, cu_requests))
    return np.repeat(np.arange(len(cu) - 1), np.diff(cu)), len(cu) - 1


def residual_norm(x, y=None, norm="rms", weight=None, scale=None, shift=None, gate=None, branch_norm="none",
                  branch_weight=None, residual_scale=1.0, cu_requests=None, eps=1e-6):
    """(x', h); h is None with norm "none"."""
    x = _f64(x)
    r, _ = requests_of(x.shape[0], cu_requests)
    if y is not None:
        u = unit(_f64(y), branch_norm, eps)[0]
        u = u if branch_weight is None else u * _f64(branch_weight)
        x = residual_scale * x + (u if gate is None else u * _f64(gate)[r])
    if norm == "none":
        return x, None
    h = unit(x, norm, eps)[0]
    h = h if weight is None else h * _f64(weight)
    h = h if scale is None else h * (1.0 + _f64(scale)[r])
    return x, h if shift is None else h + _f64(shift)[r]


def residual_norm_grad(dx_out, dh, x_out, y=None, norm="rms", weight=None, scale=None, shift=None, gate=None,
                       branch_norm="none", branch_weight=None, residual_scale=1.0, cu_requests=None, eps=1e-6):
    """dict of dx, dy, weight, branch_weight, scale, shift, gate, all of them (as if every vector were there)."""
    x = _f64(x_out)
    n, dim = x.shape
    r, requests = requests_of(n, cu_requests)
    one, zero = np.ones(dim), np.zeros((requests, dim))
    w, wb = (one if t is None else _f64(t) for t in (weight, branch_weight))
    sc = zero if scale is None else _f64(scale)
    gt = zero + 1.0 if gate is None else _f64(gate)

    def per_request(v):
        s = np.zeros((requests, dim))
        np.add.at(s, r, v)
        return s

    t = np.zeros(x.shape) if dx_out is None else _f64(dx_out)
    out = {}
    if norm != "none":
        dh = _f64(dh)
        z, f = unit(x, norm, eps)
        u = per_request(dh * z)
        out.update(shift=per_request(dh), scale=u * w, weight=(u * (1.0 + sc)).sum(0))
        t = t + unit_grad(dh * w * (1.0 + sc)[r], z, f, norm)
    out["dx"] = residual_scale * t
    if y is not None:
        z, f = unit(_f64(y), branch_norm, eps)
        v = per_request(t * z)
        out.update(gate=v * wb, branch_weight=(v * gt).sum(0), dy=unit_grad(t * wb * gt[r], z, f, branch_norm))
    return out
