"""fp64 RMS norm of query and key rows per head with the tagged rotation, and its gradient.

Test infrastructure only, never product code.

For one row x (a token's head, D values), weight w and the rotation R(phi) of ``rope``:
    y = R(phi) (x * w / sqrt(mean(x^2) + eps))
The gradient is the chain rule written out:  with dz = R(-phi) dy, u = x / sqrt(mean(x^2) + eps),
    dw = sum over rows of dz * u,    dx = (dz w - u mean(dz w u)) / sqrt(mean(x^2) + eps).
"""
from __future__ import annotations

import numpy as np

from .rope import request_time_offsets, rope_angles, rotate_pairs


def _f64(x) -> np.ndarray:
    return x.detach().cpu().double().numpy() if hasattr(x, "detach") else np.asarray(x, dtype=np.float64)


def _phi(n, head_dim, pos, tag, cu_requests, start_frames, cfg):
    if pos is None:
        return np.zeros((n, head_dim // 2))
    if start_frames is not None and cu_requests is None:
        cu_requests = [0, n]
    off = request_time_offsets(n, cu_requests, start_frames, cfg)
    return rope_angles(np.asarray(pos)[:n], np.asarray(tag)[:n], head_dim, cfg, off)


def norm_rope(x, weight, pos=None, tag=None, cu_requests=None, start_frames=None, cfg=None, eps=1e-6):
    """y [N, H, D] of x [N, H, D]; without pos the norm alone."""
    x, w = _f64(x), _f64(weight)
    z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate_pairs(z, _phi(x.shape[0], x.shape[2], pos, tag, cu_requests, start_frames, cfg))


def norm_rope_grad(dy, x, weight, pos=None, tag=None, cu_requests=None, start_frames=None, cfg=None, eps=1e-6):
    """(dx [N, H, D], dweight [D]) of norm_rope."""
    x, w, dy = _f64(x), _f64(weight), _f64(dy)
    dz = rotate_pairs(dy, -_phi(x.shape[0], x.shape[2], pos, tag, cu_requests, start_frames, cfg))
    length = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x / length
    g = dz * w
    return (g - u * (g * u).mean(-1, keepdims=True)) / length, (dz * u).sum((0, 1))
