"""residual_norm and its gradient where a CTA has many more rows than its ring in shared memory has stages, so that
stages are loaded again, the ring's and the exchanges' phases turn over many times, and a column's sum is long.

Bounds as in test_gpu_residual_norm.py, but for the sums over tokens: a CTA of n rows adds n terms in turn, then at
most 40 steps join strands and requests, each off by 2^-24 of what it has summed up, so E there is 1e-5 for the terms
themselves and (n + 40) 2^-24 for the sums.
"""
import numpy as np
import pytest
import torch

import test_gpu_residual_norm as base
from test_gpu_residual_norm import _case, _check_bwd, _check_fwd, _clean, _on, _rand, dev, h3  # noqa: F401

BF, F32 = torch.bfloat16, torch.float32


def _requests(n):
    """Offsets whose borders lie inside the CTAs' ranges: an empty request and one of a single row among them."""
    a, b = n // 3 + 1, n // 3 + 2
    return [0, a, a, b, n - n // 5 - 3, n]


# rows, dim, norm, branch norm, stream, has y, alpha, rows of a CTA on 152 SMs: at least twice its ring's stages (2 to 8)
BACKWARD = [
    (1830, 5120, "rms", "rms", BF, True, 0.75, 13),
    (1370, 5120, "layer", "rms", F32, True, 1.0, 10),
    (1370, 5120, "rms", "none", F32, True, 1.0, 10),
    (780, 8192, "layer", "layer", F32, True, 0.5, 6),
    (1070, 8192, "rms", "rms", BF, True, 1.0, 8),
    (3350, 2560, "rms", "layer", BF, True, 1.0, 12),
    (3350, 2504, "none", "rms", F32, True, 2.0, 12),
    (6700, 1536, "layer", "none", BF, True, 1.0, 12),
    (9200, 1000, "rms", "rms", F32, True, 1.0, 13),
    (9200, 1000, "layer", "none", BF, False, 1.0, 13),
    (17100, 512, "layer", "layer", BF, True, 1.0, 15),
    (17100, 264, "rms", "rms", BF, True, 1.0, 15),
    (243300, 40, "rms", "rms", BF, True, 1.0, 201),
    (60900, 8, "layer", "layer", F32, True, 1.0, 51),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", BACKWARD)
def test_backward(h3, dev, shape, monkeypatch):  # noqa: F811
    n, dim, norm, branch_norm, stream, has_y, alpha, rows = shape
    cu = _requests(n)
    x, y, step = _case((n, dim, cu, norm, branch_norm, F32, BF, stream, has_y, alpha), seed=21)
    rng = np.random.default_rng(22)
    dx_out, dh = _rand(rng, n, dim, kind=stream), None if norm == "none" else _rand(rng, n, dim)
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    args, here = (to(dx_out), to(dh), x.to(dev), to(y)), _on(dev, step)
    g = h3.residual_norm_bwd(*args, **here)
    # in place, with a workspace of NaN: the same bits
    ws = torch.full((h3.residual_norm_bwd_workspace_size(n, dim, len(cu) - 1) // 4,), float("nan"), device=dev)
    mine = [None if t is None else t.clone() for t in args]
    again = h3.residual_norm_bwd(*mine, **here, dx=mine[0], dy=mine[3] if has_y else None, workspace=ws.view(torch.uint8))
    _clean(h3, dev)
    for a, b in zip(g, again):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    monkeypatch.setattr(base, "E", 1e-5 + (rows + 40) * 2.0 ** -24)
    _check_bwd(h3.ResidualNormGrads(*(None if t is None else t.cpu() for t in g)), dx_out, dh, x, y, step)


FORWARD = [
    (3100, 5120, "layer", "none", BF, True, 1.0),
    (2500, 5120, "rms", "rms", F32, True, 0.75),
    (920, 8192, "layer", "layer", F32, True, 1.0),
    (5500, 2560, "none", "rms", F32, True, 0.5),
    (7700, 1536, "rms", "none", BF, False, 1.0),
    (13500, 1000, "layer", "rms", BF, True, 1.0),
    (30500, 264, "rms", "layer", F32, True, 1.0),
    (60900, 40, "layer", "none", BF, True, 1.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", FORWARD)
def test_forward(h3, dev, shape):  # noqa: F811
    n, dim, norm, branch_norm, stream, has_y, alpha = shape
    x, y, step = _case((n, dim, _requests(n), norm, branch_norm, F32, BF, stream, has_y, alpha), seed=23)
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    here = _on(dev, step)
    s, h = h3.residual_norm(x.to(dev), to(y), **here)
    if has_y:  # in place: the same bits
        mx, my = x.to(dev), y.to(dev)
        s2, h2 = h3.residual_norm(mx, my, **here, x_out=mx, h_out=None if norm == "none" else my)
        assert torch.equal(s, s2) and (h is None or torch.equal(h, h2))
    _clean(h3, dev)
    _check_fwd(s.cpu(), None if h is None else h.cpu(), x, y, step)
