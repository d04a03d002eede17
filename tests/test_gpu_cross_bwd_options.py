"""Gradient of cross attention: a scale of the caller's, bounds looser than the lengths, and the gradient of
packed self attention on a long segment.

Tolerances as in test_gpu_cross_attn_bwd.py, with the caller's scale in the exponent and in dq and dk."""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_cross_attn import CASES, HALF, Case
from tests.test_gpu_cross_attn_bwd import LARGE, _given
from tests.test_gpu_cross_attn_bwd import _check as check_default_scale

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h3():
    import __graft_entry__

    __graft_entry__.build()
    import packed_varlen_attention_modality_gb300 as h3

    h3.load_library()
    return h3


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    return torch.device("cuda", 0)


SCALED = {  # rows, keys, heads, key heads, dim, used
    "whole": ([37, 1, 130], [150, 90, 0], 4, 2, 64, None),
    "rows_cut": ([3000], [60], 2, 2, 64, None),
    "keys_cut": ([130, 20], [2500, 700], 4, 4, 128, [2400, 700]),
}


@pytest.mark.parametrize("scale", [0.05, 1.0])
@pytest.mark.parametrize("name", SCALED)
def test_scale(h3, dev, name, scale):
    c = Case(*SCALED[name], seed=13, scale=0.6)
    args, where = c.on(dev)
    o, l, _ = c.reference(scale)
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16)
    lse = torch.full((c.q.shape[1], c.cq), float("nan"))
    out[:c.nq], lse[:, :c.nq] = torch.from_numpy(o).to(torch.bfloat16), torch.from_numpy(l).float()
    got = h3.varlen_cross_attn_bwd(c.do.to(dev), **args, out=out.to(dev), lse=lse.to(dev), **where,
                                   softmax_scale=scale)
    assert h3.get_device_error(dev) == 0
    ref = oracle.cross_attention_grad(c.do, c.q, c.k, c.v, c.cu_q, c.cu_k, c.used, scale)
    for x, r, b, n in zip(got, ref, _bounds(c, scale), (c.nq, c.nk, c.nk)):
        err = np.abs(x.double().cpu().numpy()[:n] - r[:n])
        assert np.all(err <= (1 + HALF) * b[:n] + HALF * np.abs(r[:n]))


def _bounds(c, scale):
    """Error bounds of (dq, dk, dv) before their own rounding."""
    q, k, v, do = (t.double().numpy() for t in (c.q, c.k, c.v, c.do))
    group = q.shape[1] // k.shape[1]
    bq, bk, bv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for g in range(len(c.lq)):
        rows = slice(int(c.cu_q[g]), int(c.cu_q[g + 1]))
        n = c.lk[g] if c.used is None else c.used[g]
        keys = slice(int(c.cu_k[g]), int(c.cu_k[g]) + n)
        for h in range(q.shape[1] if n > 0 else 0):
            x = h // group
            p, _ = oracle.cross._probabilities(q[rows, h], k[keys, x], scale)
            dp = do[rows, h] @ v[keys, x].T
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            mass = 1e-5 * (np.abs(do[rows, h]) @ np.abs(v[keys, x]).T)
            mass += HALF * (np.abs(do[rows, h]) * np.abs(p @ v[keys, x])).sum(1, keepdims=True)
            e = (HALF + 1e-4) * np.abs(ds) + p * mass
            bq[rows, h] = scale * (e @ np.abs(k[keys, x]))
            bk[keys, x] += scale * (e.T @ np.abs(q[rows, h]))
            bv[keys, x] += (HALF + 1e-4) * (p.T @ np.abs(do[rows, h]))
    return bq, bk, bv


@pytest.mark.parametrize("name", ["padded_batch", "shared_heads", "few_rows_many_keys", "tokens", "many_segments",
                                  "text_states", "padded_shared", "many_key_tiles"])
def test_looser_bounds(h3, dev, name):
    """Bounds of the capacities give another workspace and may give another cut, not another gradient."""
    c = Case(*{**CASES, **LARGE}[name], seed=5)
    args, where = c.on(dev)
    out, lse = _given(c, dev)
    where.update(max_seqlen_q=c.cq, max_seqlen_k=c.ck)
    got = h3.varlen_cross_attn_bwd(c.do.to(dev), **args, out=out, lse=lse, **where)
    assert h3.get_device_error(dev) == 0
    check_default_scale(c, got)


def check_one_head(q, k, v, do, got):
    """dq, dk and dv of one segment and head, [rows, D] each, against fp64 on the GPU.  They come from the
    forward's own o, so the row sum carries its two roundings: |o - o*| <= 2^-8 sum P |v| + 2^-8 |o|."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    scale = q.shape[1] ** -0.5
    p = torch.softmax(scale * (q @ k.T), 1)
    dp, o = do @ v.T, p @ v
    ds = p * (dp - (p * dp).sum(1, keepdim=True))
    mass = 1e-5 * (do.abs() @ v.abs().T)
    mass += HALF * (do.abs() * (p @ v.abs() + o.abs())).sum(1, keepdim=True)
    e = (HALF + 1e-4) * ds.abs() + p * mass
    want = (scale * (ds @ k), scale * (ds.T @ q), p.T @ do)
    bound = (scale * (e @ k.abs()), scale * (e.T @ q.abs()), (HALF + 1e-4) * (p.T @ do.abs()))
    for name, x, r, w in zip(("dq", "dk", "dv"), got, want, bound):
        assert ((x.double() - r).abs() <= (1 + HALF) * w + HALF * r.abs()).all(), name


def test_gradient_of_a_long_packed_segment(h3, dev):
    """14,001 rows beside a short segment."""
    lengths, heads, d = [14001, 77], 2, 128
    n, cu = sum(lengths), torch.tensor([0, 14001, 14078], dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(17)
    q, k, v, do = (torch.randn(n, heads, d, device=dev, generator=g).to(torch.bfloat16) for _ in range(4))
    out, lse = h3.varlen_attn_fwd(q, k, v, cu, max(lengths), return_lse=True)
    got = h3.varlen_cross_attn_bwd(do, q, k, v, out, lse, cu, cu, max(lengths), max(lengths))
    assert h3.get_device_error(dev) == 0
    for a, b in ((0, 14001), (14001, 14078)):
        for h in range(heads):
            check_one_head(*(t[a:b, h] for t in (q, k, v, do)), [x[a:b, h] for x in got])
