"""Single tokens over an e4m3 cache when one value row outweighs the others by far, by its scale or by its score:
what the other rows add to columns in which that one holds zeros.

Tolerance, from the arithmetic.  o = sum_j w_j q_j / sum_j P_j, with q_j the e4m3 values of a row, 2^(e_j) its scale and
w_j = 2^(e_j) P_j.  The kernel rounds w_j to f16 over a reference that puts the largest at 2^7 or above: by 2^-11 of
itself or, below f16's normal numbers (2^-14), by half their spacing, 2^-25, which is 2^-32 of the largest.  Scores and
sums are fp32, 2e-4 of each weight at the scores used here; o is rounded to bf16, 2^-8 of itself:
    |o - o*| <= (2^-11 + 2e-4) sum_j P_j |v_j| + 2^-8 |o*| + 2^-32 max_j(w_j) sum_(w_j < 2^-21 max) |q_j|.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle.norm import _f64

PAGE = 16


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


def _cache(rows, exponents, page=PAGE):
    """e4m3 rows [n, d] that are e4m3 values, and their scales' exponents, as pages [pages, 1, page, d]."""
    n, d = rows.shape
    pages = -(-n // page)
    store = torch.zeros(pages * page, d)
    store[:n] = torch.from_numpy(rows)
    scale = torch.full((pages * page,), 127, dtype=torch.uint8)
    scale[:n] = torch.from_numpy(exponents + 127).to(torch.uint8)
    return store.to(torch.float8_e4m3fn).view(pages, 1, page, d), scale.view(pages, 1, page)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 8, 16])  # keys as the products' rows up to 8, query rows above
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("by", ["scale", "score"])
@pytest.mark.parametrize("gap", [14, 18, 22, 25])
@pytest.mark.parametrize("n", [25, 300])
def test_rows_beside_a_dominant_one(h3, dev, n, gap, by, d, heads):
    rng = np.random.default_rng(n + gap)
    q = torch.from_numpy(0.25 * rng.standard_normal((1, heads, d))).to(torch.bfloat16)
    k = oracle.e4m3_round(256 * rng.standard_normal((n, d)))
    ke = np.full(n, -8)
    v = oracle.e4m3_round(np.clip(64 + 32 * rng.standard_normal((n, d)), 1, 448))
    ve = np.full(n, -6)
    # one in every 32 rows, so that each warp of the kernel meets one; it holds zeros but for a column
    big = np.arange(0, n, 32)
    v[big] = 0.0
    v[big, 0] = 448.0
    if by == "scale":
        ve[big] += gap
    else:  # the last dimension carries the score alone
        q[..., -1] = 1.0
        k[:, -1] = 0.0
        k[big, -1], ke[big] = oracle.e4m3_round(gap * np.log(2.0) * np.sqrt(d) * 2), -1
        k[big, :-1] = 0.0
    kc, ks = _cache(k, ke)
    vc, vs = _cache(v, ve)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.arange(kc.shape[0], dtype=torch.int32, device=dev).view(1, -1)
    o, lse = h3.paged_attn_fwd(q.to(dev), kc.to(dev), vc.to(dev), table, i32(0, 1), i32(n), 1, n, k_scale=ks.to(dev),
                               v_scale=vs.to(dev), causal_block=1, return_lse=True)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    s = _f64(q[0]) @ (k * np.ldexp(1.0, ke)[:, None]).T / np.sqrt(d)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    rl = top[:, 0] + np.log(p.sum(-1))
    p /= p.sum(-1, keepdims=True)
    vals = v * np.ldexp(1.0, ve)[:, None]
    ref, size = p @ vals, p @ np.abs(vals)
    w = p * np.ldexp(1.0, ve)
    most = w.max(-1, keepdims=True)
    small = 2.0 ** -32 * most * (np.where(w < 2.0 ** -21 * most, 1.0, 0.0) @ np.abs(v))
    tol = (2.0 ** -11 + 2e-4) * size + 2.0 ** -8 * np.abs(ref) + small
    got = _f64(o[0])
    assert np.all(np.isfinite(got))
    off = np.abs(got - ref)
    assert np.all(off <= tol), ((off / tol).max(), (off - tol).max())
    assert np.all(np.abs(_f64(lse[:, 0]) - rl) <= 1e-4 * np.maximum(np.abs(rl), 1.0))
