"""Rows whose scores are all -inf: the query's products with every key of its segment overflow fp32.
Such a row has no weights, as one of a segment without keys: o = 0, lse = -inf, and a gradient of 0
in which it takes no part -- however the work is cut.  The rows next to it are checked against the fp64
oracle with the tolerances of test_gpu_cross_attn.py and test_gpu_cross_attn_bwd.py (the oracle is given a
gradient of 0 for the rows without weights, so that they add nothing to its dk and dv).

Queries of -3e38 and keys of at least 0.1: 64 products of -3e37 or less are beyond fp32's 3.4e38, and with
one sign only no NaN can arise on the way.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_cross_attn import HALF, Case
from tests.test_gpu_cross_attn_bwd import _check as check_gradient

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


CASES = {  # as in test_gpu_cross_attn.py
    "whole_items": ([150, 20], [200, 129], 2, 2, 64, None),
    "keys_cut": ([30, 40], [3000, 2100], 2, 2, 128, None),
    "keys_cut_shared_heads": ([70], [4001], 4, 2, 64, [3900]),
    "rows_cut": ([3000], [60], 2, 2, 64, None),
    "tokens": ([1, 2, 1], [40, 20, 1], 4, 2, 128, None),
    "tokens_cut": ([1, 2], [3000, 20], 8, 1, 64, [2999, 20]),
}


def _case(name):
    c = Case(*CASES[name], seed=21)
    c.k.abs_().add_(0.1)
    rng = np.random.default_rng(22)
    bad = torch.from_numpy(rng.random(c.q.shape[:2]) < 0.2)
    bad[0, 0], bad[c.nq:] = True, False
    c.q[bad] = -3e38
    return c, bad


@pytest.mark.parametrize("name", CASES)
def test_forward(h3, dev, name):
    c, bad = _case(name)
    args, where = c.on(dev)
    out, lse = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)
    assert h3.get_device_error(dev) == 0
    bad = bad[:c.nq]
    got, gl = out[:c.nq].double().cpu(), lse.T[:c.nq].double().cpu()
    assert (got[bad] == 0).all() and torch.isneginf(gl[bad]).all()
    o, l, size = c.reference()
    ok = ~bad.numpy()
    err = np.abs(got.numpy() - o)[ok]
    assert np.all(err <= ((HALF + 2e-4) * (1 + HALF) * size + HALF * np.abs(o))[ok])
    assert np.all(np.abs(gl.numpy() - l.T)[ok] <= 1e-4 * np.maximum(np.abs(l.T), 1.0)[ok])


@pytest.mark.parametrize("name", CASES)
def test_gradient(h3, dev, name):
    c, bad = _case(name)
    args, where = c.on(dev)
    o, l, _ = c.reference()
    out, lse = torch.full(c.q.shape, float("nan")), torch.full((c.q.shape[1], c.cq), float("nan"))
    out[:c.nq], lse[:, :c.nq] = torch.from_numpy(o).float(), torch.from_numpy(l).float()
    out[bad], lse.T[bad] = 0.0, float("-inf")
    got = h3.varlen_cross_attn_bwd(c.do.to(dev), **args, out=out.to(torch.bfloat16).to(dev), lse=lse.to(dev), **where)
    assert h3.get_device_error(dev) == 0
    assert (got[0].cpu()[bad] == 0).all()
    c.do[bad] = 0.0
    check_gradient(c, got)
