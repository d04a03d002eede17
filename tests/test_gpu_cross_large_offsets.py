"""Rows past 2^31 elements of queries, outputs and their gradients, in the tile kernels of cross attention,
against fp64 with the tolerances of test_gpu_cross_attn.py and test_gpu_cross_bwd_options.py."""
import pytest
import torch

from tests.test_gpu_cross_attn import HALF
from tests.test_gpu_cross_bwd_options import check_one_head

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


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("keys", [90, 2600])  # whole items; cut ones
def test_last_rows(h3, dev, keys, dim):
    heads, tail = 40, 150
    n = 2 ** 31 // (heads * dim) + 3000
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(keys)
    x = lambda *shape: torch.randn(*shape, dim, device=dev, generator=g).to(torch.bfloat16)
    q, do = (torch.zeros(n, heads, dim, dtype=torch.bfloat16, device=dev) for _ in range(2))
    assert q.numel() > 2 ** 31
    q[-tail:], do[-tail:] = x(tail, heads), x(tail, heads)
    k, v = x(keys, heads), x(keys, heads)
    where = i32(0, n - tail, n), i32(0, 0, keys), n, keys  # the rows before have no keys
    o, lse = h3.varlen_cross_attn_fwd(q, k, v, *where, return_lse=True)
    dq, dk, dv = h3.varlen_cross_attn_bwd(do, q, k, v, o, lse, *where)
    assert h3.get_device_error(dev) == 0
    assert (o[:-tail] == 0).all() and torch.isneginf(lse[:, :-tail]).all() and (dq[:-tail] == 0).all()
    for h in range(heads):
        one = [t[:, h] for t in (q[-tail:], k, v, do[-tail:])]
        qh, kh, vh = (t.double() for t in one[:3])
        s = dim ** -0.5 * (qh @ kh.T)
        p = torch.softmax(s, 1)
        r = p @ vh
        assert ((o[-tail:, h].double() - r).abs() <= (HALF + 2e-4) * (1 + HALF) * (p @ vh.abs()) + HALF * r.abs()).all()
        top = torch.logsumexp(s, 1)
        assert ((lse[h, -tail:].double() - top).abs() <= 1e-4 * top.abs().clamp(min=1)).all()
        check_one_head(*one, (dq[-tail:, h], dk[:, h], dv[:, h]))
