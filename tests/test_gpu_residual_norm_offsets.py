"""residual_norm and its gradient record request offsets that are not what the header asks for: 0 first, not falling,
num_tokens last.  The forward's results stay those of some request in range, and good offsets record nothing."""
import numpy as np
import pytest
import torch

BAD_CU_SEQLENS = 3
# offsets of three requests over 37 rows
BAD = {"first": [3, 10, 20, 37], "negative": [-1, 10, 20, 37], "falling": [0, 20, 10, 37], "short": [0, 10, 20, 36],
       "long": [0, 10, 20, 38], "falling last": [0, 10, 37, 20]}
GOOD = [[0, 10, 20, 37], [0, 0, 0, 37], [0, 37, 37, 37]]


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


def _inputs(dev, dim, requests, norm, branch_norm, stream):
    gen = torch.Generator(device=dev).manual_seed(dim)
    rand = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    x, y, dh = rand(37, dim).to(stream), rand(37, dim).bfloat16(), rand(37, dim).bfloat16()
    mod = 0.3 * rand(requests, 3, dim)
    return x, y, dh, dict(norm=norm, branch_norm=branch_norm, scale=mod[:, 0], shift=mod[:, 1], gate=mod[:, 2],
                          weight=1 + 0.1 * rand(dim))


def _error(h3, dev):
    torch.cuda.synchronize()
    return h3.get_device_error(dev)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 1024, 5120])
@pytest.mark.parametrize("norm, branch_norm, stream", [("rms", "none", torch.bfloat16), ("layer", "rms", torch.float32)])
def test_bad_offsets_are_recorded(h3, dev, norm, branch_norm, stream, dim):
    x, y, dh, step = _inputs(dev, dim, 3, norm, branch_norm, stream)
    for cu in GOOD:
        cu = torch.tensor(cu, dtype=torch.int32, device=dev)
        s, _ = h3.residual_norm(x, y, **step, cu_requests=cu)
        assert _error(h3, dev) == 0
        h3.residual_norm_bwd(x, dh, s, y, **step, cu_requests=cu)
        assert _error(h3, dev) == 0
    want = h3.residual_norm(x, y, **step, cu_requests=torch.tensor(GOOD[0], dtype=torch.int32, device=dev))
    for name, cu in BAD.items():
        cu = torch.tensor(cu, dtype=torch.int32, device=dev)
        s, h = h3.residual_norm(x, y, **step, cu_requests=cu)
        assert _error(h3, dev) == BAD_CU_SEQLENS, name
        if name in ("first", "negative", "short", "long"):  # the rows keep the requests that they have anyhow
            assert torch.equal(s, want[0]) and torch.equal(h, want[1]), name
        h3.residual_norm_bwd(x, dh, s, y, **step, cu_requests=cu)
        assert _error(h3, dev) == BAD_CU_SEQLENS, name
    # fewer rows than the buffers hold: the last offset is num_tokens, not the rows
    cu = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device=dev)
    s, _ = h3.residual_norm(x, y, **step, cu_requests=cu, num_tokens=30)
    h3.residual_norm_bwd(x, dh, s, y, **step, cu_requests=cu, num_tokens=30)
    assert _error(h3, dev) == 0


@pytest.mark.gpu
def test_many_requests(h3, dev):
    """More requests than a warp has lanes, the fault among the last."""
    n, dim = 1300, 40
    cu = np.arange(0, n + 1, 2, dtype=np.int32)
    gen = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn(n, dim, device=dev, generator=gen).bfloat16()
    scale = 0.3 * torch.randn(len(cu) - 1, dim, device=dev, generator=gen)
    for bad in (False, True):
        if bad:
            cu[-3] = cu[-2] + 1
        offsets = torch.from_numpy(cu).to(dev)
        h3.residual_norm(x, scale=scale, cu_requests=offsets)
        assert _error(h3, dev) == (BAD_CU_SEQLENS if bad else 0)
        h3.residual_norm_bwd(None, x, x, scale=scale, cu_requests=offsets)
        assert _error(h3, dev) == (BAD_CU_SEQLENS if bad else 0)
