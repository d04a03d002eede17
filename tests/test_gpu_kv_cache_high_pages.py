"""What kv_cache_write puts into pages past 2^31 and 2^32 elements, byte for byte, and what it leaves alone."""
import numpy as np
import pytest
import torch

import oracle
from oracle.norm import _f64


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


@pytest.mark.gpu
def test_bytes_and_scales(h3, dev):
    h, d, page, pages = 8, 128, 256, 17000  # 4.46e9 elements
    ids, first, n = [pages - 1, 8200, 0], 20, 700
    zeros = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=dev)  # noqa: E731
    stores, scales = [zeros(pages, h, page, d) for _ in range(2)], [zeros(pages, h, page) for _ in range(2)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    rng = np.random.default_rng(3)
    rows = [torch.from_numpy(rng.standard_normal((n, h, d)) * np.exp(rng.standard_normal((n, h, 1)))).to(torch.bfloat16)
            for _ in range(2)]
    h3.kv_cache_write(*(t.to(dev) for t in rows), *(t.view(torch.float8_e4m3fn) for t in stores), i32([ids]),
                      i32([0, n]), i32([first]), *scales)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    for x, store, scale in zip(rows, stores, scales):
        e = oracle.e4m3_scale(x)
        values = oracle.e4m3_round(_f64(x) / np.ldexp(1.0, e)[..., None])
        want = np.zeros((3 * page, h, d))
        want_scale = np.zeros((3 * page, h), dtype=np.uint8)
        want[first:first + n], want_scale[first:first + n] = values, e + 127
        for i, p in enumerate(ids):
            part = slice(i * page, (i + 1) * page)
            got = store[p].view(torch.float8_e4m3fn).cpu().float().numpy().transpose(1, 0, 2)
            assert np.array_equal(got, want[part]), p
            assert np.array_equal(scale[p].cpu().numpy().T, want_scale[part]), p
        # no other page is touched
        hit = torch.tensor(ids, device=dev)
        assert int(torch.count_nonzero(scale)) == int(torch.count_nonzero(scale[hit]))
        some = torch.tensor([1, 2, 8199, 8201, pages - 2, 4, (8200 * 8) % pages], device=dev)
        assert int(torch.count_nonzero(store[some])) == 0
