"""Offsets that the cross attention calls meet on the device: changed between calls by the kernel before,
overlapping, of many segments, and with lengths whose products pass 32 bits."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cross_attn import Case
from tests.test_gpu_cross_attn import _check as check_forward
from tests.test_gpu_cross_attn_bwd import _check as check_gradient
from tests.test_gpu_cross_attn_bwd import _given

pytestmark = pytest.mark.gpu

BAD_OFFSETS, TIMEOUT = 3, 7  # H3_ERR_BAD_CU_SEQLENS, H3_ERR_TIMEOUT


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


def _i32(dev, *v):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _random(dev, *shape, seed=0):
    return torch.randn(*shape, device=dev, generator=torch.Generator(device=dev).manual_seed(seed)).to(torch.bfloat16)


# Two layouts of the same tensors: rows and key rows of each segment.
LAYOUTS = {
    "tokens": ([[1, 2, 1], [2, 1, 1]], [[3000, 700, 900], [40, 2560, 2000]], 8, 2, 64),
    "cut_keys": ([[30, 60, 100], [90, 20, 80]], [[3000, 700, 900], [1400, 2560, 640]], 4, 4, 128),
    "cut_rows": ([[2300, 60, 100], [90, 20, 2350]], [[130, 70, 60], [60, 40, 160]], 4, 2, 64),
}


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", LAYOUTS)
def test_offsets_written_by_the_kernel_before(h3, dev, name, captured):
    rows, keys, hq, hk, d = LAYOUTS[name]
    nq, nk = sum(rows[0]), sum(keys[0])
    q, do = _random(dev, nq, hq, d), _random(dev, nq, hq, d, seed=1)
    k, v = _random(dev, nk, hk, d, seed=2), _random(dev, nk, hk, d, seed=3)
    most = max(map(max, rows)), max(map(max, keys))
    cus = [(_i32(dev, *np.cumsum([0, *r]).tolist()), _i32(dev, *np.cumsum([0, *x]).tolist()))
           for r, x in zip(rows, keys)]

    def run(cu_q, cu_k, ws, bws):
        o, lse = h3.varlen_cross_attn_fwd(q, k, v, cu_q, cu_k, *most, return_lse=True, workspace=ws)
        return (o, lse, *h3.varlen_cross_attn_bwd(do, q, k, v, o, lse, cu_q, cu_k, *most, workspace=bws))

    want = [[t.clone() for t in run(*cu, None, None)] for cu in cus]
    assert not torch.equal(want[0][0], want[1][0])
    sizes = (3, *most, nq, nk, hq, hk, d)
    ws, bws = (torch.zeros(f(*sizes), dtype=torch.uint8, device=dev)
               for f in (h3.varlen_cross_attn_workspace_size, h3.varlen_cross_attn_bwd_workspace_size))
    cu_q, cu_k = (t.clone() for t in cus[0])
    results = []

    def both():
        for a, b in cus:
            cu_q.copy_(a), cu_k.copy_(b)
            results.append(run(cu_q, cu_k, ws, bws))

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
        for _ in range(5):
            for r in results:
                for t in r:
                    t.fill_(7.0)
            graph.replay()
            assert all(torch.equal(a, b) for r, w in zip(results, want) for a, b in zip(r, w))
    else:
        for _ in range(20):
            both()
        for i, r in enumerate(results):
            assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2]))
    assert h3.get_device_error(dev) == 0


def _overlapping(dev, segments, rows):
    """Every other segment is all rows, those between run backwards."""
    return _i32(dev, *[(i % 2) * rows for i in range(segments + 1)])


def test_overlapping_query_segments_are_refused(h3, dev):
    # 32 segments of all 4,096 rows: more tiles than 4,096 rows and 64 segments can hold
    n, s = 4096, 64
    q, k, do = _random(dev, n, 2, 64), _random(dev, n, 2, 64, seed=1), _random(dev, n, 2, 64, seed=2)
    even = _i32(dev, *range(0, n + 1, n // s))
    want, lse = h3.varlen_cross_attn_fwd(q, k, k, even, even, n // s, n // s, return_lse=True)
    out, l2 = torch.full_like(q, 7.0), torch.full_like(lse, 7.0)
    assert h3.get_device_error(dev) == 0
    h3.varlen_cross_attn_fwd(q, k, k, _overlapping(dev, s, n), even, n, n // s, out=out, lse=l2)
    assert h3.get_device_error(dev) == BAD_OFFSETS
    assert (out == 7.0).all() and (l2 == 7.0).all()
    grads = [torch.full_like(q, 7.0) for _ in range(3)]
    for cu_q, cu_k, most in ((_overlapping(dev, s, n), even, (n, n // s)), (even, _overlapping(dev, s, n), (n // s, n))):
        h3.varlen_cross_attn_bwd(do, q, k, k, want, lse, cu_q, cu_k, *most, dq=grads[0], dk=grads[1], dv=grads[2])
        assert h3.get_device_error(dev) == BAD_OFFSETS
        assert all((g == 7.0).all() for g in grads)
    again, l3 = h3.varlen_cross_attn_fwd(q, k, k, even, even, n // s, n // s, return_lse=True)
    assert h3.get_device_error(dev) == 0 and torch.equal(again, want) and torch.equal(l3, lse)


def test_overlapping_packed_segments_are_refused(h3, dev):
    n, s = 4096, 64
    q = _random(dev, n, 2, 64)
    out, lse = torch.full_like(q, 7.0), torch.full((2, n), 7.0, device=dev)
    assert h3.get_device_error(dev) == 0
    h3.varlen_attn_fwd(q, q, q, _overlapping(dev, s, n), n, out=out, lse=lse)
    assert h3.get_device_error(dev) == BAD_OFFSETS
    assert (out == 7.0).all() and (lse == 7.0).all()
    h3.varlen_attn_fwd(q, q, q, _i32(dev, *range(0, n + 1, n // s)), n // s, out=out, lse=lse)
    assert h3.get_device_error(dev) == 0 and not (out == 7.0).any() and not (lse == 7.0).any()


def test_more_segments_than_threads_of_the_plan(h3, dev):
    n = 2500  # three to a thread
    c = Case([(7 * i) % 23 for i in range(n)], [(5 * i) % 31 for i in range(n)], 2, 2, 64, seed=3)
    args, where = c.on(dev)
    out, lse = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)
    check_forward(c, out, lse)
    out, lse = _given(c, dev)
    got = h3.varlen_cross_attn_bwd(c.do.to(dev), **args, out=out, lse=lse, **where)
    assert h3.get_device_error(dev) == 0
    check_gradient(c, got)


def test_as_many_segments_as_are_allowed(h3, dev):
    # one row and one key each: the weight is 1, so o = v and dv = do exactly, and dS = dP - rowsum(do * o) is
    # the difference of two fp32 sums of the same 64 products
    n = 65535
    q, do, v = (_random(dev, n, 1, 64, seed=s) for s in range(3))
    cu = torch.arange(n + 1, dtype=torch.int32, device=dev)
    out, lse = h3.varlen_cross_attn_fwd(q, q, v, cu, cu, 17, 1, return_lse=True)  # 17: not the form for tokens
    assert torch.equal(out, v)
    dq, dk, dv = h3.varlen_cross_attn_bwd(do, q, q, v, out, lse, cu, cu, 17, 1)
    assert h3.get_device_error(dev) == 0
    assert torch.equal(dv, do)
    # two sums of 64 terms, 2^-24 relative a step, of sum |do v| < 100 (5 standard deviations over all rows),
    # times scale |q| <= 0.125 * 6: 2 * 64 * 6e-8 * 100 * 0.75 = 6e-4
    assert dq.float().abs().max() < 1e-3 and dk.float().abs().max() < 1e-3


def _chunks(sms, slots, tiles, steps):
    """The gradient plan's rule: chunks of the tiles behind the whole waves."""
    rest, best = tiles % sms, (float("inf"), 0)
    for c in range(1, 17):
        cost = np.float32(-(-rest * c // sms)) * (np.float32(steps) / np.float32(c) + np.float32(3))
        cost += np.float32(2 if c > 1 else 0)
        if c > 1 and rest * c > slots:
            continue
        best = min(best, (float(cost), c))
    return best[1]


def test_work_of_the_plan_past_32_bits(h3, dev):
    """2^32 steps in all.  The loaders stop after three tiles, as in test_gpu_cross_timeout.py, so the two
    product kernels leave by their waits' limit; the plan before them is complete."""
    nq, nk, heads = 1 << 20, 1 << 24, 4
    q, k = (torch.zeros(n, h, 64, dtype=torch.bfloat16, device=dev) for n, h in ((nq, heads), (nk, 1)))
    lse = torch.zeros(heads, nq, device=dev)
    size = h3.varlen_cross_attn_bwd_workspace_size(1, nq, nk, nq, nk, heads, 1, 64)
    ws = torch.zeros(size, dtype=torch.uint8, device=dev)
    assert h3.get_device_error(dev) == 0
    h3.set_wait_limit_ns(20_000_000)
    h3.debug_stall_loads(3)
    try:
        h3.varlen_cross_attn_bwd(q, q, k, k, q, lse, _i32(dev, 0, nq), _i32(dev, 0, nk), nq, nk, workspace=ws)
        torch.cuda.synchronize()
    finally:
        h3.debug_stall_loads(-1)
        h3.set_wait_limit_ns(0)
    assert h3.get_device_error(dev) == TIMEOUT
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    q_tiles, k_tiles = nq // 128 * heads, nk // 128
    slots = 4 * 152
    items_q, items_k, whole_q, whole_k, chunks_q, chunks_k = ws[:24].view(torch.int32).tolist()
    assert (whole_q, whole_k) == (q_tiles - q_tiles % sms, k_tiles - k_tiles % sms)
    assert chunks_q == _chunks(sms, slots, q_tiles, nk // 128) > 1
    assert chunks_k == _chunks(sms, slots, k_tiles, heads * nq // 128) > 1
    assert items_q == whole_q + q_tiles % sms * chunks_q and items_k == whole_k + k_tiles % sms * chunks_k
