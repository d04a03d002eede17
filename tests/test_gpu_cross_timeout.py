"""The cross attention kernels' bounded waits, made to run out on purpose: as for the attention kernels
in test_gpu_timeout.py, the loaders stop after three tiles and the limit is 20 ms, so the waits of the
warps that consume those tiles end by their limit in the middle of an otherwise valid launch.  Nothing
faults or hangs: no load is issued that would not be issued normally, and what the unwinding kernels
wait for completes by itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TIMEOUT = 7  # H3_ERR_TIMEOUT


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


def _inputs(dev, rows, keys, heads):
    gen = torch.Generator(device=dev).manual_seed(rows)
    x = lambda n: torch.randn(n, heads, 128, device=dev, generator=gen).to(torch.bfloat16)
    i32 = lambda v: torch.tensor([0, v], dtype=torch.int32, device=dev)
    return x(rows), x(keys), x(keys), x(rows), (i32(rows), i32(keys), rows, keys)


def _run_out(h3, dev, run, shapes):
    """run(outputs) launches one call; shapes: (shape, dtype) of its outputs."""
    make = lambda v: [torch.full(s, v, dtype=t, device=dev) for s, t in shapes]
    assert h3.get_device_error(dev) == 0
    ref = make(5.0)
    run(ref)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    h3.set_wait_limit_ns(20_000_000)
    h3.debug_stall_loads(3)
    try:
        run(make(0.0))
        torch.cuda.synchronize()  # the launch ends although its waits ran out
        later = make(7.0)
        run(later)  # leaves at once while the timeout is recorded
        torch.cuda.synchronize()
    finally:
        h3.debug_stall_loads(-1)
        h3.set_wait_limit_ns(0)
    assert all((x == 7.0).all() for x in later)
    assert h3.get_device_error(dev) == TIMEOUT
    assert h3.get_device_error(dev) == 0
    again = make(5.0)
    run(again)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    assert all(torch.equal(x, y) for x, y in zip(again, ref))


@pytest.mark.parametrize("rows, keys, heads", [(9000, 600, 8),     # whole items, several a CTA
                                               (300, 9000, 2)])    # every item cut and merged
def test_forward_timeout_unwinds(h3, dev, rows, keys, heads):
    q, k, v, _, where = _inputs(dev, rows, keys, heads)
    _run_out(h3, dev, lambda o: h3.varlen_cross_attn_fwd(q, k, v, *where, out=o[0], lse=o[1]),
             [(q.shape, torch.bfloat16), ((heads, rows), torch.float32)])


@pytest.mark.parametrize("rows, keys, heads", [(9000, 600, 8), (3000, 2500, 8)])
def test_backward_timeout_unwinds(h3, dev, rows, keys, heads):
    q, k, v, do, where = _inputs(dev, rows, keys, heads)
    out, lse = h3.varlen_cross_attn_fwd(q, k, v, *where, return_lse=True)
    _run_out(h3, dev,
             lambda o: h3.varlen_cross_attn_bwd(do, q, k, v, out, lse, *where, dq=o[0], dk=o[1], dv=o[2]),
             [(x.shape, torch.bfloat16) for x in (q, k, v)])
