"""Calls from threads: a new thread has no CUDA context until something gives it one, and each call
must; several threads at once, each on a stream and with workspaces of its own, get the results of one."""
import threading

import pytest
import torch

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


def _calls(h3, dev):
    g = torch.Generator(device=dev).manual_seed(5)
    x = lambda rows, heads: torch.randn(rows, heads, 64, device=dev, generator=g).to(torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    q, k, v, do, w = x(500, 4), x(500, 4), x(500, 4), x(500, 4), torch.rand(64, device=dev, generator=g) + 0.5
    cu, one = i32(0, 200, 500), i32(0, 1, 2)
    grid = [x(4 * 8 * 8, 2) for _ in range(3)]
    o, lse = h3.varlen_cross_attn_fwd(q, k, v, cu, cu, 300, 300, return_lse=True)
    torch.cuda.synchronize()
    return {
        "norm": lambda: h3.qk_norm_rope(q, k, w, w),
        "norm_bwd": lambda: h3.qk_norm_rope_bwd(do, do, q, k, w, w),
        "packed": lambda: (h3.varlen_attn_fwd(q, k, v, cu, max_seqlen=300),),
        "window": lambda: (h3.window_attn_fwd(*grid, (4, 8, 8), (2, 4, 4), (1, 2, 2)),),
        "cross": lambda: (h3.varlen_cross_attn_fwd(q, k, v, cu, cu, 300, 300),),
        "cross_tokens": lambda: (h3.varlen_cross_attn_fwd(q[:2], k, v, one, cu, 1, 300),),
        "cross_bwd": lambda: h3.varlen_cross_attn_bwd(do, q, k, v, o, lse, cu, cu, 300, 300),
    }


NAMES = ["norm", "norm_bwd", "packed", "window", "cross", "cross_tokens", "cross_bwd"]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_first_call_of_a_new_thread(h3, dev, name):
    call = _calls(h3, dev)[name]
    expected = call()
    torch.cuda.synchronize()
    got = []
    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert len(got) == 1, "the call raised"
    assert _same(got[0], expected)


def test_threads_on_streams_of_their_own(h3, dev):
    calls = _calls(h3, dev)
    expected = {n: calls[n]() for n in NAMES}
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream(dev)):
            results = [(n, calls[n]()) for _ in range(20) for n in NAMES]
            torch.cuda.current_stream().synchronize()
            bad.extend(n for n, r in results if not _same(r, expected[n]))
            bad.append(None)  # got here

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == [None] * 4
    assert h3.get_device_error(dev) == 0
