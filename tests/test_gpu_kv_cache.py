"""Paged key/value cache on the GPU: what is written is what the format says, bit for bit, and reads back
as the values it stands for (the steps are exact but for the one rounding to e4m3, so nothing is tolerated)."""
import numpy as np
import pytest
import torch

import oracle
from oracle.norm import _f64

pytest_gpu = pytest.mark.gpu


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


# ---- refusals (no GPU) -------------------------------------------------------------------------------


@pytest.mark.parametrize("kw, status", [
    (dict(num_segments=-1), 2), (dict(num_segments=65536), 2), (dict(capacity=-1), 2), (dict(num_heads=0), 2),
    (dict(num_heads=1 << 20), 2), (dict(head_dim=96), 4), (dict(cache_type=0), 2), (dict(cache_type=3), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2), (dict(num_pages=-1), 2),
    (dict(max_pages=-1), 2), (dict(k_stride=64), 2), (dict(v_stride=132), 8), (dict(cache_type=1), 1),
])
def test_c_abi_refuses(h3, kw, status):
    import ctypes as C

    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    base = dict(num_segments=1, capacity=2, num_heads=2, head_dim=64, cache_type=2, page_size=16, num_pages=1, max_pages=1)
    d = h3._KvCacheDesc(**{**base, **kw})
    lib = h3.load_library()
    assert lib.h3_kv_cache_write(C.byref(d), p, p, p, p, p, p, p, p, p, None) == status
    assert lib.h3_kv_cache_read(C.byref(d), p, p, p, p, p, p, p, p, p, None) == status


def test_c_abi_refuses_pointers(h3):
    import ctypes as C

    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    d = h3._KvCacheDesc(num_segments=1, capacity=2, num_heads=2, head_dim=64, cache_type=2, page_size=16, num_pages=1,
                        max_pages=1)
    lib = h3.load_library()
    assert lib.h3_kv_cache_write(None, *(p,) * 9, None) == 1
    for i in range(9):
        a = [p] * 9
        a[i] = None
        assert lib.h3_kv_cache_write(C.byref(d), *a, None) == 1, i
        if i not in (4, 5):  # scales are bytes
            a[i] = C.c_void_p(p.value + 2)
            assert lib.h3_kv_cache_write(C.byref(d), *a, None) == 8, i


def test_binding_refuses(h3):
    kv = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache, table = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32)
    cu, start = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    e4, sc = cache.to(torch.float8_e4m3fn), torch.zeros(3, 2, 16, dtype=torch.uint8)
    base = dict(k=kv, v=kv, k_cache=cache, v_cache=cache, block_table=table, cu_seqlens=cu, start=start)
    for error, kw in [
        (TypeError, dict(k=kv.float())), (ValueError, dict(v=kv[:3])), (ValueError, dict(k=kv[:, :1], v=kv[:, :1])),
        (TypeError, dict(k_cache=cache.half())), (TypeError, dict(v_cache=e4)), (ValueError, dict(k_cache=cache[0])),
        (ValueError, dict(v_cache=cache[:2])), (ValueError, dict(k_scale=sc, v_scale=sc)),
        (ValueError, dict(k_cache=e4, v_cache=e4)), (ValueError, dict(k_cache=e4, v_cache=e4, k_scale=sc, v_scale=sc[:2])),
        (TypeError, dict(k_cache=e4, v_cache=e4, k_scale=sc.int(), v_scale=sc)), (TypeError, dict(block_table=table.long())),
        (ValueError, dict(block_table=table[0])), (ValueError, dict(block_table=torch.zeros(2, 2, dtype=torch.int32))),
        (TypeError, dict(cu_seqlens=cu.long())), (ValueError, dict(start=torch.zeros(2, dtype=torch.int32))),
        (ValueError, dict(k_cache=cache.transpose(1, 2), v_cache=cache.transpose(1, 2))),
    ]:
        with pytest.raises(error):
            h3.kv_cache_write(**{**base, **kw})
    with pytest.raises(ValueError):
        h3.kv_cache_read(cache, cache, table, cu, start)
    with pytest.raises(ValueError):
        h3.kv_cache_read(cache, cache, table, cu, start, k_out=kv)


# ---- GPU ---------------------------------------------------------------------------------------------

# rows and starts of the segments, heads, head_dim, page, e4m3, fused projection, extra rows
SHAPES = [
    ([1], [0], 1, 64, 16, False, False, 0),
    ([1], [0], 1, 64, 16, True, False, 0),
    ([1, 1, 1, 1], [15, 16, 0, 301], 8, 128, 16, True, True, 0),
    ([3, 0, 20], [30, 5, 127], 2, 128, 32, True, False, 3),
    ([3, 0, 20], [30, 5, 127], 3, 64, 32, False, True, 3),
    ([130, 257], [1, 255], 5, 128, 64, True, True, 0),
    ([0, 700, 0], [0, 3, 9], 40, 128, 128, True, True, 1),
    ([513, 64], [0, 1000], 7, 64, 256, True, False, 0),
    ([513, 64], [0, 1000], 1, 128, 256, False, True, 5),
    ([2100], [77], 2, 64, 16, True, True, 0),
]


def _case(dev, shape, seed=0):
    rows, start, h, d, page, e4m3, fused, extra = shape
    gen = torch.Generator(device=dev).manual_seed(seed)
    n = sum(rows) + extra
    wide = torch.randn(n, (3 if fused else 2) * h * d, device=dev, generator=gen)
    wide *= torch.exp(torch.randn(n, 1, device=dev, generator=gen) * 4)  # rows of all sizes
    wide = wide.to(torch.bfloat16)
    k, v = wide[:, :h * d].view(n, h, d), wide[:, -h * d:].view(n, h, d)
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    counts = [(a + b + page - 1) // page for a, b in zip(rows, start)]
    ids = torch.randperm(sum(counts) + 2, device=dev, generator=gen).to(torch.int32)
    table = torch.full((len(rows), max(counts) + 1), -7, dtype=torch.int32, device=dev)
    at = 0
    for g, c in enumerate(counts):
        table[g, :c] = ids[at:at + c]
        at += c
    pages = sum(counts) + 2
    cache = {}
    for name in ("k_cache", "v_cache"):
        t = torch.full((pages, h, page, d), 3.0, dtype=torch.bfloat16, device=dev)
        cache[name] = t.to(torch.float8_e4m3fn) if e4m3 else t
    if e4m3:
        for name in ("k_scale", "v_scale"):
            cache[name] = torch.full((pages, h, page), 99, dtype=torch.uint8, device=dev)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=dev)
    return k, v, cache, table, cu, torch.tensor(start, dtype=torch.int32, device=dev)


def _slots(shape, table, cu):
    rows, start, page = shape[0], shape[1], shape[4]
    out = []
    for g, n in enumerate(rows):
        out += [(int(table[g, (start[g] + i) // page]), (start[g] + i) % page) for i in range(n)]
    return out


@pytest_gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_write_then_read(h3, dev, shape):
    k, v, cache, table, cu, start = _case(dev, shape)
    e4m3, n = shape[5], sum(shape[0])
    h3.kv_cache_write(k, v, cache["k_cache"], cache["v_cache"], table, cu, start, cache.get("k_scale"), cache.get("v_scale"))
    k_out, v_out = (torch.full(k.shape, 5.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    got = h3.kv_cache_read(cache["k_cache"], cache["v_cache"], table, cu, start, k_scale=cache.get("k_scale"),
                           v_scale=cache.get("v_scale"), k_out=k_out, v_out=v_out)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    slots = _slots(shape, table.cpu(), cu.cpu())
    untouched = torch.ones(cache["k_cache"].shape[0], shape[4], dtype=torch.bool)
    for p, r in slots:
        untouched[p, r] = False
    for x, back, name in ((k, got[0], "k"), (v, got[1], "v")):
        assert torch.all(back[n:] == 5.0)  # rows past the last segment
        held = cache[name + "_cache"].cpu()
        want = _f64(x[:n])
        if e4m3:
            scale = cache[name + "_scale"].cpu()
            e = oracle.e4m3_scale(want)
            q = oracle.e4m3_round(want / np.ldexp(1.0, e)[..., None])
            for i, (p, r) in enumerate(slots):
                assert np.array_equal(scale[p, :, r].numpy(), e[i] + 127)
                assert np.array_equal(held[p, :, r].double().numpy(), q[i])
            want = q * np.ldexp(1.0, e)[..., None]
            assert torch.all(scale.transpose(1, 2)[untouched] == 99)
        else:
            for i, (p, r) in enumerate(slots):
                assert np.array_equal(held[p, :, r].double().numpy(), want[i])
        assert torch.all(held.float().transpose(1, 2)[untouched] == 3.0)
        assert np.array_equal(_f64(back[:n]), want)


@pytest_gpu
def test_rows_at_the_borders_of_the_scale(h3, dev):
    """Largest values next to 448 * 2^e on both sides, zeros, the smallest and the largest bf16, Inf and NaN."""
    rows = []
    for most in (448.0, 450.0, 446.0, 1.75, 1.7578125, 0.0, 2.0 ** -126, 2.0 ** -133, 3.3895e38, 1e-30):
        r = torch.linspace(-1, 1, 64) * most
        rows.append(r)
    x = torch.stack(rows).to(torch.bfloat16).view(-1, 1, 64).to(dev)
    n = x.shape[0]
    cache = torch.zeros(1, 1, 16, 64, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.zeros(1, 1, 16, dtype=torch.uint8, device=dev)
    where = (cache, cache.clone(), torch.zeros(1, 1, dtype=torch.int32, device=dev),
             torch.tensor([0, n], dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev))
    h3.kv_cache_write(x, x, *where, k_scale=scale, v_scale=scale.clone())
    back, _ = h3.kv_cache_read(*where, num_rows=n, k_scale=scale, v_scale=scale)
    # bf16 holds every value but one: 3.3895e38 = 255 * 2^120 rounds to 256 * 2^120 = 2^128 (steps of 16 there), which
    # lies past the largest bf16, (2 - 2^-7) * 2^127, and so is Inf in bf16
    want = oracle.e4m3_row_values(x)
    assert np.abs(want[8]).max() == 2.0 ** 128 and np.array_equal(_f64(back), np.where(want == 2.0 ** 128, np.inf, np.where(
        want == -2.0 ** 128, -np.inf, want)))
    assert np.array_equal(scale[0, 0, :n].cpu().numpy(), oracle.e4m3_scale(x)[:, 0] + 127)
    y = torch.ones(2, 1, 64, dtype=torch.bfloat16, device=dev)
    y[0, 0, 3], y[1, 0, 4] = float("nan"), float("inf")
    where = where[:3] + (torch.tensor([0, 2], dtype=torch.int32, device=dev), where[4])
    h3.kv_cache_write(y, y, *where, k_scale=scale, v_scale=scale.clone())
    back, _ = h3.kv_cache_read(*where, num_rows=2, k_scale=scale, v_scale=scale)
    back = back.float().cpu()
    assert torch.isnan(back[0, 0]).all() and scale[0, 0, 0] == 255  # a row with a NaN is one throughout
    assert back[1, 0, 4] == float("inf") and torch.all(back[1, 0, torch.arange(64) != 4] == 0.0)  # 1 next to Inf is nothing
    assert h3.get_device_error(dev) == 0


@pytest_gpu
def test_bad_places_are_skipped_and_recorded(h3, dev):
    """Positions past the table, page ids out of range, offsets out of order: nothing else is touched."""
    shape = ([40, 40], [0, 0], 2, 64, 16, False, False, 0)
    k, v, cache, table, cu, start = _case(dev, shape, seed=3)
    # (where a row also meets a table entry that is no page, either is the first)
    for bad, status in (("page", [12]), ("negative", [12]), ("position", [3, 12]), ("start", [3]), ("falling", [3, 12]),
                        ("long", [3])):
        kc, vc, t, c, s = cache["k_cache"].clone(), cache["v_cache"].clone(), table.clone(), cu.clone(), start.clone()
        if bad == "page":
            t[0, 1] = kc.shape[0]
        elif bad == "negative":
            t[0, 1] = -1
        elif bad == "position":
            s[0] = 16 * t.shape[1] - 10
        elif bad == "start":
            s[0] = -5
        elif bad == "falling":
            c[1] = 90
        else:
            c[2] = 90
        h3.kv_cache_write(k, v, kc, vc, t, c, s)
        torch.cuda.synchronize()
        assert h3.get_device_error(dev) in status, bad
        if bad in ("page", "negative"):
            good = cache["k_cache"].clone()
            h3.kv_cache_write(k, v, good, vc.clone(), table, cu, start)
            good[table[0, 1].long()] = cache["k_cache"][table[0, 1].long()]
            assert torch.equal(kc, good)
        assert h3.get_device_error(dev) == 0


@pytest_gpu
def test_empty_calls(h3, dev):
    cache = torch.full((2, 1, 16, 64), 3.0, dtype=torch.bfloat16, device=dev)
    none = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    h3.kv_cache_write(none, none, cache, cache, torch.zeros(1, 1, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32))
    h3.kv_cache_write(none, none, cache, cache, torch.zeros(0, 1, **i32), torch.zeros(1, **i32), torch.zeros(0, **i32))
    some = torch.ones(4, 1, 64, dtype=torch.bfloat16, device=dev)
    h3.kv_cache_write(some, some, cache, cache, torch.zeros(1, 1, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32))
    torch.cuda.synchronize()
    assert torch.all(cache == 3.0) and h3.get_device_error(dev) == 0


@pytest_gpu
def test_cache_past_2_31_elements(h3, dev):
    """Pages whose first element lies past 2^31 and 2^32."""
    h, d, page, pages = 8, 128, 256, 17000  # 4.46e9 elements
    cache = torch.empty(pages, h, page, d, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(pages, h, page, dtype=torch.uint8, device=dev)
    table = torch.tensor([[pages - 1, 8200, 0]], dtype=torch.int32, device=dev)
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(700, h, d, device=dev, generator=gen).to(torch.bfloat16)
    cu, start = torch.tensor([0, 700], dtype=torch.int32, device=dev), torch.tensor([20], dtype=torch.int32, device=dev)
    v_cache, v_scale = cache.clone(), scale.clone()
    h3.kv_cache_write(x, x * 2, cache, v_cache, table, cu, start, scale, v_scale)
    k, v = h3.kv_cache_read(cache, v_cache, table, cu, start, num_rows=700, k_scale=scale, v_scale=v_scale)
    assert h3.get_device_error(dev) == 0
    want = oracle.e4m3_row_values(x)
    assert np.array_equal(_f64(k), want) and np.array_equal(_f64(v), 2 * want)
    assert torch.equal(cache[pages - 1, :, 20:].float(), cache.view(torch.uint8)[pages - 1, :, 20:].view(torch.float8_e4m3fn).float())


@pytest_gpu
def test_captured_and_replayed(h3, dev):
    shape = ([1] * 6, [99] * 6, 4, 128, 16, True, True, 0)  # pages for 100 tokens each
    k, v, cache, table, cu, start = _case(dev, shape, seed=5)
    start.copy_(torch.tensor([4, 15, 16, 31, 0, 99]))
    args = (cache["k_cache"], cache["v_cache"], table, cu, start)
    scales = dict(k_scale=cache["k_scale"], v_scale=cache["v_scale"])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        h3.kv_cache_write(k, v, *args, **scales)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        h3.kv_cache_write(k, v, *args, **scales)
        back = h3.kv_cache_read(*args, num_rows=6, **scales)
    k.mul_(-3.0)
    for step in range(3):  # the stream grows by a token a replay
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(_f64(back[0]), oracle.e4m3_row_values(k)), step
        start.add_(1).remainder_(100)
    assert h3.get_device_error(dev) == 0
