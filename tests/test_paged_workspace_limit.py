"""The workspace that paged_attn_fwd allocates for a long chunk over an e4m3 cache: with room for the cache's tokens in
bf16, or the least one where the caller's limit or the device's memory do not allow that; the results are the same."""
import pytest
import torch


@pytest.fixture(scope="module")
def h3():
    import __graft_entry__

    __graft_entry__.build()
    import packed_varlen_attention_modality_gb300 as h3

    h3.load_library()
    return h3


def _call(dev, e4m3=True, rows=600, tokens=900, heads=2, d=64, page=32):
    gen = torch.Generator().manual_seed(1)
    pages = -(-tokens // page)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    cache = lambda: torch.randn(pages, heads, page, d, generator=gen).to(kind).to(dev)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    a = dict(q=torch.randn(rows, heads, d, generator=gen).to(torch.bfloat16).to(dev), k_cache=cache(), v_cache=cache(),
             block_table=torch.randperm(pages, generator=gen).to(torch.int32).view(1, -1).to(dev),
             cu_seqlens_q=i32(0, rows), seqused_k=i32(tokens), max_seqlen_q=rows, max_seqlen_k=tokens, causal_block=1)
    if e4m3:
        for name in ("k_scale", "v_scale"):
            a[name] = torch.randint(120, 130, (pages, heads, page), generator=gen, dtype=torch.uint8).to(dev)
    return a


def _sizes(h3, a):
    return [h3.paged_attn_workspace_size(1, a["max_seqlen_q"], a["max_seqlen_k"], a["q"].shape[0], a["q"].shape[1],
                                         a["k_cache"].shape[1], a["q"].shape[2], a["k_cache"].shape[2], e4m3=e,
                                         max_pages=a["block_table"].shape[1]) for e in (False, True)]


@pytest.fixture
def spy(h3, monkeypatch):
    """Workspace sizes of the calls, which end before the library; allocations past `room` bytes fail."""
    seen, room, empty = [], [None], torch.empty

    def limited(*size, **kw):
        n = size[0] if len(size) == 1 and isinstance(size[0], int) else 0
        if room[0] is not None and n > room[0]:
            raise torch.OutOfMemoryError("no room")
        return empty(*size, **kw)

    monkeypatch.setattr(h3, "_launch", lambda fn, where, dev, *args: seen.append(args[-1]))
    monkeypatch.setattr(torch, "empty", limited)
    return seen, room


def test_limit_and_failed_allocations(h3, spy):
    seen, room = spy
    a = _call("cpu")
    least, most = _sizes(h3, a)
    assert least < most

    def size(**kw):
        seen.clear()
        h3.paged_attn_fwd(**a, **kw)
        return seen[0]

    assert size() == most and size(workspace_limit=most) == most
    for limit in (most - 1, least, 0):
        assert size(workspace_limit=limit) == least, limit
    assert size(workspace=torch.zeros(least + 7, dtype=torch.uint8), workspace_limit=0) == least + 7
    room[0] = most - 1
    assert size() == least
    room[0] = least - 1
    with pytest.raises(torch.OutOfMemoryError):
        size()


def test_calls_that_unpack_nothing(h3, spy):
    seen, room = spy
    for a in (_call("cpu", e4m3=False), _call("cpu", rows=500), _call("cpu", rows=2)):
        least, _ = _sizes(h3, a)
        for kw in ({}, dict(workspace_limit=0)):
            seen.clear()
            h3.paged_attn_fwd(**a, **kw)
            assert seen[0] == least


@pytest.mark.gpu
def test_same_results(h3):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dev = torch.device("cuda", 0)
    a = _call(dev, rows=700, tokens=3000)
    least, most = _sizes(h3, a)
    want, wl = h3.paged_attn_fwd(**a, return_lse=True)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got, gl = h3.paged_attn_fwd(**a, return_lse=True, workspace_limit=least)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < most
    assert torch.equal(got, want) and torch.equal(gl, wl) and h3.get_device_error(dev) == 0
