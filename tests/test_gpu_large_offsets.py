"""Elements past 2^31 of a tensor: the last rows of large norm inputs and of a large key/value buffer.
Checked against the same rows in small tensors, bit for bit."""
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


def _i32(dev, *v):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def test_norm_rows(h3, dev):
    n, heads, tail = 430_000, 40, 50
    x = torch.zeros(n, heads, 128, dtype=torch.bfloat16, device=dev)
    assert x.numel() > 2 ** 31
    last = torch.randn(tail, heads, 128, device=dev).to(torch.bfloat16)
    x[-tail:] = last
    w = torch.linspace(0.5, 1.5, 128, device=dev)
    pos, tag = torch.rand(n, 3, device=dev) * 100, torch.ones(n, dtype=torch.uint8, device=dev)
    small = dict(pos=pos[-tail:].contiguous(), tag=tag[-tail:].contiguous())
    y, _ = h3.qk_norm_rope(x, None, w, None, pos=pos, tag=tag)
    want, _ = h3.qk_norm_rope(last, None, w, None, **small)
    assert torch.equal(y[-tail:], want)
    dx, _, _, _ = h3.qk_norm_rope_bwd(y, None, x, None, w, None, pos=pos, tag=tag, dq=y)
    ref, _, _, _ = h3.qk_norm_rope_bwd(want, None, last, None, w, None, **small)
    assert torch.equal(dx[-tail:], ref)


@pytest.mark.parametrize("rows", [1, 40])  # the key-streaming kernel and the tiled one
def test_last_keys_of_a_large_buffer(h3, dev, rows):
    n, heads, keys = 290_000, 64, 700
    kv = torch.zeros(n, 2 * heads * 64, dtype=torch.bfloat16, device=dev)
    assert kv.numel() > 2 ** 31
    k, v = kv[:, :heads * 64].view(n, heads, 64), kv[:, heads * 64:].view(n, heads, 64)
    last = torch.randn(2, keys, heads, 64, device=dev).to(torch.bfloat16)
    k[-keys:], v[-keys:] = last[0], last[1]
    q = torch.randn(2 * rows, heads, 64, device=dev).to(torch.bfloat16)
    cu_q = _i32(dev, 0, rows, 2 * rows)
    used = _i32(dev, 3, keys)
    out, lse = h3.varlen_cross_attn_fwd(q, k, v, cu_q, _i32(dev, 0, n - keys, n), rows, keys, return_lse=True,
                                        seqused_k=used)
    # the same segments (hence the same split of the work) in a small buffer
    small = torch.cat([kv[:3], kv[-keys:]]).contiguous()
    ks, vs = small[:, :heads * 64].view(-1, heads, 64), small[:, heads * 64:].view(-1, heads, 64)
    cu_s = _i32(dev, 0, 3, 3 + keys)
    want, wlse = h3.varlen_cross_attn_fwd(q, ks, vs, cu_q, cu_s, rows, keys, return_lse=True, seqused_k=used)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    do = torch.randn_like(q)
    dq, dk, dv = h3.varlen_cross_attn_bwd(do, q, k, v, out, lse, cu_q, _i32(dev, 0, n - keys, n), rows, keys,
                                          seqused_k=used)
    ref = h3.varlen_cross_attn_bwd(do, q, ks, vs, want, wlse, cu_q, cu_s, rows, keys, seqused_k=used)
    assert torch.equal(dq, ref[0])
    # one query tile a head: no key tile's sum is cut
    assert torch.equal(dk[-keys:], ref[1][-keys:]) and torch.equal(dv[-keys:], ref[2][-keys:])
    assert h3.get_device_error(dev) == 0
