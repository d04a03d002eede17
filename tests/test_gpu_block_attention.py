"""The operators as a model's block uses them: packed self attention behind the norm and rotation of a
fused projection, cross attention to text states behind the norm alone, and the gradients of both back
into the fused projections.

Tolerance: against fp64 from the raw inputs, in the relative 2-norm.  On the way to a gradient about
ten values are rounded to bf16 one after the other (y of q and k, P, o, dS, dq and dk, dx ...), each by at
most 2^-8 of itself; the score, at the size that normed rows give it, passes its error on at most
twofold: 10 * 2 * 2^-8 = 0.08.  Outputs see half of them: 0.04.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


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


H, HK, D = 6, 2, 64
SEG, TEXT, USED = [40, 17, 200], [30, 30, 30], [30, 0, 11]


def _block(seed=0):
    rng = np.random.default_rng(seed)
    n, m = sum(SEG), sum(TEXT)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16)
    x = dict(qkv=bf(n, 3 * H * D), q2=bf(n, H * D), kv=bf(m, 2 * HK * D), do1=bf(n, H, D), do2=bf(n, H, D))
    for name in ("w_q", "w_k", "w_q2", "w_k2"):
        x[name] = torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).float()
    pos = np.stack([rng.integers(0, 30, n), rng.integers(0, 9, n), rng.integers(0, 9, n)], 1).astype(np.float32)
    x["pos"], x["tag"] = torch.from_numpy(pos), torch.from_numpy((np.arange(n) % 3).astype(np.uint8))
    cu = np.concatenate([[0], np.cumsum(SEG)]).astype(np.int32)
    x["cu"], x["frames"] = torch.from_numpy(cu), torch.tensor([0.0, 119.0, 238.0])
    x["cu_text"] = torch.from_numpy(np.concatenate([[0], np.cumsum(TEXT)]).astype(np.int32))
    x["used"] = torch.tensor(USED, dtype=torch.int32)
    return x


def _run(h3, x):
    """Forward and backward with the operators; every gradient lands in its fused projection."""
    n, m, hd, kd = x["qkv"].shape[0], x["kv"].shape[0], H * D, HK * D
    qkv, kv = x["qkv"], x["kv"]
    q, k = qkv[:, :hd].view(n, H, D), qkv[:, hd:2 * hd].view(n, H, D)
    rot = dict(pos=x["pos"], tag=x["tag"], cu_requests=x["cu"], start_frames=x["frames"])
    v = qkv[:, 2 * hd:].reshape(n, H, D).contiguous()
    yq, yk = h3.qk_norm_rope(q, k, x["w_q"], x["w_k"], **rot)
    o1, lse1 = h3.varlen_attn_fwd(yq, yk, v, x["cu"], max(SEG), return_lse=True)
    q2 = x["q2"].view(n, H, D)
    k2, v2 = kv[:, :kd].view(m, HK, D), kv[:, kd:].view(m, HK, D)
    yq2, _ = h3.qk_norm_rope(q2, None, x["w_q2"], None)
    yk2, _ = h3.qk_norm_rope(k2, None, x["w_k2"], None)
    text = (x["cu"], x["cu_text"], max(SEG), max(USED), x["used"])
    o2, lse2 = h3.varlen_cross_attn_fwd(yq2, yk2, v2, *text, return_lse=True)

    dqkv, dkv = torch.empty_like(qkv), torch.empty_like(kv)
    dq, dk, dv = (dqkv[:, i * hd:(i + 1) * hd].view(n, H, D) for i in range(3))
    h3.varlen_cross_attn_bwd(x["do1"], yq, yk, v, o1, lse1, x["cu"], x["cu"], max(SEG), max(SEG), dq=dq, dk=dk, dv=dv)
    _, _, dwq, dwk = h3.qk_norm_rope_bwd(dq, dk, q, k, x["w_q"], x["w_k"], dq=dq, dk=dk, **rot)
    dk2, dv2 = dkv[:, :kd].view(m, HK, D), dkv[:, kd:].view(m, HK, D)
    dq2, _, _ = h3.varlen_cross_attn_bwd(x["do2"], yq2, yk2, v2, o2, lse2, *text, dk=dk2, dv=dv2)
    dq2, _, dwq2, _ = h3.qk_norm_rope_bwd(dq2, None, q2, None, x["w_q2"], None, dq=dq2)
    _, _, dwk2, _ = h3.qk_norm_rope_bwd(dk2, None, k2, None, x["w_k2"], None, dq=dk2)
    return dict(o1=o1, o2=o2, dqkv=dqkv, dq2=dq2, dkv=dkv, dw_q=dwq, dw_k=dwk, dw_q2=dwq2, dw_k2=dwk2)


def _reference(x):
    n, m, hd, kd = x["qkv"].shape[0], x["kv"].shape[0], H * D, HK * D
    f = lambda t: t.double().numpy()
    q, k, v = (f(x["qkv"][:, i * hd:(i + 1) * hd]).reshape(n, H, D) for i in range(3))
    rot = dict(pos=x["pos"].numpy(), tag=x["tag"].numpy(), cu_requests=x["cu"].numpy(), start_frames=x["frames"].numpy())
    cu, cut, used = x["cu"].numpy(), x["cu_text"].numpy(), USED
    yq, yk = oracle.norm_rope(q, x["w_q"], **rot), oracle.norm_rope(k, x["w_k"], **rot)
    o1, _ = oracle.cross_attention(yq, yk, v, cu, cu)
    dyq, dyk, dv = oracle.cross_attention_grad(x["do1"], yq, yk, v, cu, cu)
    dq, dwq = oracle.norm_rope_grad(dyq, q, x["w_q"], **rot)
    dk, dwk = oracle.norm_rope_grad(dyk, k, x["w_k"], **rot)
    q2 = f(x["q2"]).reshape(n, H, D)
    k2, v2 = f(x["kv"][:, :kd]).reshape(m, HK, D), f(x["kv"][:, kd:]).reshape(m, HK, D)
    yq2, yk2 = oracle.norm_rope(q2, x["w_q2"]), oracle.norm_rope(k2, x["w_k2"])
    o2, _ = oracle.cross_attention(yq2, yk2, v2, cu, cut, used)
    dyq2, dyk2, dv2 = oracle.cross_attention_grad(x["do2"], yq2, yk2, v2, cu, cut, used)
    dq2, dwq2 = oracle.norm_rope_grad(dyq2, q2, x["w_q2"])
    dk2, dwk2 = oracle.norm_rope_grad(dyk2, k2, x["w_k2"])
    return dict(o1=o1, o2=o2, dqkv=np.concatenate([t.reshape(n, hd) for t in (dq, dk, dv)], 1), dq2=dq2,
                dkv=np.concatenate([t.reshape(m, kd) for t in (dk2, dv2)], 1), dw_q=dwq, dw_k=dwk, dw_q2=dwq2,
                dw_k2=dwk2)


def test_block_against_fp64(h3, dev):
    x = _block()
    got = _run(h3, {n: t.to(dev) for n, t in x.items()})
    assert h3.get_device_error(dev) == 0
    for name, ref in _reference(x).items():
        g = got[name].double().cpu().numpy().reshape(ref.shape)
        err = np.linalg.norm(g - ref) / np.linalg.norm(ref)
        assert err <= (10 if name.startswith("o") else 20) * HALF, f"{name}: {err:.3e}"


def test_block_captured_and_on_two_streams(h3, dev):
    first, second = ({n: t.to(dev) for n, t in _block(seed).items()} for seed in (1, 2))
    want = [_run(h3, x) for x in (first, second)]
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(a[n], b[n]) for n in a)
    # both at once, each on a stream of its own
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(3):
        for i, x in enumerate((first, second)):
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                got[i] = _run(h3, x)
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(h3, first)
    for x, w in ((first, want[0]), (second, want[1])):
        for n in first:
            first[n].copy_(x[n])  # the second set's values in the captured buffers
        for t in got.values():
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, w)
    assert h3.get_device_error(dev) == 0
