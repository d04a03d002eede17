"""Gradient of packed cross attention on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (derived before the first run).  o is given as the bf16 rounding of
the exact output and lse as its fp32 rounding; with h = 2^-8 (half a bf16 step):
  * dv = P^T do: P is rounded to bf16 and carries the fp32 error of the score and the exponential
    (1e-4 of itself at the scores used here): (h + 1e-4) sum P |do|, and h |dv| for the result.
  * dS = P (dP - delta): P's 1e-4; dP's fp32 sum over D, 1e-5 sum |do| |v|; delta is taken from the
    rounded o, h sum |do| |o|; and dS itself is rounded to bf16:
        e = (h + 1e-4) |dS| + P (1e-5 sum |do| |v| + h sum |do| |o|)
    so dq is within scale sum_j e |k_j| + h |dq|, dk within scale sum_i e |q_i| + h |dk|.
Each result's own rounding applies to the value with its error, a factor 1 + h on the rest.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_cross_attn import CASES, Case

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


def _given(c, dev):
    """The forward's results as the gradient is given them: exact, rounded once."""
    o, lse, _ = c.reference()
    out = torch.full(c.q.shape, float("nan"), dtype=torch.bfloat16)
    out[:c.nq] = torch.from_numpy(o).to(torch.bfloat16)
    full = torch.full((c.q.shape[1], c.cq), float("nan"))
    full[:, :c.nq] = torch.from_numpy(lse).float()
    return out.to(dev), full.to(dev)


def _bounds(c):
    """Error bounds of (dq, dk, dv) before their own rounding."""
    q, k, v, do = (t.double().numpy() for t in (c.q, c.k, c.v, c.do))
    hq, d = q.shape[1:]
    group, scale = hq // k.shape[1], d ** -0.5
    bq, bk, bv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for g in range(len(c.lq)):
        rows = slice(int(c.cu_q[g]), int(c.cu_q[g + 1]))
        n = c.lk[g] if c.used is None else c.used[g]
        keys = slice(int(c.cu_k[g]), int(c.cu_k[g]) + n)
        if n == 0:
            continue
        for h in range(hq):
            x = h // group
            p, _ = oracle.cross._probabilities(q[rows, h], k[keys, x], scale)
            dp = do[rows, h] @ v[keys, x].T
            o = p @ v[keys, x]
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            mass = 1e-5 * (np.abs(do[rows, h]) @ np.abs(v[keys, x]).T)
            mass += HALF * (np.abs(do[rows, h]) * np.abs(o)).sum(1, keepdims=True)
            e = (HALF + 1e-4) * np.abs(ds) + p * mass
            bq[rows, h] = scale * (e @ np.abs(k[keys, x]))
            bk[keys, x] += scale * (e.T @ np.abs(q[rows, h]))
            bv[keys, x] += (HALF + 1e-4) * (p.T @ np.abs(do[rows, h]))
    return bq, bk, bv


def _check(c, got):
    ref = oracle.cross_attention_grad(c.do, c.q, c.k, c.v, c.cu_q, c.cu_k, c.used)
    for name, x, r, b, n in zip(("dq", "dk", "dv"), got, ref, _bounds(c), (c.nq, c.nk, c.nk)):
        x, r = x.double().cpu().numpy()[:n], r[:n]
        err = np.abs(x - r) - ((1 + HALF) * b[:n] + HALF * np.abs(r))
        assert np.all(err <= 0), f"{name}: {np.nanmax(err):.3e} over, {np.isnan(x).sum()} NaN"


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_backward(h3, dev, name):
    c = Case(*CASES[name], seed=2)
    args, where = c.on(dev)
    out, lse = _given(c, dev)
    do = c.do.to(dev)
    dq, dk, dv = (torch.full(t.shape, 7.0, dtype=torch.bfloat16, device=dev) for t in (c.q, c.k, c.v))
    h3.varlen_cross_attn_bwd(do, **args, out=out, lse=lse, **where, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    _check(c, (dq, dk, dv))
    assert (dq[c.nq:] == 7.0).all() and (dk[c.nk:] == 7.0).all() and (dv[c.nk:] == 7.0).all()
    again = h3.varlen_cross_attn_bwd(do, **args, out=out, lse=lse, **where)
    for a, b, n in zip(again, (dq, dk, dv), (c.nq, c.nk, c.nk)):
        assert torch.equal(a[:n], b[:n])  # no dependence on timing


LARGE = {  # more than a wave of items, cut and uncut key tiles
    "text_states": ([1500, 1300], [300, 257], 6, 6, 128, None),
    "padded_shared": ([700, 900], [320, 320], 12, 3, 64, [320, 131]),
    "both_long": ([1100], [1030], 8, 8, 128, None),
    "many_key_tiles": ([130], [5000], 8, 8, 64, None),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", LARGE)
def test_backward_large(h3, dev, name):
    c = Case(*LARGE[name], seed=4)
    args, where = c.on(dev)
    out, lse = _given(c, dev)
    got = h3.varlen_cross_attn_bwd(c.do.to(dev), **args, out=out, lse=lse, **where)
    assert h3.get_device_error(dev) == 0
    _check(c, got)


@pytest.mark.gpu
def test_into_a_fused_gradient_and_unaligned_tensors(h3, dev):
    c = Case([70, 33], [90, 140], 4, 2, 64, seed=5)
    args, where = c.on(dev)
    out, lse = _given(c, dev)
    do = c.do.to(dev)
    want = h3.varlen_cross_attn_bwd(do, **args, out=out, lse=lse, **where)
    dkv = torch.full((c.ck, 2 * 2 * 64 + 8), 7.0, dtype=torch.bfloat16, device=dev)
    dk, dv = dkv[:, :128].view(c.ck, 2, 64), dkv[:, 128:256].view(c.ck, 2, 64)
    # 16-byte aligned, not 32
    dq = torch.empty(c.cq * 4 * 64 + 8, dtype=torch.bfloat16, device=dev)[8:].view(c.cq, 4, 64)
    h3.varlen_cross_attn_bwd(do, **args, out=out, lse=lse, **where, dq=dq, dk=dk, dv=dv)
    for a, b, n in zip((dq, dk, dv), want, (c.nq, c.nk, c.nk)):
        assert torch.equal(a[:n], b[:n])
    assert (dkv[:, 256:] == 7.0).all() and (dkv[c.nk:] == 7.0).all()
    o = torch.empty(c.cq * 4 * 64 + 8, dtype=torch.bfloat16, device=dev)[8:].view(c.cq, 4, 64)
    full = h3.varlen_cross_attn_fwd(**args, **where)
    h3.varlen_cross_attn_fwd(**args, **where, out=o)
    assert torch.equal(o[:c.nq], full[:c.nq])


@pytest.mark.gpu
def test_gradient_of_the_packed_self_attention(h3, dev):
    rng = np.random.default_rng(4)
    c = Case([300, 10, 390], [300, 10, 390], 3, 3, 128, seed=7, tails=(0, 0))
    c.cu_k = c.cu_q
    args, _ = c.on(dev)
    cu = torch.from_numpy(c.cu_q).to(dev)
    q, k, v = args["q"], args["k"].contiguous(), args["v"].contiguous()
    out, lse = h3.varlen_attn_fwd(q, k, v, cu, 390, return_lse=True)
    got = h3.varlen_cross_attn_bwd(c.do.to(dev), q, k, v, out, lse, cu, cu, 390, 390)
    # the kernel's own o is within twice its rounding of the exact one here: a few times the bound
    ref = oracle.cross_attention_grad(c.do, c.q, c.k, c.v, c.cu_q, c.cu_q)
    for x, r in zip(got, ref):
        err = np.linalg.norm(x.double().cpu().numpy() - r) / np.linalg.norm(r)
        assert err <= 2 * HALF  # every rounding's relative size, twice, in the 2-norm


@pytest.mark.gpu
def test_empty_sides(h3, dev):
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    x, none = torch.ones(5, 2, 64, dtype=torch.bfloat16, device=dev), torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=dev)
    lse = torch.full((2, 5), float("-inf"), device=dev)
    dq, dk, dv = h3.varlen_cross_attn_bwd(x, x, none, none, x, lse, i32(0, 2, 5), i32(0, 0, 0), 3, 0)
    assert (dq == 0).all() and dk.shape == none.shape
    dq, dk, dv = h3.varlen_cross_attn_bwd(none, none, x, x, none, lse[:, :0], i32(0, 0), i32(0, 5), 0, 5)
    assert dq.shape == none.shape and (dk == 0).all() and (dv == 0).all()
    h3.varlen_cross_attn_bwd(none, none, none, none, none, lse[:, :0], i32(0, 0), i32(0, 0), 0, 0)
    assert h3.get_device_error(dev) == 0


@pytest.mark.gpu
def test_bad_segments_are_skipped_and_reported(h3, dev):
    c = Case([20, 30, 10], [40, 50, 60], 2, 2, 64, seed=5)
    args, where = c.on(dev)
    out, lse = _given(c, dev)
    do = c.do.to(dev)
    full = h3.varlen_cross_attn_bwd(do, **args, out=out, lse=lse, **where)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    for other, q_skip, k_skip in ((dict(seqused_k=i32(40, 51, 60)), (20, 50), (40, 90)),
                                  (dict(cu_seqlens_k=i32(0, 40, 90, 1000)), (50, 60), (90, 150)),
                                  (dict(cu_seqlens_q=i32(0, 20, 50, 64)), (50, 60), (90, 150))):
        got = [torch.full(t.shape, 7.0, dtype=torch.bfloat16, device=dev) for t in (c.q, c.k, c.v)]
        h3.varlen_cross_attn_bwd(do, **args, out=out, lse=lse, **dict(where, **other), dq=got[0], dk=got[1], dv=got[2])
        assert h3.get_device_error(dev) == 3
        for x, f, (a, b), n in zip(got, full, (q_skip, k_skip, k_skip), (c.nq, c.nk, c.nk)):
            assert (x[a:b] == 7.0).all() and torch.equal(x[:a], f[:a]) and torch.equal(x[b:n], f[b:n])


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["shared_heads", "padded_batch_past_a_tile"])
def test_side_stream_and_graph(h3, dev, name):
    c = Case(*CASES[name], seed=6)
    args, where = c.on(dev)
    out, lse = _given(c, dev)
    do = c.do.to(dev)
    call = lambda: h3.varlen_cross_attn_bwd(do, **args, out=out, lse=lse, **where)
    want = [t.clone() for t in call()]
    same = lambda got: all(torch.equal(a[:n], b[:n]) for a, b, n in zip(got, want, (c.nq, c.nk, c.nk)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert same(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got)


@pytest.mark.gpu
def test_many_calls_back_to_back(h3, dev):
    """Many items a CTA, calls that overlap at their edges: the same gradients, no wait that ran out."""
    gen = torch.Generator(device=dev).manual_seed(8)
    cu_q, cu_k = [0, 3000, 6500], [0, 300, 812]
    x = lambda n: torch.randn(n, 24, 128, device=dev, generator=gen).to(torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    sets = []
    for _ in range(3):
        q, do, k, v = x(6500), x(6500), x(812), x(812)
        where = (i32(cu_q), i32(cu_k), 3500, 512)
        out, lse = h3.varlen_cross_attn_fwd(q, k, v, *where, return_lse=True)
        sets.append((do, q, k, v, out, lse, *where))
    torch.cuda.synchronize()
    want = []
    for s in sets:
        want.append(h3.varlen_cross_attn_bwd(*s))
        torch.cuda.synchronize()
    for _ in range(10):
        got = [h3.varlen_cross_attn_bwd(*s) for s in sets]
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert h3.get_device_error(dev) == 0


# ---- refusals (no GPU) ---------------------------------------------------------------------------


@pytest.mark.parametrize("kw, status", [
    (dict(num_segments=-1), 2), (dict(max_seqlen_q=5), 2), (dict(num_q_heads=3), 2), (dict(head_dim=80), 4),
    (dict(softmax_scale=float("nan")), 2), (dict(k_stride=132), 8), (dict(dq_stride=64), 2), (dict(dk_stride=132), 8),
    (dict(dv_stride=-128), 2), (dict(), 5),
])
def test_c_abi_refuses(h3, kw, status):
    import ctypes as C

    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    base = dict(num_segments=1, max_seqlen_q=4, max_seqlen_k=4, capacity_q=4, capacity_k=4, num_q_heads=2,
                num_kv_heads=2, head_dim=64)
    d = h3._CrossAttnDesc(**{**base, **kw})
    assert h3.load_library().h3_varlen_cross_attn_bwd(C.byref(d), p, p, p, p, p, p, p, p, None, p, p, p, None, 0,
                                                      None) == status


def test_c_abi_refuses_pointers(h3):
    import ctypes as C

    lib = h3.load_library()
    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    odd, two = C.c_void_p(p.value + 8), C.c_void_p(p.value + 2)
    d = h3._CrossAttnDesc(num_segments=1, max_seqlen_q=4, max_seqlen_k=4, capacity_q=4, capacity_k=4, num_q_heads=2,
                          num_kv_heads=2, head_dim=64)
    n = lib.h3_varlen_cross_attn_bwd_workspace_size(C.byref(d))
    assert n > 0
    good = [p] * 13 + [n]
    good[8] = None  # seqused_k

    def call(at, x):
        args = list(good)
        args[at] = x
        return lib.h3_varlen_cross_attn_bwd(C.byref(d), *args, None)

    for at in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11):
        assert call(at, None) == 1, at
    for at in (0, 1, 2, 3, 4, 9, 10, 11, 12):
        assert call(at, odd) == 8, at
    for at in (5, 6, 7, 8):
        assert call(at, two) == 8, at
    assert call(12, None) == 5 and call(13, n - 1) == 5


def test_binding_refuses(h3):
    q, k = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    cu, cuk = torch.tensor([0, 4], dtype=torch.int32), torch.tensor([0, 6], dtype=torch.int32)
    lse = torch.zeros(4, 4)
    call = lambda do=q, out=q, lse=lse, **kw: h3.varlen_cross_attn_bwd(do, q, k, k, out, lse, cu, cuk, 4, 6, **kw)
    with pytest.raises(TypeError):
        call(do=q.float())
    with pytest.raises(TypeError):
        call(lse=lse.double())
    for bad in (dict(do=q[:3]), dict(out=q.transpose(0, 1)), dict(lse=lse[:, :3]), dict(dq=q[:3]),
                dict(dk=k.transpose(1, 2)), dict(dv=k[:5])):
        with pytest.raises(ValueError):
            call(**bad)
