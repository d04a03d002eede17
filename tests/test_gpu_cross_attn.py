"""Packed cross attention on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (derived before the first run).  S and the sums are fp32; the
weights are rounded to bf16 (half a step, 2^-8 of each) before the product with V, and o is rounded
to bf16 once more:
    |o - o*| <= 2^-8 sum_j P_j |v_j| + 2^-8 |o| + fp32 terms,
fp32 terms: the score's error (D products, 2^-24 each of |q||k|, and the exponential's 2^-22) moves
each weight by under 1e-4 of itself at the scores used here: 2e-4 sum_j P_j |v_j|.
lse: the same error of the scores, absolute: 1e-4 * max(|lse|, 1) as elsewhere in this suite.
"""
import numpy as np
import pytest
import torch

import oracle

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


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def _offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


class Case:
    """lq, lk: rows and key rows of each segment; used: keys used, or None; tails: rows behind the
    last segment on either side."""

    def __init__(self, lq, lk, hq, hk, d, used=None, seed=0, tails=(3, 5), scale=1.0):
        rng = np.random.default_rng(seed)
        self.lq, self.lk, self.used = lq, lk, used
        self.cu_q, self.cu_k = _offsets(lq), _offsets(lk)
        self.nq, self.nk = int(self.cu_q[-1]), int(self.cu_k[-1])
        self.cq, self.ck = self.nq + tails[0], self.nk + tails[1]
        self.q = _bf16(rng, self.cq, hq, d, scale=scale)
        kv = _bf16(rng, self.ck, 2 * hk * d, scale=scale)
        self.k, self.v = kv[:, :hk * d].view(self.ck, hk, d), kv[:, hk * d:].view(self.ck, hk, d)
        self.do = _bf16(rng, self.cq, hq, d)
        # what no segment uses must not matter: NaN and Inf there
        for t in (self.k, self.v):
            t[self.nk:] = float("nan")
            if used is not None:
                for g, n in enumerate(used):
                    t[int(self.cu_k[g]) + n:int(self.cu_k[g + 1])] = float("inf") if g % 2 else float("nan")
        self.q[self.nq:] = float("nan")
        self.do[self.nq:] = float("nan")
        keys = used if used is not None else lk
        self.max_q, self.max_k = max(lq), max(keys)

    def on(self, dev):
        kv = torch.empty(self.ck, 2, *self.k.shape[1:], dtype=torch.bfloat16, device=dev)
        kv[:, 0], kv[:, 1] = self.k.to(dev), self.v.to(dev)
        return dict(q=self.q.to(dev), k=kv[:, 0], v=kv[:, 1]), dict(
            cu_seqlens_q=torch.from_numpy(self.cu_q).to(dev), cu_seqlens_k=torch.from_numpy(self.cu_k).to(dev),
            max_seqlen_q=self.max_q, max_seqlen_k=self.max_k,
            seqused_k=None if self.used is None else torch.tensor(self.used, dtype=torch.int32, device=dev))

    def reference(self, scale=None):
        args = (self.cu_q, self.cu_k, self.used, scale)
        o, lse = oracle.cross_attention(self.q, self.k, self.v, *args)
        size, _ = oracle.cross_attention(self.q, self.k, self.v.abs(), *args)
        return o[:self.nq], lse[:, :self.nq], size[:self.nq]


def _check(c, out, lse, scale=None):
    o, l, size = c.reference(scale)
    got = out.double().cpu().numpy()[:c.nq]
    tol = (HALF + 2e-4) * (1 + HALF) * size + HALF * np.abs(o)
    err = np.abs(got - o)
    assert np.all(err <= tol), f"o: {np.nanmax(err - tol):.3e} over, {np.isnan(got).sum()} NaN"
    gl = lse.double().cpu().numpy()[:, :c.nq]
    assert np.array_equal(np.isneginf(gl), np.isneginf(l))
    f = np.isfinite(l)
    assert np.all(np.abs(gl[f] - l[f]) <= 1e-4 * np.maximum(np.abs(l[f]), 1.0))


# rows per segment, key rows per segment, q heads, k heads, head_dim, keys used
CASES = {
    "one_row_one_key": ([1], [1], 1, 1, 64, None),
    "worked_example_rows": ([10, 20, 15], [7, 33, 2], 2, 2, 64, None),
    "empty_sides": ([5, 0, 3, 7, 0], [4, 6, 0, 9, 0], 2, 1, 128, None),
    "no_key_anywhere": ([5, 3], [0, 0], 2, 2, 64, None),
    "padded_batch": ([130, 1, 257], [40, 40, 40], 3, 3, 128, [40, 17, 0]),
    "padded_batch_past_a_tile": ([64, 100, 31, 9], [300, 300, 300, 300], 4, 2, 64, [129, 300, 1, 256]),
    "tile_edges": ([127, 128, 129, 255, 256, 257], [128, 129, 127, 256, 1, 255], 2, 2, 128, None),
    "shared_heads": ([70, 300], [200, 513], 24, 8, 64, None),
    "one_key_head": ([33, 65], [77, 140], 16, 1, 128, None),
    "few_rows_many_keys": ([20, 3, 41], [3000, 1025, 2047], 4, 2, 128, None),
    "split_keys_partly_used": ([18, 200], [4100, 2500], 3, 3, 64, [3999, 1]),
    "many_segments": ([(7 * i) % 23 for i in range(300)], [(5 * i) % 31 for i in range(300)], 2, 2, 64, None),
    "tokens": ([1] * 9, [600, 1, 0, 77, 1300, 16, 15, 17, 2049], 8, 1, 128, None),
    "tokens_one_head_each": ([1, 1, 0, 1], [200, 33, 9, 1024], 5, 5, 64, [190, 33, 9, 1000]),
    "a_few_tokens": ([2, 1, 3, 0, 2], [64, 700, 129, 12, 0], 4, 1, 64, None),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_forward(h3, dev, name):
    c = Case(*CASES[name])
    args, where = c.on(dev)
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((c.q.shape[1], c.cq), 7.0, device=dev)
    h3.varlen_cross_attn_fwd(**args, **where, out=out, lse=lse)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    _check(c, out, lse)
    assert (out[c.nq:] == 7.0).all() and (lse[:, c.nq:] == 7.0).all()  # rows of no segment
    again, lse2 = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)
    assert torch.equal(again[:c.nq], out[:c.nq]) and torch.equal(lse2[:, :c.nq], lse[:, :c.nq])
    assert torch.equal(h3.varlen_cross_attn_fwd(**args, **where)[:c.nq], out[:c.nq])  # without an LSE
    # looser bounds may take another split, not another result
    where.update(max_seqlen_q=c.cq, max_seqlen_k=c.ck)
    wide, wide_lse = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)
    _check(c, wide, wide_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.05, 1.0])
def test_scale(h3, dev, scale):
    c = Case([37, 1], [150, 90], 2, 2, 64, seed=3, scale=0.6)
    args, where = c.on(dev)
    out, lse = h3.varlen_cross_attn_fwd(**args, **where, softmax_scale=scale, return_lse=True)
    _check(c, out, lse, scale)


@pytest.mark.gpu
def test_equal_offsets_are_the_packed_self_attention(h3, dev):
    rng = np.random.default_rng(4)
    q, k, v = (_bf16(rng, 700, 3, 128).to(dev) for _ in range(3))
    cu = torch.tensor([0, 300, 310, 700], dtype=torch.int32, device=dev)
    a, la = h3.varlen_attn_fwd(q, k, v, cu, 390, return_lse=True)
    b, lb = h3.varlen_cross_attn_fwd(q, k, v, cu, cu, 390, 390, return_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.gpu
def test_bad_segments_are_skipped_and_reported(h3, dev):
    c = Case([20, 30, 10], [40, 50, 60], 2, 2, 64, seed=5)
    args, where = c.on(dev)
    full, _ = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)

    def run(**other):
        out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device=dev)
        h3.varlen_cross_attn_fwd(**args, **dict(where, **other), out=out)
        return out, h3.get_device_error(dev)

    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    for other, skipped in ((dict(seqused_k=i32(40, 51, 60)), [(20, 50)]), (dict(seqused_k=i32(-1, 50, 60)), [(0, 20)]),
                           (dict(cu_seqlens_k=i32(0, 40, 90, 1000)), [(50, 60)]),
                           (dict(cu_seqlens_q=i32(0, 20, 50, 64)), [(50, 64)])):
        out, err = run(**other)
        assert err == 3
        for a, b in skipped:
            assert (out[a:b] == 7.0).all()
        ok = torch.ones(c.nq, dtype=torch.bool)
        for a, b in skipped:
            ok[a:b] = False
        assert torch.equal(out[:c.nq][ok.to(dev)], full[:c.nq][ok.to(dev)])
    out, err = run(max_seqlen_k=55)  # a longer segment is computed all the same, and reported
    assert err == 3 and torch.equal(out[:c.nq], full[:c.nq])
    out, err = run()
    assert err == 0 and torch.equal(out[:c.nq], full[:c.nq])


@pytest.mark.gpu
def test_no_keys_and_no_rows_at_all(h3, dev):
    q = torch.ones(5, 2, 64, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=dev)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    out, lse = h3.varlen_cross_attn_fwd(q, k, k, i32(0, 2, 5), i32(0, 0, 0), 3, 0, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = h3.varlen_cross_attn_fwd(k, q, q, i32(0, 0), i32(0, 5), 0, 5, return_lse=True)
    assert out.shape == k.shape and lse.shape == (2, 0)
    out = torch.full_like(q, 7.0)
    h3.varlen_cross_attn_fwd(q, q, q, i32(0), i32(0), 0, 0, out=out)  # no segment
    assert (out == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["shared_heads", "few_rows_many_keys", "tokens"])
def test_side_stream_and_graph(h3, dev, name):
    c = Case(*CASES[name], seed=6)
    args, where = c.on(dev)
    want = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)
    want = [want[0][:c.nq].clone(), want[1][:, :c.nq].clone()]
    same = lambda got: torch.equal(got[0][:c.nq], want[0]) and torch.equal(got[1][:, :c.nq], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)
    side.synchronize()
    assert same(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)
    for _ in range(2):
        got[0].fill_(7.0), got[1].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got)


# ---- refusals (no GPU) ---------------------------------------------------------------------------


def _desc(h3, **kw):
    base = dict(num_segments=1, max_seqlen_q=4, max_seqlen_k=4, capacity_q=4, capacity_k=4, num_q_heads=2,
                num_kv_heads=2, head_dim=64, softmax_scale=0.0)
    return h3._CrossAttnDesc(**{**base, **kw})


@pytest.mark.parametrize("kw, status", [
    (dict(num_segments=-1), 2), (dict(num_segments=65536), 2), (dict(max_seqlen_q=5), 2), (dict(max_seqlen_k=5), 2),
    (dict(max_seqlen_k=-1), 2), (dict(capacity_q=-1), 2), (dict(num_q_heads=0), 2), (dict(num_kv_heads=0), 2),
    (dict(num_q_heads=3), 2), (dict(num_q_heads=65536, num_kv_heads=65536), 2), (dict(head_dim=80), 4),
    (dict(softmax_scale=float("inf")), 2), (dict(softmax_scale=float("nan")), 2), (dict(q_stride=64), 2),
    (dict(k_stride=132), 8), (dict(v_stride=-128), 2), (dict(), 5),
    (dict(capacity_q=2000000000, num_q_heads=65534), 2), (dict(capacity_k=2000000000, num_q_heads=65534), 2),
])
def test_c_abi_refuses(h3, kw, status):
    import ctypes as C

    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    d = _desc(h3, **kw)
    assert h3.load_library().h3_varlen_cross_attn_fwd(C.byref(d), p, p, p, p, None, p, p, None, None, 0, None) == status


def test_c_abi_refuses_pointers(h3):
    import ctypes as C

    lib = h3.load_library()
    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    odd, two = C.c_void_p(p.value + 8), C.c_void_p(p.value + 2)
    d = _desc(h3)
    n = lib.h3_varlen_cross_attn_workspace_size(C.byref(d))
    assert n > 0
    good = [p, p, p, p, p, p, p, p, p, n]

    def call(at, x):
        args = list(good)
        args[at] = x
        return lib.h3_varlen_cross_attn_fwd(C.byref(d), *args, None)

    for at in (0, 1, 2, 3, 5, 6):
        assert call(at, None) == 1
    for at in (0, 1, 2, 3, 8):
        assert call(at, odd) == 8
    for at in (4, 5, 6, 7):
        assert call(at, two) == 8
    assert call(8, None) == 5 and call(9, n - 1) == 5
    assert lib.h3_varlen_cross_attn_fwd(None, *good, None) == 1
    assert lib.h3_varlen_cross_attn_workspace_size(None) == 0
    assert lib.h3_varlen_cross_attn_workspace_size(C.byref(_desc(h3, num_q_heads=3))) == 0


def test_binding_refuses(h3):
    q, k = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    cu, cuk = torch.tensor([0, 4], dtype=torch.int32), torch.tensor([0, 6], dtype=torch.int32)
    call = lambda q=q, k=k, v=k, cu=cu, cuk=cuk, **kw: h3.varlen_cross_attn_fwd(q, k, v, cu, cuk, 4, 6, **kw)
    for bad in (dict(q=q.float()), dict(k=k.float()), dict(cu=cu.long()), dict(seqused_k=cu[:1].long())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(q=q[0]), dict(v=k[:5]), dict(k=k.transpose(1, 2)), dict(k=k[:, :, :32], v=k[:, :, :32]),
                dict(cuk=cuk[:1]), dict(cu=cu[:0], cuk=cuk[:0]), dict(seqused_k=cuk), dict(out=q[:3]),
                dict(lse=torch.zeros(4, 5)), dict(out=q.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**bad)


# Work dealt in shares (a last wave of items is cut where a CTA's share ends): rows, keys, heads.
SHARES = {
    "heads_apart": ([200, 300], [3000, 2500], 5, 5, 64, None),
    "shared_heads_apart": ([100, 40], [2500, 5000], 12, 3, 64, None),
    "one_item": ([30], [20000], 1, 1, 64, None),
    "long_and_short_keys": ([30, 270, 20, 5, 140], [9000, 200, 1100, 1, 3001], 4, 4, 64, [8990, 150, 1024, 1, 3001]),
    "behind_a_whole_wave": ([20, 30, 17, 140, 40, 21, 33], [1100, 2300, 1500, 1300, 3000, 1025, 0], 24, 24, 64, None),
    "more_heads_than_ctas": ([20], [1300], 160, 160, 64, None),
    "two_items_a_cta_or_none": ([257] * 3, [1600] * 3, 20, 10, 128, None),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", SHARES)
def test_shares(h3, dev, name):
    c = Case(*SHARES[name], seed=6)
    args, where = c.on(dev)
    where["max_seqlen_k"] = max(where["max_seqlen_k"], 1024)
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((c.q.shape[1], c.cq), 7.0, device=dev)
    n = h3.varlen_cross_attn_workspace_size(len(c.lq), c.max_q, where["max_seqlen_k"], c.cq, c.ck, c.q.shape[1],
                                            c.k.shape[1], c.q.shape[2])
    ws = torch.full((n + 16,), 255, dtype=torch.uint8, device=dev)  # 16 bytes past a 32-byte boundary
    h3.varlen_cross_attn_fwd(**args, **where, out=out, lse=lse, workspace=ws[16:])
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    _check(c, out, lse)
    assert (out[c.nq:] == 7.0).all() and (lse[:, c.nq:] == 7.0).all()
    again, lse2 = h3.varlen_cross_attn_fwd(**args, **where, return_lse=True)
    assert torch.equal(again[:c.nq], out[:c.nq]) and torch.equal(lse2[:, :c.nq], lse[:, :c.nq])
