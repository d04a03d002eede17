"""Attention over a paged cache on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (the terms of 2^-126 and 2^-25 were added, with theirs, after runs that met
them).  The cache's values are exact in bf16, so
both sides start from the same keys and values.  S and the sums are fp32; the weights are rounded to bf16
(half a step, 2^-8 of each) before the product with V, and o is rounded to bf16 once more:
    |o - o*| <= 2^-8 sum_j P_j |v_j| + 2^-8 |o| + fp32 terms,
fp32 terms: the score's error (D products, 2^-24 each of |q||k|, and the exponential's 2^-22) moves each weight
by under 1e-4 of itself at the scores used here: 2e-4 sum_j P_j |v_j|.
A weight under 2^-126 of its row's largest is 0 (the exponential flushes it), which is an absolute error of
2^-126 |v_j| for each key: it shows where every larger weight meets a value of exactly 0, as in e4m3.
The token form of an e4m3 cache rounds the weights times V's scales, 2^(e_j) P_j, to f16 over a reference that is at
most their largest: by 2^-11 of each or, below 2^-14 of the reference, by 2^-25 of the reference.  The first is inside
2^-8 of each; the second adds 2^-25 max_j(2^(e_j)) sum_j |q_j|, with v_j = 2^(e_j) q_j and P_j <= 1.
lse: the same error of the scores, absolute: 1e-4 * max(|lse|, 1) as elsewhere in this suite.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle.norm import _f64

HALF = 2.0 ** -8
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


def _desc(h3, **kw):
    base = dict(num_segments=1, max_seqlen_q=2, max_seqlen_k=8, capacity_q=2, num_q_heads=4, num_kv_heads=2, head_dim=64,
                cache_type=2, page_size=16, num_pages=1, max_pages=1)
    return h3._PagedAttnDesc(**{**base, **kw})


@pytest.mark.parametrize("kw, status", [
    (dict(num_segments=-1), 2), (dict(num_segments=65536), 2), (dict(max_seqlen_q=-1), 2), (dict(max_seqlen_q=3), 2),
    (dict(max_seqlen_k=-1), 2), (dict(capacity_q=-1), 2), (dict(num_q_heads=0), 2), (dict(num_kv_heads=3), 2),
    (dict(num_q_heads=258, num_kv_heads=2), 2), (dict(num_kv_heads=-2), 2), (dict(head_dim=96), 4), (dict(cache_type=0), 2),
    (dict(page_size=8), 2), (dict(page_size=100), 2), (dict(num_pages=-1), 2), (dict(max_pages=-1), 2),
    (dict(causal_block=-1), 2), (dict(softmax_scale=float("nan")), 2), (dict(softmax_scale=float("inf")), 2),
    (dict(q_stride=128), 2), (dict(q_stride=260), 8), (dict(cache_type=1), 1), (dict(num_pages=1 << 30, num_kv_heads=2), 2),
])
def test_c_abi_refuses(h3, kw, status):
    import ctypes as C

    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    assert h3.load_library().h3_paged_attn_fwd(C.byref(_desc(h3, **kw)), *(p,) * 11, 1 << 40, None) == status


def test_c_abi_refuses_pointers(h3):
    import ctypes as C

    lib = h3.load_library()
    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    d = _desc(h3)
    fwd = lambda a, d=d, n=1 << 40: lib.h3_paged_attn_fwd(C.byref(d), *a, n, None)  # noqa: E731
    assert lib.h3_paged_attn_fwd(None, *(p,) * 11, 1 << 40, None) == 1
    # q, k, v, their scales, table, offsets, lengths, o, lse, workspace
    for i in range(11):
        a = [p] * 11
        a[i] = None
        if i != 9:  # no LSE is fine
            assert fwd(a) == (5 if i == 10 else 1), i
        a[i] = C.c_void_p(p.value + (2 if i in (5, 6, 7, 9) else 8))
        assert fwd(a) == 8, i
    for rows in (2, 9):
        d = _desc(h3, max_seqlen_q=rows, capacity_q=rows)
        need = lib.h3_paged_attn_workspace_size(C.byref(d))
        assert need > 0 and fwd([p] * 11, d, need - 1) == 5
    assert lib.h3_paged_attn_workspace_size(C.byref(_desc(h3, page_size=24))) == 0
    assert lib.h3_paged_attn_workspace_size(C.byref(_desc(h3, head_dim=32))) == 0
    assert lib.h3_paged_attn_workspace_size(None) == 0


def test_binding_refuses(h3):
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    cache, table = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32)
    cu, used = torch.tensor([0, 4], dtype=torch.int32), torch.tensor([8], dtype=torch.int32)
    base = dict(q=q, k_cache=cache, v_cache=cache, block_table=table, cu_seqlens_q=cu, seqused_k=used, max_seqlen_q=4,
                max_seqlen_k=8)
    sc = torch.zeros(3, 2, 16, dtype=torch.uint8)
    for error, kw in [
        (TypeError, dict(q=q.float())), (ValueError, dict(q=q[0])), (TypeError, dict(k_cache=cache.float())),
        (ValueError, dict(q=torch.zeros(4, 4, 128, dtype=torch.bfloat16))), (ValueError, dict(k_scale=sc, v_scale=sc)),
        (ValueError, dict(k_cache=cache.to(torch.float8_e4m3fn), v_cache=cache.to(torch.float8_e4m3fn))),
        (ValueError, dict(v_cache=cache[:2])), (TypeError, dict(block_table=table.long())),
        (ValueError, dict(block_table=torch.zeros(2, 2, dtype=torch.int32))), (TypeError, dict(seqused_k=used.long())),
        (ValueError, dict(seqused_k=torch.zeros(2, dtype=torch.int32))), (TypeError, dict(cu_seqlens_q=cu.long())),
        (TypeError, dict(out=q.float())), (ValueError, dict(out=q[:3])), (ValueError, dict(lse=torch.zeros(4, 3))),
        (TypeError, dict(workspace=torch.zeros(4))),
    ]:
        with pytest.raises(error):
            h3.paged_attn_fwd(**{**base, **kw})


# ---- cases ---------------------------------------------------------------------------------------------


class Case:
    """Segments of lq new rows, the last of lk cached tokens.  Whatever no segment uses (other pages, rows past
    the end, table entries past the last page, rows of q behind the last segment) is NaN or out of range."""

    def __init__(self, lq, lk, hq, hk, d, page, e4m3, block, seed=0, tail=3, scale=1.0):
        rng = np.random.default_rng(seed)
        bf = lambda *s: torch.from_numpy((rng.standard_normal(s) * scale).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
        self.lq, self.lk, self.hq, self.block, self.e4m3 = lq, lk, hq, block, e4m3
        self.cu = np.concatenate([[0], np.cumsum(lq)]).astype(np.int32)
        self.n = int(self.cu[-1])
        self.q = bf(self.n + tail, hq, d)
        self.q[self.n:] = float("nan")
        counts = [(n + page - 1) // page for n in lk]
        pages = sum(counts) + 3
        ids = rng.permutation(pages)
        self.table = np.full((len(lk), max(counts) + 1), -5, dtype=np.int32)
        self.rows, self.cache = {"k": [], "v": []}, {}
        self.scales = []  # of V, e4m3: exponents [n, hk] of each segment
        for name in "kv":
            kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
            store = torch.full((pages, hk, page, d), 448.0 if e4m3 else float("nan")).to(kind)
            scales = torch.full((pages, hk, page), 255, dtype=torch.uint8)
            at = 0
            for g, n in enumerate(lk):
                mine = ids[at:at + counts[g]]
                self.table[g, :counts[g]] = mine
                at += counts[g]
                x = bf(n, hk, d)
                if e4m3:
                    x = x.float() * torch.from_numpy(np.exp(rng.standard_normal((n, hk, 1)))).float()  # rows of unlike sizes
                    e = oracle.e4m3_scale(x) if n else np.zeros((0, hk), int)
                    if name == "v":
                        self.scales.append(e)
                    values = oracle.e4m3_round(_f64(x) / np.ldexp(1.0, e)[..., None])
                    self.rows[name].append(values * np.ldexp(1.0, e)[..., None])
                    put, es = torch.from_numpy(values).float().to(kind), torch.from_numpy(e + 127).to(torch.uint8)
                else:
                    self.rows[name].append(_f64(x))
                    put, es = x, None
                view = store.view(torch.uint8) if e4m3 else store
                src = put.view(torch.uint8) if e4m3 else put
                for i in range(counts[g]):
                    part = src[i * page:(i + 1) * page]
                    view[int(mine[i]), :, :part.shape[0]] = part.transpose(0, 1)
                    if e4m3:
                        scales[int(mine[i]), :, :part.shape[0]] = es[i * page:(i + 1) * page].transpose(0, 1)
            self.cache[name + "_cache"] = store
            if e4m3:
                self.cache[name + "_scale"] = scales
        self.max_q, self.max_k = max(lq), max(lk)

    def on(self, dev):
        i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)  # noqa: E731
        return dict(q=self.q.to(dev), block_table=i32(self.table), cu_seqlens_q=i32(self.cu), seqused_k=i32(self.lk),
                    max_seqlen_q=self.max_q, max_seqlen_k=self.max_k, causal_block=self.block,
                    **{k: v.to(dev) for k, v in self.cache.items()})

    def check(self, o, lse, scale=None):
        n = self.n
        ref, rl = oracle.paged_attention(self.q[:n], self.rows["k"], self.rows["v"], self.cu, self.lk, self.block, scale)
        size, _ = oracle.paged_attention(self.q[:n], self.rows["k"], [np.abs(v) for v in self.rows["v"]], self.cu, self.lk,
                                         self.block, scale)
        got = _f64(o[:n])
        assert np.all(np.isfinite(got))
        off = np.abs(got - ref)
        most = max([np.abs(v).sum(0).max() for v in self.rows["v"] if len(v)], default=0.0)
        tol = (HALF + 2e-4) * size + HALF * np.abs(ref) + 2.0 ** -126 * most
        if self.e4m3 and self.max_q * self.hq // self.rows["k"][0].shape[1] <= 16:
            for g, e in enumerate(self.scales):
                if e.size:
                    q = np.abs(self.rows["v"][g]) / np.ldexp(1.0, e)[..., None]
                    more = 2.0 ** -25 * np.ldexp(1.0, e.max(0))[:, None] * q.sum(0)  # [hk, d]
                    tol[self.cu[g]:self.cu[g + 1]] += np.repeat(more, self.hq // e.shape[1], axis=0)
        assert np.all(off <= tol), (off - tol).max()
        if lse is not None:
            gl = _f64(lse[:, :n])
            none = np.isneginf(rl)
            assert np.array_equal(np.isneginf(gl), none)
            gl, rl = gl[~none], rl[~none]
            assert np.all(np.abs(gl - rl) <= 1e-4 * np.maximum(np.abs(rl), 1.0))


def _run(h3, dev, case, **kw):
    a = case.on(dev)
    out = torch.full(a["q"].shape, 5.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((case.hq, a["q"].shape[0]), 5.0, device=dev)
    h3.paged_attn_fwd(**a, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    assert torch.all(out[case.n:] == 5.0) and torch.all(lse[:, case.n:] == 5.0)  # rows of no segment
    return out, lse


_RNG = np.random.default_rng(11)
# new rows, cached tokens, query heads, key heads, page, causal block: few rows (times shared heads)
TOKENS = [
    ([1], [1], 1, 1, 16, 1),
    ([1], [0], 2, 1, 16, 0),
    ([1, 1, 1], [5, 64, 65], 8, 1, 16, 1),
    ([2, 0, 1], [100, 50, 1000], 16, 2, 32, 1),
    ([3], [2], 4, 1, 16, 1),                       # more rows than tokens: the first sees nothing
    ([4, 4], [777, 130], 4, 4, 64, 3),
    ([16], [901], 2, 2, 128, 1),
    ([5, 2], [333, 17], 6, 2, 256, 0),
    ([1] * 40, [int(x) for x in _RNG.integers(1, 600, 40)], 64, 8, 16, 1),
    ([1, 0] * 150, [int(x) for x in _RNG.integers(0, 70, 300)], 2, 1, 16, 1),  # more segments than a scan takes at once
    ([1], [20011], 8, 1, 64, 1),                    # one pair over many CTAs
    ([1, 1], [9000, 3], 10, 2, 128, 1),
]


@pytest_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shape", TOKENS)
def test_few_rows(h3, dev, shape, e4m3, d):
    lq, lk, hq, hk, page, block = shape
    case = Case(lq, lk, hq, hk, d, page, e4m3, block)
    case.check(*_run(h3, dev, case))


@pytest_gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_few_rows_large_scores_and_scale(h3, dev, e4m3):
    """Scores of some hundreds: the running maximum moves often."""
    case = Case([2, 1], [3000, 500], 8, 2, 128, 32, e4m3, 1, scale=2.0)
    case.check(*_run(h3, dev, case, softmax_scale=0.2), scale=0.2)


# more rows than the token form takes: the tile form
CHUNKS = [
    ([17], [17], 1, 1, 16, 1),
    ([20], [0], 2, 1, 16, 1),                        # no cached token at all
    ([40, 3], [25, 130], 2, 2, 16, 1),               # more rows than tokens
    ([9, 0, 33], [700, 40, 129], 8, 2, 32, 0),
    ([7, 26, 1], [640, 26, 127], 40, 8, 64, 1),      # five heads share: 25 tokens a tile
    ([130, 257], [131, 1000], 3, 3, 128, 5),
    ([300], [555], 6, 2, 256, 100),
    ([64, 65, 128, 129], [64, 193, 128, 257], 4, 1, 16, 1),
    ([3, 2], [4000, 5], 128, 1, 64, 1),              # a tile per token
    ([2, 1], [900, 40], 100, 1, 32, 1),              # 100 heads share: 28 rows of the tile stay empty
    ([1000], [1000], 2, 1, 64, 1),                   # a first chunk, causal by token
    ([600, 600], [2600, 1800], 4, 4, 64, 50),        # the last wave is cut
    ([30, 500], [20000, 700], 2, 2, 128, 1),         # one item over many CTAs
    ([20] * 300, [int(x) for x in _RNG.integers(0, 90, 300)], 2, 2, 16, 3),  # more segments than are ordered
    ([700] * 3, [700, 1400, 2100], 24, 8, 64, 1),    # several waves of items of unlike length
]


@pytest_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shape", CHUNKS)
def test_chunks(h3, dev, shape, e4m3, d):
    lq, lk, hq, hk, page, block = shape
    case = Case(lq, lk, hq, hk, d, page, e4m3, block)
    case.check(*_run(h3, dev, case))


# more than 512 rows of a key head over an e4m3 cache: it is unpacked first, where the workspace has room
UNPACKED = [
    ([513], [513], 1, 1, 16, 1),
    ([600, 0, 3], [1400, 900, 77], 2, 2, 32, 0),       # a segment without new rows is not unpacked
    ([300, 700], [20, 1300], 4, 2, 64, 50),            # more rows than tokens
    ([140, 5], [1000, 0], 24, 3, 128, 7),
    ([1030], [2100], 1, 1, 256, 1),
]


@pytest_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", UNPACKED)
def test_unpacked_chunks(h3, dev, shape, d):
    lq, lk, hq, hk, page, block = shape
    case = Case(lq, lk, hq, hk, d, page, True, block, seed=d)
    a = case.on(dev)
    sizes = [h3.paged_attn_workspace_size(len(lq), case.max_q, case.max_k, a["q"].shape[0], hq, hk, d, page, e4m3=e,
                                          max_pages=a["block_table"].shape[1]) for e in (False, True)]
    pages = len(lq) * -(-case.max_k // page)
    assert sizes[1] - sizes[0] >= 4 * pages * page * hk * d
    space = torch.full((sizes[1],), 255, dtype=torch.uint8, device=dev)  # NaN wherever the call does not write
    out, lse = _run(h3, dev, case, workspace=space)
    case.check(out, lse)
    again, lse2 = _run(h3, dev, case, workspace=space[:sizes[0]].fill_(255))
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # captured, then replayed with fewer tokens of each sequence, while another call runs beside it
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        got = h3.paged_attn_fwd(**a)
    a["seqused_k"].sub_(3).clamp_(min=0)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    graph.replay()
    with torch.cuda.stream(other):
        want = h3.paged_attn_fwd(**a)
    torch.cuda.synchronize()
    assert torch.equal(got[:case.n], want[:case.n]) and h3.get_device_error(dev) == 0


@pytest_gpu
def test_unpacked_bad_lengths_and_pages(h3, dev):
    case = Case([520, 520, 520], [700, 650, 90], 2, 2, 64, 16, True, 1)
    good = case.on(dev)
    want = h3.paged_attn_fwd(**good)
    for what, status in (("used", 3), ("negative", 3), ("long", 3), ("page", 12), ("below", 12)):
        a = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in good.items()}
        same = [0, 1, 2]
        if what == "used":
            a["seqused_k"][1], same = 16 * a["block_table"].shape[1] + 1, [0, 2]
        elif what == "negative":
            a["seqused_k"][1], same = -1, [0, 2]
        elif what == "long":  # the first is past what the bound makes room for
            a["max_seqlen_k"], same = 660, [1, 2]
        else:
            a["block_table"][2, 1], same = (a["k_cache"].shape[0] if what == "page" else -3), [0, 1]
        out = torch.full_like(a["q"], 5.0)
        h3.paged_attn_fwd(**a, out=out)
        torch.cuda.synchronize()
        assert h3.get_device_error(dev) == status, what
        for g in range(3):
            part = slice(520 * g, 520 * (g + 1))
            if g in same:
                assert torch.equal(out[part], want[part]), (what, g)
            elif status == 3:
                assert torch.all(out[part] == 5.0), (what, g)


@pytest_gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_large_scores_and_scale(h3, dev, e4m3):
    case = Case([150, 40], [1800, 300], 4, 2, 128, 32, e4m3, 7, scale=2.0)
    case.check(*_run(h3, dev, case, softmax_scale=0.2), scale=0.2)


@pytest_gpu
@pytest.mark.parametrize("seed", range(8))
def test_random_layouts(h3, dev, seed):
    rng = np.random.default_rng(100 + seed)
    for _ in range(6):
        hk = int(rng.choice([1, 2, 3, 8]))
        hq = hk * int(rng.choice([1, 2, 3, 5, 8]))
        s = int(rng.integers(1, 7))
        few = rng.random() < 0.4
        lq = [int(x) for x in rng.integers(0, (16 * hk // hq) + 1 if few else 200, s)]
        lk = [max(0, q + int(rng.integers(-5, 700))) for q in lq]
        if max(lq) == 0:
            continue
        case = Case(lq, lk, hq, hk, int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128, 256])),
                    bool(rng.random() < 0.5), int(rng.choice([0, 1, 2, 17, 64, 1000, 2 ** 31 - 1])), seed=seed)
        case.check(*_run(h3, dev, case))


@pytest_gpu
def test_loose_bounds_and_no_lse(h3, dev):
    """max_seqlen bounds above the lengths take another form and give the same within its tolerances."""
    case = Case([2, 1], [300, 77], 8, 2, 128, 16, True, 1)
    a = case.on(dev)
    for mq, mk in ((2, 300), (3, 5000), (1000, 100000)):
        a["q"] = torch.cat([case.q, torch.zeros(1000, 8, 128, dtype=torch.bfloat16)]).to(dev)
        out = h3.paged_attn_fwd(**{**a, "max_seqlen_q": mq, "max_seqlen_k": mk})
        torch.cuda.synchronize()
        assert h3.get_device_error(dev) == 0
        case.check(out, None)


@pytest_gpu
@pytest.mark.parametrize("rows", [2, 40])
def test_bad_lengths_and_pages(h3, dev, rows):
    """A bad segment is skipped and recorded, the others are computed; a bad page id is recorded."""
    case = Case([rows, rows, rows], [200, 150, 90], 4, 2, 64, 16, False, 1)
    good = case.on(dev)
    want = h3.paged_attn_fwd(**good)
    for what, status in (("used", 3), ("negative", 3), ("rows", 3), ("many", 3), ("long", 3), ("page", 12), ("below", 12)):
        a = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in good.items()}
        skipped = None
        if what == "used":
            a["seqused_k"][1], skipped = 16 * a["block_table"].shape[1] + 1, 1
        elif what == "negative":
            a["seqused_k"][1], skipped = -1, 1
        elif what == "rows":
            a["cu_seqlens_q"][1] = 4 * rows  # falls at the second segment, and too many rows in the first
        elif what == "many":
            a["max_seqlen_q"] = rows - 1
        elif what == "long":
            a["max_seqlen_k"] = 149  # computed all the same
        elif what == "page":
            a["block_table"][2, 1] = a["k_cache"].shape[0]
        else:
            a["block_table"][2, 1] = -3
        out = torch.full_like(a["q"], 5.0)
        h3.paged_attn_fwd(**a, out=out)
        torch.cuda.synchronize()
        assert h3.get_device_error(dev) == status, what
        if skipped is not None:
            at = [0, rows, 2 * rows, 3 * rows]
            for g in range(3):
                part = slice(at[g], at[g + 1])
                assert torch.all(out[part] == 5.0) if g == skipped else torch.equal(out[part], want[part]), (what, g)
        if what == "long":
            assert torch.equal(out[:case.n], want[:case.n])
        if what in ("page", "below"):
            assert torch.equal(out[:2 * rows], want[:2 * rows])
        if what == "many":
            assert torch.all(out == 5.0)
    out = h3.paged_attn_fwd(**good)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0 and torch.equal(out[:case.n], want[:case.n])


@pytest_gpu
@pytest.mark.parametrize("rows", [2, 40])
def test_empty_calls_and_no_pages(h3, dev, rows):
    i32 = dict(dtype=torch.int32, device=dev)
    q = torch.ones(rows, 4, 64, dtype=torch.bfloat16, device=dev)
    none = torch.zeros(0, 2, 16, 64, dtype=torch.bfloat16, device=dev)
    out, lse = h3.paged_attn_fwd(q, none, none, torch.zeros(1, 0, **i32), torch.tensor([0, rows], **i32),
                                 torch.zeros(1, **i32), rows, 0, return_lse=True)
    torch.cuda.synchronize()
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse)) and h3.get_device_error(dev) == 0
    out = torch.full_like(q, 5.0)
    h3.paged_attn_fwd(q, none, none, torch.zeros(1, 0, **i32), torch.tensor([0, rows], **i32), torch.ones(1, **i32), rows,
                      1, out=out)  # a token that no page can hold
    torch.cuda.synchronize()
    assert torch.all(out == 5.0) and h3.get_device_error(dev) == 3
    h3.paged_attn_fwd(q, none, none, torch.zeros(0, 0, **i32), torch.zeros(1, **i32), torch.zeros(0, **i32), 0, 0, out=out)
    torch.cuda.synchronize()
    assert torch.all(out == 5.0) and h3.get_device_error(dev) == 0


@pytest_gpu
@pytest.mark.parametrize("lq", [[2, 1], [40, 129]])
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_nan_key_reaches_the_rows_that_see_it_alone(h3, dev, lq, e4m3):
    case = Case(lq, [300, 280], 4, 2, 64, 32, e4m3, 1)
    a = case.on(dev)
    clean = h3.paged_attn_fwd(**a)
    p = lq[0] - 1  # the first segment's last token alone, at position 299 of its key head 1
    page = int(a["block_table"][0, 299 // 32])
    if e4m3:
        a["k_scale"][page, 1, 299 % 32] = 255
    else:
        a["k_cache"][page, 1, 299 % 32] = float("nan")
    out = h3.paged_attn_fwd(**a)
    torch.cuda.synchronize()
    assert torch.isnan(out[p, 2:]).all()
    keep = torch.ones(sum(lq), 4, dtype=torch.bool)
    keep[p, 2:] = False
    assert torch.equal(out[:case.n][keep], clean[:case.n][keep])


@pytest_gpu
@pytest.mark.parametrize("lq, lk", [([1, 2], [5000, 40]), ([200, 90], [1500, 2000])])
def test_strides_streams_graphs_and_two_calls_at_once(h3, dev, lq, lk):
    case = Case(lq, lk, 8, 2, 128, 32, True, 1)
    a = case.on(dev)
    out, lse = h3.paged_attn_fwd(**a, return_lse=True)
    wide = torch.full((a["q"].shape[0], 12, 128), 3.0, dtype=torch.bfloat16, device=dev)
    wide[:, 2:10] = a["q"]
    assert torch.equal(h3.paged_attn_fwd(**{**a, "q": wide[:, 2:10]})[:case.n], out[:case.n])
    torch.cuda.synchronize()
    streams, results = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            for _ in range(4):
                results.append(h3.paged_attn_fwd(**a, return_lse=True))
    torch.cuda.synchronize()
    for o, l in results:
        assert torch.equal(o[:case.n], out[:case.n]) and torch.equal(l[:, :case.n], lse[:, :case.n])
    # captured, then replayed on new contents: other lengths, other pages
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        o, l = h3.paged_attn_fwd(**a, return_lse=True)
    for step in (0, 1):
        a["seqused_k"].sub_(13 * step)
        a["q"][:case.n].mul_(1 - 0.5 * step)
        graph.replay()
        want, wl = h3.paged_attn_fwd(**a, return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(o[:case.n], want[:case.n]) and torch.equal(l[:, :case.n], wl[:, :case.n])
    assert h3.get_device_error(dev) == 0


@pytest_gpu
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [1, 30])
def test_cache_past_2_31_elements(h3, dev, e4m3, rows):
    """Pages whose first element lies past 2^31 and 2^32 elements."""
    h, d, page, pages = 8, 128, 256, 17000  # 4.46e9 elements
    case = Case([rows], [700], 16, h, d, page, e4m3, 1)
    a = case.on(dev)
    ids = [pages - 1, 8200, 16385]
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if name not in a:
            continue
        kind = torch.uint8 if a[name].dtype is torch.float8_e4m3fn else a[name].dtype
        big = torch.empty((pages, *a[name].shape[1:]), dtype=kind, device=dev)
        for i, p in enumerate(ids):
            big[p] = a[name].view(kind)[int(case.table[0, i])]
        a[name] = big.view(a[name].dtype)
    a["block_table"] = torch.tensor([ids], dtype=torch.int32, device=dev)
    out, lse = h3.paged_attn_fwd(**a, return_lse=True)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    case.check(out, lse)


@pytest_gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_wait_that_runs_out_ends_the_call(h3, dev, e4m3):
    """As in test_gpu_cross_timeout.py: the loader stops after three tiles, the waits end by their limit."""
    case = Case([200], [1500], 4, 2, 128, 64, e4m3, 1)
    a = case.on(dev)
    want = h3.paged_attn_fwd(**a)
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
    h3.set_wait_limit_ns(20_000_000)
    h3.debug_stall_loads(3)
    try:
        h3.paged_attn_fwd(**a)
        torch.cuda.synchronize()
        later = torch.full_like(a["q"], 7.0)
        h3.paged_attn_fwd(**a, out=later)  # leaves at once while the timeout is recorded
        torch.cuda.synchronize()
    finally:
        h3.debug_stall_loads(-1)
        h3.set_wait_limit_ns(0)
    assert torch.all(later == 7.0)
    assert h3.get_device_error(dev) == 7 and h3.get_device_error(dev) == 0
    assert torch.equal(h3.paged_attn_fwd(**a)[:case.n], want[:case.n])
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0
