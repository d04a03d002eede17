"""Attention over a paged cache on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (derived before the first run).  The cache's values are exact in bf16, so
both sides start from the same keys and values.  S and the sums are fp32; the weights are rounded to bf16
(half a step, 2^-8 of each) before the product with V, and o is rounded to bf16 once more:
    |o - o*| <= 2^-8 sum_j P_j |v_j| + 2^-8 |o| + fp32 terms,
fp32 terms: the score's error (D products, 2^-24 each of |q||k|, and the exponential's 2^-22) moves each weight
by under 1e-4 of itself at the scores used here: 2e-4 sum_j P_j |v_j|.
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
    for rows in (2,):
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
        tol = (HALF + 2e-4) * size + HALF * np.abs(ref)
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
