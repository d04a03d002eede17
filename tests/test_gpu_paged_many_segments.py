"""Attention over a paged cache for many short streams: more (segment, key head) pairs a CTA than its list holds at
once, more segments than a scan takes, and an e4m3 cache of more pages than one round of the unpacking warps and more
segments than one of their counts.  Cases and tolerances as in test_gpu_paged_attn.py."""
import numpy as np
import pytest
import torch

from test_gpu_paged_attn import Case, _run, dev, h3  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3, heads", [(False, 8), (False, 16), (True, 8), (True, 16), (True, 96)])
def test_more_pairs_than_a_list_holds(h3, dev, e4m3, heads, d):  # noqa: F811
    # 1,000 streams x 8 key heads, a unit each: 26 and more pairs to each of 304 CTAs, 16 of them listed at once.
    # Some streams have no new row, some no cached token, a few several units.
    rng = np.random.default_rng(heads + d)
    lk = [int(x) for x in rng.integers(1, 61, 1000)]
    lq = [1] * 1000
    for g in range(0, 1000, 37):
        lq[g] = 0
    for g in range(5, 1000, 97):
        lk[g] = 0
    for g in range(11, 1000, 199):
        lk[g] = int(rng.integers(300, 1500))
    case = Case(lq, lk, heads, 8, d, 16, e4m3, 1, seed=d)
    out, lse = _run(h3, dev, case)
    case.check(out, lse)
    again, lse2 = _run(h3, dev, case)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_unpacking_many_segments_and_pages(h3, dev, d):  # noqa: F811
    # 8 warps x 8 CTAs an SM take 9,728 of the parts at once: two a page of 16 and key head, of K and of V
    rng = np.random.default_rng(d)
    lk = [int(x) for x in rng.integers(100, 700, 75)]
    lq = [int(x) for x in rng.integers(0, 9, 75)]
    lq[40], lk[40] = 530, 900
    for g in (0, 31, 32, 33, 63, 64):
        lq[g] = 0
    parts = sum(-(-n // 16) * 2 * 8 for q, n in zip(lq, lk) if q)
    assert parts > 2 * 9728
    case = Case(lq, lk, 8, 8, d, 16, True, 1, seed=d)
    a = case.on(dev)
    sizes = [h3.paged_attn_workspace_size(75, case.max_q, case.max_k, a["q"].shape[0], 8, 8, d, 16, e4m3=e,
                                          max_pages=a["block_table"].shape[1]) for e in (False, True)]
    assert sizes[1] > sizes[0]
    space = torch.full((sizes[1],), 255, dtype=torch.uint8, device=dev)  # NaN wherever the call does not write
    out, lse = _run(h3, dev, case, workspace=space)
    case.check(out, lse)
    again, lse2 = _run(h3, dev, case, workspace=space[:sizes[0]].fill_(255))  # converted as it is read
    assert torch.equal(out, again) and torch.equal(lse, lse2)
