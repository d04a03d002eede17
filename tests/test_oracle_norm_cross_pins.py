"""Pins of the fp64 norm and cross attention oracles: closed forms, the oracles of the parts they
are made of, and central differences for every gradient."""
import numpy as np
import pytest

import oracle

RNG = np.random.default_rng


def _tokens(n, seed):
    rng = RNG(seed)
    pos = np.stack([rng.integers(0, 30, n), rng.integers(0, 9, n), rng.integers(0, 9, n)], 1).astype(np.float32)
    return pos, (np.arange(n) % 3).astype(np.uint8)


def _difference(f, x, at, h=1e-5):
    a, b = x.copy(), x.copy()
    a[at] += h
    b[at] -= h
    return (f(a) - f(b)) / (2 * h)


def test_norm_gives_unit_mean_square_and_ignores_scale():
    x = RNG(0).standard_normal((5, 3, 64))
    y = oracle.norm_rope(x, np.ones(64), eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    assert np.allclose(oracle.norm_rope(7.0 * x, np.ones(64), eps=0.0), y)


def test_norm_of_a_zero_row_is_zero():
    assert np.all(oracle.norm_rope(np.zeros((2, 1, 64)), np.ones(64)) == 0.0)


def test_norm_rope_is_rope_of_the_norm():
    n = 7
    pos, tag = _tokens(n, 1)
    x, w = RNG(2).standard_normal((n, 2, 64)), RNG(3).standard_normal(64)
    z = oracle.norm_rope(x, w)
    ref = oracle.rope_apply(z, pos, tag, [0, 3, n], [119.0, 238.0])
    got = oracle.norm_rope(x, w, pos, tag, [0, 3, n], [119.0, 238.0])
    assert np.allclose(got, ref, atol=1e-12)


@pytest.mark.parametrize("rotate", [False, True])
def test_norm_gradient_matches_differences(rotate):
    n, d = 4, 64
    pos, tag = _tokens(n, 4) if rotate else (None, None)
    rng = RNG(5)
    x, w, dy = rng.standard_normal((n, 2, d)), rng.standard_normal(d), rng.standard_normal((n, 2, d))
    dx, dw = oracle.norm_rope_grad(dy, x, w, pos, tag)
    for at in [(0, 0, 0), (1, 1, 17), (3, 0, 63)]:
        num = _difference(lambda v: (oracle.norm_rope(v, w, pos, tag) * dy).sum(), x, at)
        assert abs(num - dx[at]) < 1e-7
    for at in [(0,), (31,), (63,)]:
        num = _difference(lambda v: (oracle.norm_rope(x, v, pos, tag) * dy).sum(), w, at)
        assert abs(num - dw[at]) < 1e-7


def test_cross_with_equal_offsets_is_the_packed_self_attention():
    rng = RNG(6)
    q, k, v = (rng.standard_normal((45, 2, 64)) for _ in range(3))
    cu = [0, 10, 30, 45]
    o, lse = oracle.cross_attention(q, k, v, cu, cu)
    ro, rl = oracle.varlen_attention(q, k, v, cu)
    assert np.allclose(o, ro, atol=1e-12) and np.allclose(lse, rl, atol=1e-12)


def test_cross_shares_key_heads_and_skips_unused_keys():
    rng = RNG(7)
    q, k, v = rng.standard_normal((5, 4, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    cu_q, cu_k, used = [0, 2, 5], [0, 4, 9], [3, 2]
    o, lse = oracle.cross_attention(q, k, v, cu_q, cu_k, used)
    k2, v2 = k.copy(), v.copy()
    for rows in (slice(3, 4), slice(6, 9)):
        k2[rows], v2[rows] = np.nan, np.inf
    o2, lse2 = oracle.cross_attention(q, k2, v2, cu_q, cu_k, used)
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)
    one, _ = oracle.cross_attention(q[:, 3:], k[:, 1:], v[:, 1:], cu_q, cu_k, used)
    assert np.allclose(o[:, 3:], one, atol=1e-13)


def test_cross_of_a_segment_without_keys():
    q, k = np.ones((3, 1, 64)), np.ones((2, 1, 64))
    o, lse = oracle.cross_attention(q, k, k, [0, 1, 3], [0, 2, 2])
    assert np.all(o[1:] == 0.0) and np.all(lse[0, 1:] == -np.inf)
    assert np.allclose(o[0], 1.0) and np.isclose(lse[0, 0], 8.0 + np.log(2.0))
    dq, dk, dv = oracle.cross_attention_grad(q, q, k, k, [0, 1, 3], [0, 2, 2])
    assert np.all(dq[1:] == 0.0) and np.allclose(dv, 0.5) and np.allclose(dk, 0.0)


def test_cross_gradient_matches_differences():
    rng = RNG(8)
    q, k, v = rng.standard_normal((5, 4, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    do = rng.standard_normal(q.shape)
    cu_q, cu_k, used = [0, 2, 5], [0, 4, 9], [4, 3]

    def value(q, k, v):
        return (oracle.cross_attention(q, k, v, cu_q, cu_k, used)[0] * do).sum()

    dq, dk, dv = oracle.cross_attention_grad(do, q, k, v, cu_q, cu_k, used)
    for at in [(0, 0, 0), (1, 3, 17), (4, 2, 63)]:
        assert abs(_difference(lambda x: value(x, k, v), q, at) - dq[at]) < 1e-7
    for at in [(0, 0, 0), (5, 1, 17), (6, 0, 63), (8, 1, 5)]:
        assert abs(_difference(lambda x: value(q, x, v), k, at) - dk[at]) < 1e-7
        assert abs(_difference(lambda x: value(q, k, x), v, at) - dv[at]) < 1e-7
