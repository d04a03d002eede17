"""Pins of the oracle's residual-norm step and paged cache: closed forms, differences, a table of e4m3."""
import numpy as np
import pytest
import torch

import oracle
from oracle.paged import key_limit

ALL = ["dx", "dy", "weight", "branch_weight", "scale", "shift", "gate"]


def _step(rng, n=7, dim=16, requests=3):
    return dict(weight=1 + 0.3 * rng.standard_normal(dim), branch_weight=1 + 0.3 * rng.standard_normal(dim),
                scale=rng.standard_normal((requests, dim)), shift=rng.standard_normal((requests, dim)),
                gate=rng.standard_normal((requests, dim)), residual_scale=0.7, cu_requests=[0, 2, 2, n])


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("branch_norm", ["none", "rms", "layer"])
def test_residual_norm_gradient_is_that_of_differences(norm, branch_norm):
    rng = np.random.default_rng(5)
    n, dim = 7, 16
    x, y = rng.standard_normal((n, dim)) + 0.4, 2 * rng.standard_normal((n, dim))
    p = dict(x=x, y=y, **_step(rng))
    a, b = rng.standard_normal((n, dim)), rng.standard_normal((n, dim))

    def value(q):
        s, h = oracle.residual_norm(q["x"], q["y"], norm=norm, branch_norm=branch_norm,
                                    **{k: v for k, v in q.items() if k not in "xy"})
        return (a * s).sum() + (b * h).sum()

    step = {k: v for k, v in p.items() if k not in "xy"}
    x_out, _ = oracle.residual_norm(x, y, norm=norm, branch_norm=branch_norm, **step)
    grads = oracle.residual_norm_grad(a, b, x_out, y, norm=norm, branch_norm=branch_norm, **step)
    for name in ALL:
        key = name[1:] if name in ("dx", "dy") else name
        d = rng.standard_normal(np.shape(p[key]))
        t = 1e-5
        slope = (value({**p, key: p[key] + t * d}) - value({**p, key: p[key] - t * d})) / (2 * t)
        assert abs(slope - (grads[name] * d).sum()) <= 1e-7 * max(1.0, abs(slope)), name


def test_residual_norm_closed_forms():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    s, h = oracle.residual_norm(x, norm="rms", eps=0.0)
    assert s is not None and np.allclose(h, x / 2.5)  # rms of (3, 4, 0, 0) is 2.5
    _, h = oracle.residual_norm(x + 100.0, norm="layer", eps=0.0)
    assert np.allclose(h.mean(), 0.0) and np.allclose((h * h).mean(), 1.0)
    s, h = oracle.residual_norm(x, np.ones((1, 4)), norm="none", gate=np.full((1, 4), 2.0), residual_scale=0.5)
    assert h is None and np.array_equal(s, [[3.5, 4.0, 2.0, 2.0]])


def _e4m3_table():
    """The finite values that sign, four exponent bits with bias 7 and three mantissa bits stand for."""
    table = []
    for e in range(16):
        for m in range(8):
            if e == 15 and m == 7:
                continue  # NaN
            table.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(sorted({s * t for t in table for s in (1, -1)}))


def test_e4m3_rounding_is_to_the_nearest_value_with_ties_to_even():
    table = _e4m3_table()
    assert table.max() == 448 and len(table) == 253
    assert np.array_equal(oracle.e4m3_round(table), table)
    x = np.random.default_rng(1).standard_normal(4000) * 2.0 ** np.random.default_rng(2).integers(-12, 8, 4000)
    x = x[np.abs(x) < 448]
    got, off = oracle.e4m3_round(x), np.abs(x[:, None] - table)
    assert np.array_equal(np.abs(x - got), off.min(1)) and np.isin(got, table).all()
    mid = (table[1:] + table[:-1]) / 2
    lower_even = (np.arange(len(mid)) - np.flatnonzero(table == 0)[0]) % 2 == 0
    assert np.array_equal(oracle.e4m3_round(mid), np.where(lower_even, table[:-1], table[1:]))
    # torch's own type, another statement of the same format
    t = torch.from_numpy(x).float()
    assert np.array_equal(t.to(torch.float8_e4m3fn).double().numpy(), oracle.e4m3_round(t.double().numpy()))


def test_row_scale_is_the_least_that_holds_the_row():
    for most, e in ((448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (1.75, -8), (1.76, -7), (0.0, -110),
                    (2.0 ** 127, 119), (2.0 ** -126, -110)):
        assert oracle.e4m3_scale(np.array([[most, 0.0, -most / 3]])) == e, most
    x = np.array([[448.0, 1.0, 2.0 ** -9, 2.0 ** -11]])
    assert np.array_equal(oracle.e4m3_row_values(x), [[448.0, 1.0, 2.0 ** -9, 0.0]])


def test_key_limits():
    assert [key_limit(p, 10, 1) for p in range(4)] == [1, 2, 3, 4]
    assert [key_limit(p, 10, 4) for p in (0, 3, 4, 7, 8, 9)] == [4, 4, 8, 8, 10, 10]
    assert [key_limit(p, 10, 0) for p in (0, 9)] == [10, 10]
    assert [key_limit(p, 3, 4) for p in (-1, -4, -5)] == [0, 0, 0]


def test_paged_attention_against_one_row_at_a_time():
    rng = np.random.default_rng(3)
    used, cu = [9, 2, 0], [0, 4, 7, 8]  # the second segment has a row more than it has keys, the third no key
    q = rng.standard_normal((9, 4, 8))
    k, v = ([rng.standard_normal((n, 2, 8)) for n in used] for _ in range(2))
    o, lse = oracle.paged_attention(q, k, v, cu, used, block=2)
    for g in range(3):
        for i in range(cu[g], cu[g + 1]):
            p = used[g] - (cu[g + 1] - cu[g]) + (i - cu[g])
            n = min(used[g], max(0, (p // 2 + 1) * 2))
            for h in range(4):
                if n == 0:
                    assert np.all(o[i, h] == 0) and lse[h, i] == -np.inf
                    continue
                s = k[g][:n, h // 2] @ q[i, h] / np.sqrt(8)
                w = np.exp(s) / np.exp(s).sum()
                assert np.allclose(o[i, h], w @ v[g][:n, h // 2]) and np.isclose(lse[h, i], np.log(np.exp(s).sum()))
    assert np.isnan(o[8]).all()
