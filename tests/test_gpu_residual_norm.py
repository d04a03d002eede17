"""residual_norm and its gradient on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (derived before the first run).  Everything is fp32 (E = 1e-5 covers the
chains: a row's sums are trees of under 30 steps of 2^-24, products a few steps each) and each result is
rounded once: bf16 by 2^-8 of the value at most, fp32 by 2^-24.  Errors carried along, with |.| of the values:
  * x' = alpha x + u:  d = E (|alpha x| + |u|), plus the error of u's norm, which is of the same form.
  * norm(x), an input error d: the centred row is off by c = d + mean d + E (|x| + mean |x|) (the means for a
    layer norm only), the factor by f = rms(c) rs + E of itself, so unit z by rs c + |z| f.
  * back through a norm, an input error eg of g and ez of z:
      rs (eg + mean eg + |z| mean(eg |z| + |g| ez) + ez mean |g z|) + E rs (|g| + mean |g| + |z| mean |g z|).
  * sums over tokens: the sum of the terms' errors, plus E times the sum of the terms' sizes (chains of
    under 100 rows a CTA, then a few).
"""
import numpy as np
import pytest
import torch

import oracle
from oracle.norm import _f64
from oracle.residual import requests_of, unit

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E = 1e-5
EPS = 1e-6
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


# ---- bounds ----------------------------------------------------------------------------------------


def _m(x):
    return x.mean(-1, keepdims=True)


def _unit_error(x, kind, d, eps):
    """(unit z, factor, error of z) of rows x that are off by d."""
    z, f = unit(x, kind, eps)
    if kind == "none":
        return z, f, d
    layer = kind == "layer"
    c = d + E * np.abs(x) + ((_m(d) + E * _m(np.abs(x))) if layer else 0.0)
    return z, f, f * c + np.abs(z) * (np.sqrt(_m(c * c)) * f + E)


def _back_error(g, eg, z, ez, f, kind):
    if kind == "none":
        return eg
    ag, az = np.abs(g), np.abs(z)
    return f * (eg + _m(eg) + az * _m(eg * az + ag * ez) + ez * _m(ag * az)) + E * f * (ag + _m(ag) + az * _m(ag * az))


def _near(got, ref, err, kind, what):
    got = _f64(got)
    tol = HALF[kind] * np.abs(ref) + (1 + HALF[kind]) * err
    assert got.shape == ref.shape, what
    assert np.all(np.isfinite(got)), what
    off = np.abs(got - ref)
    assert np.all(off <= tol), (what, (off - tol).max(), off.max())


def _check_fwd(x_out, h, x, y, step, eps=EPS):
    p = {k: None if v is None or isinstance(v, (str, float, list)) else _f64(v) for k, v in step.items()}
    xf = _f64(x)
    r, requests = requests_of(x.shape[0], step.get("cu_requests"))
    d = np.zeros(xf.shape)
    ref_x, ref_h = oracle.residual_norm(x, y, eps=eps, **step)
    if y is not None:
        yf = _f64(y)
        gate = np.ones(xf.shape) if p.get("gate") is None else p["gate"][r]
        if p.get("branch_weight") is not None:
            gate = gate * p["branch_weight"]
        z, _, ez = _unit_error(yf, step.get("branch_norm", "none"), np.zeros(yf.shape), eps)
        alpha = step.get("residual_scale", 1.0)
        d = ez * np.abs(gate) + E * (np.abs(alpha * xf) + np.abs(z * gate))
        _near(x_out, ref_x, d, x.dtype, "x_out")
    if step.get("norm", "rms") == "none":
        assert h is None
        return
    z, _, ez = _unit_error(ref_x, step.get("norm", "rms"), d, eps)
    gain = np.ones(xf.shape)
    if p.get("weight") is not None:
        gain = gain * p["weight"]
    if p.get("scale") is not None:
        gain = gain * (1 + p["scale"][r])
    shift = 0.0 if p.get("shift") is None else np.abs(p["shift"][r])
    _near(h, ref_h, ez * np.abs(gain) + E * (np.abs(z * gain) + shift), torch.bfloat16, "h")


def _check_bwd(g, dx_out, dh, x_out, y, step, eps=EPS):
    ref = oracle.residual_norm_grad(dx_out, dh, x_out, y, eps=eps, **step)
    n, dim = x_out.shape
    r, requests = requests_of(n, step.get("cu_requests"))
    one = np.ones((n, dim))
    vec = lambda k: None if step.get(k) is None else _f64(step[k])  # noqa: E731
    w = one if vec("weight") is None else one * vec("weight")
    sc = one if vec("scale") is None else 1 + vec("scale")[r]

    def sums(v):
        s = np.zeros((requests, dim))
        np.add.at(s, r, v)
        return s

    def small(name, got, terms, errors, per_request_factor):
        """A vector's gradient: sums of terms (already times the factor) over tokens."""
        if got is None:
            return
        size, err = sums(np.abs(terms) * np.abs(per_request_factor)), sums(errors * np.abs(per_request_factor))
        if got.dim() == 1:
            size, err = size.sum(0), err.sum(0)
        off = np.abs(_f64(got) - ref[name])
        assert np.all(off <= err + E * size + 1e-30), (name, (off - err - E * size).max())

    t, et = np.zeros((n, dim)) if dx_out is None else _f64(dx_out), np.zeros((n, dim))
    if step.get("norm", "rms") != "none":
        z, f, ez = _unit_error(_f64(x_out), step.get("norm", "rms"), np.zeros((n, dim)), eps)
        dhf = _f64(dh)
        gg = dhf * w * sc
        et = _back_error(gg, E * np.abs(gg), z, ez, f, step.get("norm", "rms")) + E * np.abs(t)
        terms, errors = dhf * z, np.abs(dhf) * ez
        small("shift", g.shift, dhf, np.zeros((n, dim)), one)
        small("scale", g.scale, terms, errors, w)
        small("weight", g.weight, terms, errors, sc)
    alpha = step.get("residual_scale", 1.0)
    t = ref["dx"] / alpha if alpha else t
    if alpha:
        _near(g.dx, ref["dx"], abs(alpha) * et + E * np.abs(ref["dx"]), x_out.dtype, "dx")
    if y is None:
        assert g.dy is None and g.gate is None
        return
    gate = one if vec("gate") is None else vec("gate")[r]
    wb = one if vec("branch_weight") is None else one * vec("branch_weight")
    kind = step.get("branch_norm", "none")
    z, f, ez = _unit_error(_f64(y), kind, np.zeros((n, dim)), eps)
    gy = t * wb * gate
    _near(g.dy, ref["dy"], _back_error(gy, et * np.abs(wb * gate) + E * np.abs(gy), z, ez, f, kind) +
          E * np.abs(ref["dy"]), torch.bfloat16, "dy")
    terms, errors = t * z, et * np.abs(z) + np.abs(t) * ez
    small("gate", g.gate, terms, errors, wb)
    small("branch_weight", g.branch_weight, terms, errors, gate)


# ---- refusals (no GPU) -------------------------------------------------------------------------------


def _desc(h3, **kw):
    base = dict(num_tokens=2, dim=64, num_requests=1, norm=1, branch_norm=0, stream_type=1, residual_scale=1.0)
    return h3._ResidualNormDesc(**{**base, **kw})


@pytest.mark.parametrize("kw, status", [
    (dict(num_tokens=-1), 2), (dict(dim=0), 2), (dict(dim=-8), 2), (dict(num_requests=0), 2), (dict(num_requests=2), 2),
    (dict(norm=3), 2), (dict(norm=-1), 2), (dict(branch_norm=3), 2), (dict(stream_type=2), 2), (dict(weight_type=2), 2),
    (dict(mod_type=-1), 2), (dict(eps=float("nan")), 2), (dict(residual_scale=float("inf")), 2), (dict(dim=68), 4),
    (dict(dim=8200), 4), (dict(x_stride=56), 2), (dict(x_stride=68), 8), (dict(y_stride=65), 8), (dict(h_stride=-64), 2),
    (dict(gate_stride=66), 8), (dict(x_out_stride=1 << 40), 2), (dict(norm=0), 1),
])
def test_c_abi_refuses(h3, kw, status):
    import ctypes as C

    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    d = _desc(h3, **kw)
    lib = h3.load_library()
    assert lib.h3_residual_norm(C.byref(d), p, p, None, None, None, None, None, None, p, p, None) == status


def test_c_abi_refuses_pointers(h3):
    import ctypes as C

    lib = h3.load_library()
    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    odd = C.c_void_p(p.value + 8)
    d, none = _desc(h3), _desc(h3, norm=0)
    fwd = lambda d, *a: lib.h3_residual_norm(C.byref(d), *a, None)  # noqa: E731
    assert lib.h3_residual_norm(None, p, p, *(None,) * 6, p, p, None) == 1
    assert fwd(d, None, p, *(None,) * 6, p, p) == 1
    assert fwd(d, p, p, *(None,) * 6, None, p) == 1       # y without x_out
    assert fwd(d, p, None, *(None,) * 6, p, p) == 1       # x_out without y
    assert fwd(d, p, p, *(None,) * 6, p, None) == 1       # a norm without h
    assert fwd(none, p, None, *(None,) * 6, None, None) == 2  # nothing to do
    assert fwd(none, p, p, p, *(None,) * 5, p, None) == 2  # a weight that no norm uses
    assert fwd(d, p, None, None, None, None, None, p, None, None, p) == 2  # a gate without y
    assert fwd(_desc(h3, residual_scale=0.5), p, None, *(None,) * 6, None, p) == 2
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9):
        a = [p, p, p, p, p, p, p, None, p, p]
        a[i] = odd
        assert fwd(d, *a) == 8, i
    assert fwd(d, p, p, None, None, None, None, None, C.c_void_p(p.value + 2), p, p) == 8
    bwd = lambda d, *a: lib.h3_residual_norm_bwd(C.byref(d), *a, None)  # noqa: E731
    head, tail = (p, p, p, p) + (None,) * 5, (None,) * 5
    assert bwd(d, *head, p, p, *tail, None, 0) == 5
    assert bwd(d, *head, p, p, *tail, p, 64) == 5
    assert bwd(d, *head, None, p, *tail, p, 1 << 30) == 1
    assert bwd(d, *head, p, None, *tail, p, 1 << 30) == 1
    assert bwd(d, p, None, *head[2:], p, p, *tail, p, 1 << 30) == 1
    assert bwd(none, None, None, *head[2:], p, p, *tail, p, 1 << 30) == 1
    assert bwd(none, p, None, *head[2:], p, p, p, *tail[1:], p, 1 << 30) == 2  # dweight without a norm
    assert bwd(d, *head, p, p, odd, *tail[1:], odd, 1 << 30) == 8
    assert lib.h3_residual_norm_bwd_workspace_size(C.byref(_desc(h3, dim=0))) == 0
    assert lib.h3_residual_norm_bwd_workspace_size(None) == 0


def test_binding_refuses(h3):
    x, y, v = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(1, 64)
    bad = [
        (TypeError, dict(x=x.double())), (TypeError, dict(x=x.half())), (TypeError, dict(x=None)),
        (ValueError, dict(x=x[0])), (ValueError, dict(x=torch.zeros(64, 4).t())), (ValueError, dict(y=y[:3])),
        (TypeError, dict(y=x)), (ValueError, dict(norm="batch")), (ValueError, dict(branch_norm="l2")),
        (ValueError, dict(y=None, gate=v)), (ValueError, dict(y=None, residual_scale=0.5)),
        (ValueError, dict(y=None, branch_norm="rms")), (ValueError, dict(y=None, norm="none")),
        (ValueError, dict(norm="none", scale=v)), (ValueError, dict(norm="none", h_out=y)),
        (ValueError, dict(weight=torch.ones(32))), (TypeError, dict(weight=torch.ones(64).double())),
        (TypeError, dict(weight=torch.ones(64), branch_weight=torch.ones(64, dtype=torch.bfloat16))),
        (ValueError, dict(scale=torch.zeros(2, 64))), (ValueError, dict(gate=torch.zeros(64))),
        (TypeError, dict(scale=v, gate=v.bfloat16())), (TypeError, dict(shift=[0.0] * 64)),
        (ValueError, dict(num_tokens=5)), (ValueError, dict(num_tokens=-1)),
        (ValueError, dict(cu_requests=torch.tensor([0], dtype=torch.int32))), (TypeError, dict(cu_requests=torch.tensor([0, 4]))),
        (ValueError, dict(x_out=torch.zeros(3, 64))), (TypeError, dict(x_out=y)), (TypeError, dict(h_out=x)),
        (ValueError, dict(y=None, x_out=x)),
    ]
    for error, kw in bad:
        a = {**dict(x=x, y=y), **kw}
        with pytest.raises(error):
            h3.residual_norm(a.pop("x"), a.pop("y"), **a)
    with pytest.raises(ValueError):
        h3.residual_norm_bwd(None, None, x, y, norm="none")
    with pytest.raises(ValueError):
        h3.residual_norm_bwd(x, y, x, y, norm="none")
    with pytest.raises(TypeError):
        h3.residual_norm_bwd(x, None, x, y)
    with pytest.raises(TypeError):
        h3.residual_norm_bwd(y, y, x, y)
    with pytest.raises(ValueError):
        h3.residual_norm_bwd(x, y, x, None, dy=y)


def test_no_tokens_at_all(h3):
    x, y = torch.zeros(0, 64), torch.zeros(0, 64, dtype=torch.bfloat16)
    s, h = h3.residual_norm(x, y)
    assert s.shape == x.shape and h.shape == x.shape
    g = h3.residual_norm_bwd(x, y, x, y, weight=torch.ones(64), gate=torch.ones(1, 64))
    assert torch.equal(g.weight, torch.zeros(64)) and torch.equal(g.gate, torch.zeros(1, 64)) and g.scale is None


# ---- GPU ---------------------------------------------------------------------------------------------

# tokens, dim, offsets of the requests, norm, branch norm, weights, modulation, stream, has y, alpha, seed
SHAPES = [
    (1, 8, None, "rms", "none", None, None, torch.bfloat16, False, 1.0),
    (1, 5120, [0, 1], "layer", "none", None, torch.bfloat16, torch.bfloat16, True, 1.0),
    (3, 72, [0, 0, 2, 2, 3], "layer", "rms", torch.float32, torch.float32, torch.float32, True, 0.5),
    (5, 264, None, "rms", "layer", torch.bfloat16, torch.bfloat16, torch.bfloat16, True, -1.25),
    (45, 2560, [0, 10, 30, 45], "rms", "rms", torch.float32, torch.bfloat16, torch.bfloat16, True, 1.0),
    (317, 1000, [0, 317], "layer", "layer", torch.bfloat16, torch.float32, torch.float32, True, 0.75),
    (701, 520, [0, 1, 2, 300, 300, 699, 701], "rms", "none", None, torch.float32, torch.bfloat16, True, 1.0),
    (611, 2568, [0, 305, 306, 611], "layer", "rms", torch.float32, torch.bfloat16, torch.float32, True, 2.0),
    (160, 5128, [0, 80, 160], "rms", "rms", torch.float32, torch.float32, torch.bfloat16, True, 1.0),
    (155, 8192, [0, 152, 155], "layer", "layer", torch.bfloat16, torch.bfloat16, torch.float32, True, 1.0),
    (400, 1536, [0, 7, 400], "none", "rms", torch.float32, torch.bfloat16, torch.bfloat16, True, 0.5),
    (331, 512, [0, 331], "layer", "none", torch.float32, torch.float32, torch.float32, False, 1.0),
    (1300, 40, list(range(0, 1301, 2)), "rms", "none", torch.float32, torch.bfloat16, torch.bfloat16, True, 1.0),
]


def _rand(rng, *shape, kind=torch.bfloat16, scale=1.0, at=0.0):
    return torch.from_numpy(at + scale * rng.standard_normal(shape)).to(kind)


def _case(shape, seed=0, far=0.0):
    n, dim, cu, norm, branch_norm, weights, mod, stream, has_y, alpha = shape
    rng = np.random.default_rng(seed)
    x = _rand(rng, n, dim, kind=stream, scale=2.0, at=far)
    y = _rand(rng, n, dim, scale=1.5, at=far) if has_y else None
    step = dict(norm=norm, branch_norm=branch_norm, residual_scale=alpha, cu_requests=cu)
    if weights is not None and norm != "none":
        step["weight"] = _rand(rng, dim, kind=weights, scale=0.3, at=1.0)
    if weights is not None and has_y:
        step["branch_weight"] = _rand(rng, dim, kind=weights, scale=0.3, at=1.0)
    if mod is not None:
        requests = 1 if cu is None else len(cu) - 1
        wide = _rand(rng, requests, 6, dim, kind=mod, scale=0.5)  # the six vectors of a block; these are three of them
        if norm != "none":
            step["shift"], step["scale"] = wide[:, 3], wide[:, 4]
        if has_y:
            step["gate"] = wide[:, 2]
    return x, y, step


def _on(dev, step):
    return {k: torch.tensor(v, dtype=torch.int32, device=dev) if isinstance(v, list) else
            v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in step.items()}


def _clean(h3, dev):
    torch.cuda.synchronize()
    assert h3.get_device_error(dev) == 0


@pytest_gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(h3, dev, shape):
    x, y, step = _case(shape)
    s, h = h3.residual_norm(x.to(dev), None if y is None else y.to(dev), **_on(dev, step))
    _clean(h3, dev)
    _check_fwd(s.cpu(), None if h is None else h.cpu(), x, y, step)


@pytest_gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(h3, dev, shape):
    x, y, step = _case(shape, seed=1)
    rng = np.random.default_rng(2)
    n, dim = x.shape
    dx_out = _rand(rng, n, dim, kind=x.dtype) if shape[3] == "none" or n % 2 else None
    dh = None if shape[3] == "none" else _rand(rng, n, dim)
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    g = h3.residual_norm_bwd(to(dx_out), to(dh), x.to(dev), to(y), **_on(dev, step))
    again = h3.residual_norm_bwd(to(dx_out), to(dh), x.to(dev), to(y), **_on(dev, step))
    _clean(h3, dev)
    for a, b in zip(g, again):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    _check_bwd(h3.ResidualNormGrads(*(None if t is None else t.cpu() for t in g)), dx_out, dh, x, y, step)
    for name in ("weight", "branch_weight", "scale", "shift", "gate"):
        assert (getattr(g, name) is None) == (step.get(name) is None)


@pytest_gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_large_means_and_tiny_rows(h3, dev, kind):
    """A layer norm of rows far from zero keeps its digits; rows of zeros come out as the shift."""
    shape = (64, 1024, None, kind, "layer", torch.float32, torch.float32, torch.float32, True, 1.0)
    x, y, step = _case(shape, seed=3, far=300.0)
    x[5] = 0.0
    y[5] = 0.0
    x[6] *= 1e-20
    y[6] *= 1e-20
    s, h = h3.residual_norm(x.to(dev), y.to(dev), **_on(dev, step))
    _clean(h3, dev)
    _check_fwd(s.cpu(), h.cpu(), x, y, step)
    if kind == "layer":
        assert torch.equal(h[5].cpu(), step["shift"][0].bfloat16())


@pytest_gpu
def test_strided_rows_padding_and_in_place(h3, dev):
    shape = (37, 512, [0, 20, 37], "layer", "rms", torch.float32, torch.bfloat16, torch.bfloat16, True, 1.0)
    x, y, step = _case(shape, seed=4)
    want_s, want_h = h3.residual_norm(x.to(dev), y.to(dev), **_on(dev, step))
    # rows inside wider ones, more rows than tokens, results in place of x and y
    wide = torch.full((50, 3, 512), 7.0, dtype=torch.bfloat16, device=dev)
    wide[:37, 0], wide[:37, 2] = x.to(dev), y.to(dev)
    xs, ys = wide[:, 0], wide[:, 2]
    s, h = h3.residual_norm(xs, ys, **_on(dev, step), num_tokens=37, x_out=xs, h_out=ys)
    _clean(h3, dev)
    assert s is xs and h is ys and torch.equal(s[:37], want_s) and torch.equal(h[:37], want_h)
    assert torch.all(wide[37:] == 7.0) and torch.all(wide[:, 1] == 7.0)
    rng = np.random.default_rng(5)
    dxo, dh = _rand(rng, 37, 512).to(dev), _rand(rng, 37, 512).to(dev)
    want = h3.residual_norm_bwd(dxo, dh, want_s, y.to(dev), **_on(dev, step))
    wide = torch.full((50, 4, 512), 7.0, dtype=torch.bfloat16, device=dev)
    for i, t in enumerate((dxo, dh, want_s, y.to(dev))):
        wide[:37, i] = t
    a, b, c, d = (wide[:, i] for i in range(4))
    ws = torch.empty(h3.residual_norm_bwd_workspace_size(37, 512, 2), dtype=torch.uint8, device=dev)
    got = h3.residual_norm_bwd(a, b, c, d, **_on(dev, step), num_tokens=37, dx=a, dy=d, workspace=ws)
    _clean(h3, dev)
    assert torch.equal(got.dx[:37], want.dx) and torch.equal(got.dy[:37], want.dy)
    for k in ("weight", "branch_weight", "scale", "shift", "gate"):
        assert torch.equal(getattr(got, k), getattr(want, k))
    assert torch.all(wide[37:] == 7.0) and torch.equal(wide[:37, 1], dh) and torch.equal(wide[:37, 2], want_s)


@pytest_gpu
def test_infinities_and_nan_stay_in_their_row(h3, dev):
    shape = (40, 256, [0, 40], "rms", "rms", torch.float32, torch.float32, torch.bfloat16, True, 1.0)
    x, y, step = _case(shape, seed=6)
    want_s, want_h = h3.residual_norm(x.to(dev), y.to(dev), **_on(dev, step))
    x[3, 5], y[9, 200] = float("inf"), float("nan")
    s, h = h3.residual_norm(x.to(dev), y.to(dev), **_on(dev, step))
    _clean(h3, dev)
    keep = [i for i in range(40) if i not in (3, 9)]
    assert torch.equal(s[keep], want_s[keep]) and torch.equal(h[keep], want_h[keep])
    assert torch.isnan(s[9]).all() and torch.isinf(s[3, 5]) and torch.isnan(h[3, 5])


@pytest_gpu
def test_rows_past_2_31_elements(h3, dev):
    n, dim = 262_200, 8192  # the last rows start past 2^31 elements
    x = torch.zeros(n, dim, dtype=torch.bfloat16, device=dev)
    x[-2:] = _rand(np.random.default_rng(7), 2, dim).to(dev)
    _, h = h3.residual_norm(x, norm="rms")
    _clean(h3, dev)
    _check_fwd(None, h[-2:].cpu(), x[-2:].cpu(), None, dict(norm="rms"))
    assert torch.all(h[:-2:5000] == 0)


@pytest_gpu
def test_streams_graphs_and_two_calls_at_once(h3, dev):
    shape = (300, 1024, [0, 100, 300], "layer", "rms", torch.float32, torch.bfloat16, torch.bfloat16, True, 1.0)
    x, y, step = _case(shape, seed=8)
    x, y, step = x.to(dev), y.to(dev), _on(dev, step)
    rng = np.random.default_rng(9)
    dxo, dh = _rand(rng, 300, 1024).to(dev), _rand(rng, 300, 1024).to(dev)
    s, h = h3.residual_norm(x, y, **step)
    want = h3.residual_norm_bwd(dxo, dh, s, y, **step)
    torch.cuda.synchronize()
    # two streams, each with its own workspace
    streams, results = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            a = h3.residual_norm(x, y, **step)
            results.append((a, h3.residual_norm_bwd(dxo, dh, a[0], y, **step)))
    torch.cuda.synchronize()
    for (a, b), g in results:
        assert torch.equal(a, s) and torch.equal(b, h)
        assert all(torch.equal(p, q) for p, q in zip(g, want))
    # captured and replayed on new contents
    xs, graph = x.clone(), torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        h3.residual_norm_bwd(dxo, dh, h3.residual_norm(xs, y, **step)[0], y, **step)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        s2, h2 = h3.residual_norm(xs, y, **step)
        g2 = h3.residual_norm_bwd(dxo, dh, s2, y, **step)
    xs.copy_(x * 0.5)
    graph.replay()
    s3, h3_ = h3.residual_norm(xs, y, **step)
    g3 = h3.residual_norm_bwd(dxo, dh, s3, y, **step)
    torch.cuda.synchronize()
    assert torch.equal(s2, s3) and torch.equal(h2, h3_) and all(torch.equal(p, q) for p, q in zip(g2, g3))
