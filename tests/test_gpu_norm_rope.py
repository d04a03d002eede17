"""qk_norm_rope and its gradient on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (derived before the first run).  The kernels compute in fp32 and
round each bf16 result once, by at most half a step: 2^-8 of the value, plus the fp32 error d.
  * y: x^2 summed over D, rsqrt, two products and a rotation are under 2^-24 * 100 = 6e-6 of the
    pair's length, and the angle (1e-7 turns) adds 6e-7 of it: d = 1e-5 * |pair|.
  * dx = r (g - u mean(g u)): each of the two terms carries the same relative error, so
    d = 2e-5 * r * (|g's pair| + |u| mean|g u|).
  * dw: fp32 terms with relative error under 1e-6, added in chains of at most about 100 terms
    (2^-24 each): 1e-5 * sum |dz u|.
"""
import numpy as np
import pytest
import torch

import oracle

HALF = 2.0 ** -8  # half a bf16 step, relative


def _tokens(n, seed, far=0):
    rng = np.random.default_rng(seed)
    pos = np.stack([rng.integers(0, 600, n) + far, rng.integers(0, 48, n), rng.integers(0, 84, n)], 1)
    return pos.astype(np.float32), rng.integers(0, 4, n).astype(np.uint8)


def _pair_norm(x):
    p = np.hypot(x[..., 0::2], x[..., 1::2])
    return np.repeat(p, 2, axis=-1)


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def _check_y(got, x, w, where, eps=1e-6):
    ref = oracle.norm_rope(x, w, eps=eps, **where)
    tol = HALF * np.abs(ref) + (1 + HALF) * 1e-5 * _pair_norm(ref)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), (err - tol).max()


def _check_grad(dx, dw, dy, x, w, where, eps=1e-6):
    rdx, rdw = oracle.norm_rope_grad(dy, x, w, eps=eps, **where)
    dz = oracle.norm.rotate_pairs(oracle.norm._f64(dy), -oracle.norm._phi(
        x.shape[0], x.shape[2], where.get("pos"), where.get("tag"), where.get("cu_requests"),
        where.get("start_frames"), where.get("cfg")))
    xf, wf = oracle.norm._f64(x), oracle.norm._f64(w)
    r = 1.0 / np.sqrt((xf * xf).mean(-1, keepdims=True) + eps)
    u, g = xf * r, _pair_norm(dz) * np.abs(wf)
    size = r * (g + np.abs(u) * np.abs(g * u).mean(-1, keepdims=True))
    err = np.abs(dx.double().cpu().numpy() - rdx)
    tol = HALF * np.abs(rdx) + (1 + HALF) * 2e-5 * size
    assert np.all(err <= tol), (err - tol).max()
    assert np.all(np.abs(dw.double().cpu().numpy() - rdw) <= 1e-5 * np.abs(dz * u).sum((0, 1)) + 1e-30)


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


# ---- refusals (no GPU) ---------------------------------------------------------------------------


def _desc(h3, **kw):
    base = dict(num_tokens=2, num_q_heads=2, num_k_heads=0, head_dim=64, weight_type=0, eps=1e-6)
    return h3._QkNormDesc(**{**base, **kw})


@pytest.mark.parametrize("kw, status", [
    (dict(num_tokens=-1), 2), (dict(num_q_heads=0), 2), (dict(num_k_heads=1), 2), (dict(weight_type=2), 2),
    (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(head_dim=96), 4), (dict(q_stride=64), 2),
    (dict(q_stride=129), 8), (dict(q_out_stride=132), 8), (dict(q_stride=-128), 2), (dict(num_q_heads=1 << 20), 2),
])
def test_c_abi_refuses(h3, kw, status):
    import ctypes as C

    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    d = _desc(h3, **kw)
    assert h3.load_library().h3_qk_norm_rope(C.byref(d), p, p, None, None, p, None, None, None, None, 0, None,
                                             None, None) == status


def test_c_abi_refuses_pointers(h3):
    import ctypes as C

    lib = h3.load_library()
    buf = (C.c_uint8 * 4096)()
    p = C.c_void_p((C.addressof(buf) + 255) // 256 * 256)
    odd = C.c_void_p(p.value + 2)
    d = _desc(h3)
    fwd = lambda *a: lib.h3_qk_norm_rope(C.byref(d), *a, None)
    none = (None,) * 5
    assert fwd(None, p, None, None, p, None, None, None, None, 0, None, None) == 1
    assert fwd(p, None, None, None, p, None, None, None, None, 0, None, None) == 1
    assert fwd(p, p, None, None, None, None, None, None, None, 0, None, None) == 1
    assert fwd(p, p, None, None, p, None, p, None, None, 0, None, None) == 1  # pos without tag
    assert fwd(odd, p, None, None, p, None, None, None, None, 0, None, None) == 8
    assert fwd(p, odd, None, None, p, None, None, None, None, 0, None, None) == 8
    assert fwd(p, p, None, None, odd, None, None, None, None, 0, None, None) == 8
    assert fwd(p, p, None, None, p, None, p, p, p, 0, None, None) == 2  # cu_requests, no requests
    cfg = h3.RopeConfig(video_dims_t=32, video_dims_h=16, video_dims_w=14)
    assert fwd(p, p, None, None, p, None, p, p, None, 0, None, C.byref(cfg)) == 2
    bwd = lambda *a: lib.h3_qk_norm_rope_bwd(C.byref(d), *a, None)
    args = (p, None, p, None, p, None) + none[:3] + (0, None, None)
    assert bwd(*args, p, None, None, None, p, 1 << 30) == 1  # no weight gradient
    assert bwd(*args, p, None, p, None, None, 0) == 5
    assert bwd(*args, p, None, p, None, p, 64) == 5
    assert lib.h3_qk_norm_rope_bwd_workspace_size(96) == 0


def test_binding_refuses(h3):
    q, w = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.ones(64)
    pos, tag = torch.zeros(4, 3), torch.zeros(4, dtype=torch.uint8)
    with pytest.raises(TypeError):
        h3.qk_norm_rope(q.float(), None, w, None)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q[0], None, w, None)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q.transpose(1, 2), None, w, None)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q[:1].expand(4, 2, 64), None, w, None)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q, None, torch.ones(32), None)
    with pytest.raises(TypeError):
        h3.qk_norm_rope(q, None, w.double(), None)
    with pytest.raises(TypeError):
        h3.qk_norm_rope(q, q, w, w.to(torch.bfloat16))
    with pytest.raises(TypeError):
        h3.qk_norm_rope(q, q, w, None)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q, q[:3], w, w)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q, None, w, None, pos=pos)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q, None, w, None, start_frames=torch.zeros(1))
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q, None, w, None, pos=pos[:3].contiguous(), tag=tag)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q, None, w, None, num_tokens=5)
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q, None, w, None, pos=pos, tag=tag,
                        cu_requests=torch.tensor([0, 2, 4], dtype=torch.int32), start_frames=torch.zeros(1))
    with pytest.raises(ValueError):
        h3.qk_norm_rope(q, None, w, None, q_out=torch.zeros(3, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        h3.qk_norm_rope_bwd(q[:3], None, q, None, w, None)


def test_no_tokens_at_all(h3):
    q, w = torch.zeros(0, 2, 64, dtype=torch.bfloat16), torch.ones(64)
    assert h3.qk_norm_rope(q, None, w, None)[0].shape == q.shape
    dq, dk, dw, dkw = h3.qk_norm_rope_bwd(q, None, q, None, w, None)
    assert dq.shape == q.shape and dk is None and dkw is None and torch.equal(dw, torch.zeros(64))


# ---- GPU -----------------------------------------------------------------------------------------

SHAPES = [  # tokens, q heads, k heads, head_dim, rotate, requests, weights, fused projection
    (1, 1, 1, 64, True, 1, torch.float32, False),
    (1, 40, 8, 128, True, 1, torch.bfloat16, True),
    (3, 2, 2, 64, False, 0, torch.bfloat16, False),
    (5, 3, 1, 128, True, 2, torch.float32, True),
    (45, 2, 2, 64, True, 3, torch.float32, True),
    (17, 5, 0, 128, True, 1, torch.bfloat16, False),
    (129, 24, 8, 64, True, 4, torch.bfloat16, True),
    (701, 7, 3, 128, True, 5, torch.float32, True),
    (2433, 2, 1, 64, True, 2, torch.bfloat16, True),   # groups of four tokens, the last one short
    (2435, 1, 1, 128, False, 0, torch.float32, False),
    (9801, 2, 1, 64, True, 2, torch.bfloat16, False),
]


def _case(shape, seed=0, far=0):
    n, hq, hk, d, rotate, requests, kind, fused = shape
    rng = np.random.default_rng(seed)
    if fused:
        qkv = _bf16(rng, n, (hq + 2 * hk) * d, scale=1.5)
        q, k = qkv[:, :hq * d].view(n, hq, d), qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
    else:
        q, k = _bf16(rng, n, hq, d), _bf16(rng, n, hk, d, scale=3.0)
    qw, kw = (torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).float().to(kind) for _ in range(2))
    where = {}
    if rotate:
        pos, tag = _tokens(n, seed + 1, far)
        cuts = np.unique(np.concatenate([[0, n], rng.integers(0, n + 1, requests - 1)]))
        if len(cuts) < requests + 1:  # some requests hold no token
            cuts = np.sort(np.concatenate([cuts, np.full(requests + 1 - len(cuts), n)]))
        where = dict(pos=pos, tag=tag, cu_requests=cuts.astype(np.int32),
                     start_frames=(rng.integers(0, 4, requests) * 119).astype(np.float32))
    return q, (k if hk else None), qw, (kw if hk else None), where


def _gpu(dev, x):
    if x is None:
        return None
    x = torch.from_numpy(x) if isinstance(x, np.ndarray) else x
    if x.dim() == 3 and not x.is_contiguous():  # keep a fused projection's strides
        base = torch.empty(x.shape[0], x.stride(0) if x.shape[0] > 1 else x[0].numel(), dtype=x.dtype, device=dev)
        view = base[:, :x.shape[1] * x.shape[2]].view(x.shape)
        view.copy_(x)
        return view
    return x.to(dev)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(h3, dev, shape):
    q, k, qw, kw, where = _case(shape)
    on = {n: _gpu(dev, x) for n, x in where.items()}
    yq, yk = h3.qk_norm_rope(_gpu(dev, q), _gpu(dev, k), _gpu(dev, qw), _gpu(dev, kw), **on)
    _check_y(yq, q, qw, where)
    if k is None:
        assert yk is None
    else:
        _check_y(yk, k, kw, where)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(h3, dev, shape):
    q, k, qw, kw, where = _case(shape, seed=3)
    rng = np.random.default_rng(9)
    dyq, dyk = _bf16(rng, *q.shape), None if k is None else _bf16(rng, *k.shape)
    on = {n: _gpu(dev, x) for n, x in where.items()}
    args = [_gpu(dev, x) for x in (dyq, dyk, q, k, qw, kw)]
    got = h3.qk_norm_rope_bwd(*args, **on)
    _check_grad(got[0], got[2], dyq, q, qw, where)
    if k is None:
        assert got[1] is None and got[3] is None
    else:
        _check_grad(got[1], got[3], dyk, k, kw, where)
    again = h3.qk_norm_rope_bwd(*args, **on)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))  # no dependence on timing


@pytest.mark.gpu
def test_far_positions_keep_their_angle(h3, dev):
    shape = (65, 2, 2, 128, True, 2, torch.float32, False)
    q, k, qw, kw, where = _case(shape, seed=5, far=1_000_000)
    where["start_frames"] = np.array([238.0, 100_001.0], dtype=np.float32)
    yq, yk = h3.qk_norm_rope(*(_gpu(dev, x) for x in (q, k, qw, kw)), **{n: _gpu(dev, x) for n, x in where.items()})
    _check_y(yq, q, qw, where)
    _check_y(yk, k, kw, where)


@pytest.mark.gpu
def test_other_frequencies(h3, dev):
    q, k, qw, kw, where = _case((45, 2, 2, 128, True, 2, torch.float32, False), seed=6)
    kw_cfg = dict(base_text=2500.0, base_video=900.0, base_audio=400.0, video_dims_t=24, video_dims_h=64,
                  video_dims_w=40, audio_hz=48.0, video_fps=25.0)
    on = {n: _gpu(dev, x) for n, x in where.items()}
    yq, _ = h3.qk_norm_rope(*(_gpu(dev, x) for x in (q, k, qw, kw)), cfg=h3.RopeConfig(**kw_cfg), **on)
    _check_y(yq, q, qw, dict(where, cfg=oracle.RopeConfig(**kw_cfg)))


@pytest.mark.gpu
def test_one_start_frame_for_all_rows(h3, dev):
    q, k, qw, kw, where = _case((9, 2, 2, 64, True, 1, torch.float32, False), seed=7)
    where["start_frames"] = np.array([357.0], dtype=np.float32)
    on = {n: _gpu(dev, x) for n, x in where.items() if n != "cu_requests"}
    yq, _ = h3.qk_norm_rope(*(_gpu(dev, x) for x in (q, k, qw, kw)), **on)
    _check_y(yq, q, qw, where)


@pytest.mark.gpu
def test_zero_tiny_and_large_rows(h3, dev):
    x = torch.ones(5, 2, 64, dtype=torch.bfloat16)
    x[0], x[1], x[2], x[3] = 0.0, 1e-20, 1e15, -2e-3
    w = torch.linspace(-1, 1, 64)
    for eps in (1e-6, 1e-2):
        y, _ = h3.qk_norm_rope(x.to(dev), None, w.to(dev), None, eps=eps)
        _check_y(y, x, w, {}, eps)
        dy = torch.ones_like(x)
        dx, _, dw, _ = h3.qk_norm_rope_bwd(dy.to(dev), None, x.to(dev), None, w.to(dev), None, eps=eps)
        _check_grad(dx, dw, dy, x, w, {}, eps)


@pytest.mark.gpu
def test_in_place_and_rows_past_the_end(h3, dev):
    shape = (45, 2, 2, 64, True, 3, torch.float32, True)
    q, k, qw, kw, where = _case(shape, seed=8)
    on = {n: _gpu(dev, x) for n, x in where.items()}
    gq, gk, gqw, gkw = (_gpu(dev, x) for x in (q, k, qw, kw))
    yq, yk = h3.qk_norm_rope(gq, gk, gqw, gkw, **on)
    n = 37
    tq, tk = gq.clone(), gk.clone()
    h3.qk_norm_rope(tq, tk, gqw, gkw, num_tokens=n, q_out=tq, k_out=tk, **on)
    for t, y, x in ((tq, yq, gq), (tk, yk, gk)):
        assert torch.equal(t[:n], y[:n]) and torch.equal(t[n:], x[n:])
    # NaN behind the last row does not reach the weights' gradient; dq may be written over dq_out,
    # and into one half of a fused gradient
    dyq = _bf16(np.random.default_rng(1), *q.shape).to(dev)
    dyk = _bf16(np.random.default_rng(2), *k.shape).to(dev)
    ref = h3.qk_norm_rope_bwd(dyq[:n], dyk[:n], gq[:n], gk[:n], gqw, gkw,
                              **dict(on, cu_requests=on["cu_requests"].clamp(max=n)))
    dyq[n:], dyk[n:] = float("nan"), float("nan")
    fused = torch.full((45, 2 * 2 * 64), 5.0, dtype=torch.bfloat16, device=dev)
    dk = fused[:, 128:].view(45, 2, 64)
    got = h3.qk_norm_rope_bwd(dyq, dyk, gq, gk, gqw, gkw, num_tokens=n, dq=dyq, dk=dk, **on)
    assert got[0] is dyq and torch.equal(dyq[:n], ref[0]) and dyq[n:].isnan().all()
    assert torch.equal(dk[:n], ref[1]) and (fused[:, :128] == 5.0).all() and (fused[n:] == 5.0).all()
    assert torch.equal(got[2], ref[2]) and torch.equal(got[3], ref[3])


@pytest.mark.gpu
def test_no_tokens_gives_zero_weight_gradients(h3, dev):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    _, _, dqw, dkw = h3.qk_norm_rope_bwd(q, q, q, q, w, w, num_tokens=0)
    assert torch.equal(dqw, torch.zeros_like(w)) and torch.equal(dkw, torch.zeros_like(w))


@pytest.mark.gpu
def test_nothing_is_taken_from_what_a_launch_left_in_shared_memory(h3, dev):
    n = 5000
    x, w = torch.ones(n, 1, 128, dtype=torch.bfloat16, device=dev), torch.ones(128, device=dev)
    bad = dict(pos=torch.full((n, 3), float("nan"), device=dev), tag=torch.zeros(n, dtype=torch.uint8, device=dev))
    q, k, qw, kw, where = _case((320, 24, 24, 128, True, 1, torch.float32, True), seed=12)
    dyq, dyk = _bf16(np.random.default_rng(1), *q.shape), _bf16(np.random.default_rng(2), *k.shape)
    args = [_gpu(dev, t) for t in (dyq, dyk, q, k, qw, kw)]
    on = {n: _gpu(dev, t) for n, t in where.items()}
    for _ in range(3):
        h3.qk_norm_rope_bwd(x, None, x, None, w, None, **bad)
        dq, dk, dqw, dkw = h3.qk_norm_rope_bwd(*args, **on)
    _check_grad(dq, dqw, dyq, q, qw, where)
    _check_grad(dk, dkw, dyk, k, kw, where)


@pytest.mark.gpu
def test_side_stream_and_graph(h3, dev):
    shape = (129, 4, 2, 64, True, 2, torch.float32, True)
    q, k, qw, kw, where = _case(shape, seed=11)
    args = [_gpu(dev, x) for x in (q, k, qw, kw)]
    on = {n: _gpu(dev, x) for n, x in where.items()}
    dy = [torch.randn_like(args[0]).contiguous(), torch.randn_like(args[1]).contiguous()]
    want = (*h3.qk_norm_rope(*args, **on), *h3.qk_norm_rope_bwd(*dy, *args, **on))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = (*h3.qk_norm_rope(*args, **on), *h3.qk_norm_rope_bwd(*dy, *args, **on))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*h3.qk_norm_rope(*args, **on), *h3.qk_norm_rope_bwd(*dy, *args, **on))
    for _ in range(2):
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
