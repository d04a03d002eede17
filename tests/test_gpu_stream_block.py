"""A block's calls in the order in which a running stream makes them (join the branch and norm, norm and rotate
queries and keys, write the cache, attend over it, join again) and, for training, the gradients back through
the same block.  The projections between them are plain products.

Tolerances: against fp64 from the raw inputs, in the relative 2-norm.  Each rounding to bf16 is off by 2^-8 of its
value at most, and the score, at the size that normed rows give it, passes its error on at most twofold.  Forward
about seven follow one another (h, the projection, q and k, P, o, its projection, the second step's results):
7 * 2 * 2^-8 = 0.055.  Back there are about twice as many: 0.11.  An e4m3 cache is off by 2^-4 of its values on top
(of the row's scaled ones, 2^-10 of its unit for the smallest), and attention is then compared over the rows that
the cache holds, read back.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle.norm import _f64

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
DIM, H, HK, D, PAGE = 256, 4, 2, 64, 16


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


def _weights(rng, stream_type):
    f32 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    w = {"qkv": f32(DIM, (H + 2 * HK) * D) / 16, "o": f32(H * D, DIM) / 16, "norm": 1 + 0.2 * f32(DIM),
         "branch": 1 + 0.2 * f32(DIM), "q": 1 + 0.2 * f32(D), "k": 1 + 0.2 * f32(D)}
    w["qkv"], w["o"] = w["qkv"].to(torch.bfloat16), w["o"].to(torch.bfloat16)
    w["type"] = stream_type
    return w


def _rows(rng, n, requests, stream_type):
    f32 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    return dict(x=f32(n, DIM).to(stream_type), y=f32(n, DIM).to(torch.bfloat16), mod=0.3 * f32(requests, 6, DIM))


def _steps(w, mod, cu):
    """Arguments of the two joins: what follows a branch and goes into the next."""
    first = dict(norm="layer", scale=mod[:, 1], shift=mod[:, 0], gate=mod[:, 5], cu_requests=cu)
    second = dict(norm="rms", weight=w["norm"], scale=mod[:, 4], shift=mod[:, 3], gate=mod[:, 2], branch_norm="rms",
                  branch_weight=w["branch"], cu_requests=cu)
    return first, second


def _heads(t):
    return tuple(c.reshape(len(t), -1, D) for c in (t[:, :H * D], t[:, H * D:(H + HK) * D], t[:, (H + HK) * D:]))


def _off(got, ref):
    got = _f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


class Stream:
    """The cache of some sequences and the block's calls for their new tokens."""

    def __init__(self, h3, dev, w, streams, room, e4m3, rng):
        self.h3, self.w = h3, {n: t.to(dev) if torch.is_tensor(t) else t for n, t in w.items()}
        pages = -(-room // PAGE)
        self.table = torch.from_numpy(rng.permutation(streams * pages).astype(np.int32).reshape(streams, pages)).to(dev)
        self.cache = [torch.zeros(streams * pages, HK, PAGE, D, device=dev).to(
            torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in range(2)]
        self.scales = {n: torch.zeros(streams * pages, HK, PAGE, dtype=torch.uint8, device=dev)
                       for n in ("k_scale", "v_scale")} if e4m3 else {}
        self.room = room

    def __call__(self, x, y, mod, pos, cu, start, used, most):
        h3, w = self.h3, self.w
        first, second = _steps(w, mod, cu)
        x1, h = h3.residual_norm(x, y, **first)
        q, k, v = (t.view(len(x), -1, D) for t in (h @ w["qkv"]).split([H * D, HK * D, HK * D], 1))
        tag, frames = torch.zeros(len(x), dtype=torch.uint8, device=x.device), torch.zeros(len(cu) - 1, device=x.device)
        rot = dict(tag=tag, cu_requests=cu, start_frames=frames)
        q, k = h3.qk_norm_rope(q, k, w["q"], w["k"], pos=pos, **rot)
        h3.kv_cache_write(k, v, *self.cache, self.table, cu, start, **self.scales)
        o = h3.paged_attn_fwd(q, *self.cache, self.table, cu, used, most, self.room, causal_block=1, **self.scales)
        x2, h2 = h3.residual_norm(x1, o.view(len(x), -1) @ w["o"], **second)
        return dict(x1=x1, h=h, x2=x2, h2=h2)

    def read(self, lengths):
        dev = self.table.device
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=dev)
        zero = torch.zeros(len(lengths), dtype=torch.int32, device=dev)
        return [_f64(t) for t in self.h3.kv_cache_read(*self.cache, self.table, cu, zero, num_rows=int(sum(lengths)),
                                                       **self.scales)]


@pytest.mark.parametrize("stream_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_chunk_then_tokens_then_chunks(h3, dev, stream_type, e4m3):
    rng = np.random.default_rng(7)
    w = _weights(rng, stream_type)
    rounds = [[40, 17, 130], [1, 1, 1], [1, 0, 1], [60, 3, 20], [1, 1, 0]]
    lengths = np.zeros(3, dtype=np.int64)
    net = Stream(h3, dev, w, 3, 300, e4m3, rng)
    f = {n: _f64(t) for n, t in w.items() if torch.is_tensor(t)}
    keys, values = [np.zeros((0, HK, D))] * 3, [np.zeros((0, HK, D))] * 3
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32)
    for new in rounds:
        n = sum(new)
        cu = np.concatenate([[0], np.cumsum(new)])
        rows = _rows(rng, n, 3, stream_type)
        pos = torch.from_numpy(np.concatenate([np.stack([np.arange(a, a + c)] * 3, 1) for a, c in zip(lengths, new)])
                               .astype(np.float32))
        used = lengths + new
        got = net(*(t.to(dev) for t in (rows["x"], rows["y"], rows["mod"], pos, i32(cu), i32(lengths), i32(used))),
                  max(new))
        assert h3.get_device_error(dev) == 0
        # fp64, from the raw rows
        first, second = _steps(f, _f64(rows["mod"]), cu)
        x1, h = oracle.residual_norm(rows["x"], rows["y"], **first)
        q, k, v = _heads(h @ f["qkv"])
        rot = dict(pos=pos.numpy(), tag=np.zeros(n, np.uint8), cu_requests=cu, start_frames=np.zeros(3))
        q, k = oracle.norm_rope(q, f["q"], **rot), oracle.norm_rope(k, f["k"], **rot)
        for g in range(3):
            keys[g] = np.concatenate([keys[g], k[cu[g]:cu[g + 1]]])
            values[g] = np.concatenate([values[g], v[cu[g]:cu[g + 1]]])
        held = net.read(used)
        for name, t, ref in zip("kv", held, (keys, values)):
            ref = np.concatenate(ref)
            assert _off(t, ref) <= 7 * HALF + (2.0 ** -4 if e4m3 else 0.0), name
        cut = np.cumsum(used)[:-1]
        held = [np.split(t, cut) for t in held] if e4m3 else (keys, values)
        o, _ = oracle.paged_attention(q, *held, cu, used, block=1)
        x2, h2 = oracle.residual_norm(x1, o.reshape(n, -1) @ f["o"], **second)
        for name, ref in dict(x1=x1, h=h, x2=x2, h2=h2).items():
            off = _off(got[name], ref)
            assert off <= 14 * HALF, (new, name, off)
        lengths = used


def test_tokens_from_a_graph(h3, dev):
    """Single tokens of one captured step: positions, lengths and the rows themselves move on the device."""
    rng = np.random.default_rng(11)
    w = _weights(rng, torch.float32)
    nets = [Stream(h3, dev, w, 3, 300, True, np.random.default_rng(3)) for _ in range(2)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    cu, one = i32(0, 40, 57, 187), i32(0, 1, 2, 3)
    begin = [t.to(dev) for t in _rows(rng, 187, 3, torch.float32).values()]
    pos = torch.cat([torch.arange(c, device=dev) for c in (40, 17, 130)]).float()[:, None].repeat(1, 3)
    for net in nets:
        net(*begin, pos, cu, i32(0, 0, 0), i32(40, 17, 130), 130)
    tokens = [[t.to(dev) for t in _rows(rng, 3, 3, torch.float32).values()] for _ in range(6)]
    start = i32(40, 17, 130)
    want = [nets[0](*rows, (start + i).float()[:, None].repeat(1, 3), one, start + i, start + i + 1, 1)
            for i, rows in enumerate(tokens)]
    # the captured step: rows come into its buffers, and it ends by moving each stream on by a token
    held, at = [t.clone() for t in tokens[0]], start.clone()
    step = lambda: nets[1](*held, at.float()[:, None].repeat(1, 3), one, at, at + 1, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a first pass outside the capture, as a library's own set-up wants one
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
        at.add_(1)
    for rows, ref in zip(tokens, want):
        for t, r in zip(held, rows):
            t.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], ref[n]) for n in ref)
    assert h3.get_device_error(dev) == 0
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(nets[0].cache, nets[1].cache))


def _train(h3, w, x, y, mod, cu, dx2, dh2):
    n = len(x)
    first, second = _steps(w, mod, cu)
    x1, h = h3.residual_norm(x, y, **first)
    raw = tuple(t.view(n, -1, D) for t in (h @ w["qkv"]).split([H * D, HK * D, HK * D], 1))
    q, k = h3.qk_norm_rope(raw[0], raw[1], w["q"], w["k"])
    v = raw[2].contiguous()
    o, lse = h3.varlen_cross_attn_fwd(q, k, v, cu, cu, n, n, return_lse=True)
    a = o.view(n, -1) @ w["o"]
    x2, h2 = h3.residual_norm(x1, a, **second)
    back = h3.residual_norm_bwd(dx2, dh2, x2, a, **second)
    do = (back.dy @ w["o"].t()).view(n, H, D)
    dq, dk, dv = h3.varlen_cross_attn_bwd(do, q, k, v, o, lse, cu, cu, n, n)
    dq, dk, dwq, dwk = h3.qk_norm_rope_bwd(dq, dk, raw[0], raw[1], w["q"], w["k"])
    dqkv = torch.cat([t.reshape(n, -1) for t in (dq, dk, dv)], 1)
    front = h3.residual_norm_bwd(back.dx, dqkv @ w["qkv"].t(), x1, y, **first)
    return dict(x2=x2, h2=h2, dx=front.dx, dy=front.dy, dscale=front.scale, dshift=front.shift, dgate=front.gate,
                dscale2=back.scale, dshift2=back.shift, dgate2=back.gate, dw=back.weight, dwb=back.branch_weight,
                dwq=dwq, dwk=dwk)


@pytest.mark.parametrize("stream_type", [torch.float32, torch.bfloat16])
def test_training_through_a_block(h3, dev, stream_type):
    rng = np.random.default_rng(19)
    w = _weights(rng, stream_type)
    cu = np.array([0, 40, 57, 257])
    rows = _rows(rng, 257, 3, stream_type)
    d = _rows(rng, 257, 3, stream_type)  # gradients of the stream and of h
    on = {n: t.to(dev) if torch.is_tensor(t) else t for n, t in w.items()}
    got = _train(h3, on, rows["x"].to(dev), rows["y"].to(dev), rows["mod"].to(dev),
                 torch.tensor(cu, dtype=torch.int32, device=dev), d["x"].to(dev), d["y"].to(dev))
    assert h3.get_device_error(dev) == 0
    f = {n: _f64(t) for n, t in w.items() if torch.is_tensor(t)}
    first, second = _steps(f, _f64(rows["mod"]), cu)
    x1, h = oracle.residual_norm(rows["x"], rows["y"], **first)
    rq, rk, v = _heads(h @ f["qkv"])
    q, k = oracle.norm_rope(rq, f["q"]), oracle.norm_rope(rk, f["k"])
    o, _ = oracle.cross_attention(q, k, v, cu, cu)
    a = o.reshape(257, -1) @ f["o"]
    x2, h2 = oracle.residual_norm(x1, a, **second)
    back = oracle.residual_norm_grad(d["x"], d["y"], x2, a, **second)
    dq, dk, dv = oracle.cross_attention_grad((back["dy"] @ f["o"].T).reshape(257, H, D), q, k, v, cu, cu)
    dq, dwq = oracle.norm_rope_grad(dq, rq, f["q"])
    dk, dwk = oracle.norm_rope_grad(dk, rk, f["k"])
    dqkv = np.concatenate([t.reshape(257, -1) for t in (dq, dk, dv)], 1)
    front = oracle.residual_norm_grad(back["dx"], dqkv @ f["qkv"].T, x1, rows["y"], **first)
    ref = dict(x2=x2, h2=h2, dx=front["dx"], dy=front["dy"], dscale=front["scale"], dshift=front["shift"],
               dgate=front["gate"], dscale2=back["scale"], dshift2=back["shift"], dgate2=back["gate"],
               dw=back["weight"], dwb=back["branch_weight"], dwq=dwq, dwk=dwk)
    for name, r in ref.items():
        off = _off(got[name], r)
        assert off <= (14 if name in ("x2", "h2") else 28) * HALF, (name, off)


def _thread_calls(h3, dev):
    g = torch.Generator(device=dev).manual_seed(5)
    bf = lambda *s: torch.randn(*s, device=dev, generator=g).to(torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    x, y, w = bf(300, 512), bf(300, 512), torch.rand(512, device=dev, generator=g) + 0.5
    cache, table = [bf(40, 2, 16, 64) for _ in range(2)], torch.arange(40, dtype=torch.int32, device=dev).view(2, 20)
    q, cu, used = bf(300, 4, 64), i32(0, 200, 300), i32(300, 290)
    one = i32(0, 1, 2)

    def write():
        place = [torch.zeros_like(t) for t in cache]
        h3.kv_cache_write(q[:, :2], q[:, 2:], *place, table, cu, i32(90, 0))
        return place

    torch.cuda.synchronize()
    return {"norm": lambda: h3.residual_norm(x, y, weight=w, branch_norm="layer"),
            "norm_bwd": lambda: h3.residual_norm_bwd(x, y, x, y, weight=w, branch_norm="layer", branch_weight=w)[:4],
            "write": write, "read": lambda: h3.kv_cache_read(*cache, table, cu, i32(90, 0), num_rows=300),
            "tokens": lambda: (h3.paged_attn_fwd(q[:2], *cache, table, one, used, 1, 320),),
            "chunk": lambda: (h3.paged_attn_fwd(q, *cache, table, cu, used, 200, 320, causal_block=1),)}


@pytest.mark.parametrize("name", ["norm", "norm_bwd", "write", "read", "tokens", "chunk"])
def test_first_call_of_a_new_thread(h3, dev, name):
    import threading

    call = _thread_calls(h3, dev)[name]
    expected = call()
    torch.cuda.synchronize()
    out = []

    def run():
        try:
            with torch.cuda.stream(torch.cuda.Stream(dev)):
                out.append(call())
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            out.append(e)

    threads = [threading.Thread(target=run) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(out) == 3
    for r in out:
        assert not isinstance(r, Exception), r
        assert all(torch.equal(a, b) for a, b in zip(r, expected))
