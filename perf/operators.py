"""Operator benchmark cases: per-head norm of queries and keys with the tagged rotation, and cross
attention to states of another length, each with its gradient.

A case is a dict of plain values.  ``run`` takes a prepared state through one operator: in the
plain form (elementary torch operations in fp32, angles in fp64) when ``own`` is false, through
this package's entry points when it is true.  ``exact`` is the operator's definition in fp64.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0      # frequency ladder of every modality (the library's default)
HZ, FPS = 40.0, 24.0  # continuation shift: t + s * 40 / 24

# ------------------------------------------------------------------------------------------------
# cases


def _norm(name, direction, tokens, heads_q, heads_k, dim, rotate, requests, weights):
    """tokens rows of a fused qkv projection; requests > 0 adds per-request start frames."""
    return {"name": name, "op": "norm", "direction": direction, "tokens": tokens, "heads_q": heads_q,
            "heads_k": heads_k, "dim": dim, "rotate": rotate, "requests": requests, "weights": weights}


def _cross(name, direction, segments, min_q, max_q, min_k, max_k, heads_q, heads_k, dim, padded, empty, layout):
    """segments sequences with query and key lengths drawn from the ranges by the layout number.
    padded: the keys come as [segments, max_k] with valid lengths (an encoder's padded batch);
    otherwise back to back.  empty: one segment has no valid key."""
    return {"name": name, "op": "cross", "direction": direction, "segments": segments, "min_q": min_q,
            "max_q": max_q, "min_k": min_k, "max_k": max_k, "heads_q": heads_q, "heads_k": heads_k,
            "dim": dim, "padded": padded, "empty": empty, "layout": layout}


def listed():
    return [
        # one new token of an autoregressive stream: latency
        _norm("norm_rope_token", "fwd", 1, 40, 8, 128, True, 1, "bf16"),
        # the queries and keys of cross attention: norm without rotation, shared key heads, odd length
        _norm("norm_only_gqa", "fwd", 4097, 24, 8, 64, False, 0, "fp32"),
        # a full packed video request (text + audio + video) of four continued windows
        _norm("norm_rope_request", "fwd", 58758, 40, 40, 128, True, 4, "bf16"),
        # a short training sample: the gradient's latency
        _norm("norm_rope_bwd_short", "bwd", 320, 24, 24, 128, True, 1, "fp32"),
        # a training step's packed batch
        _norm("norm_rope_bwd_batch", "bwd", 29001, 40, 40, 128, True, 3, "bf16"),
        # one token per stream against encoder states, eight query heads to a key head
        _cross("cross_tokens", "fwd", 32, 1, 1, 512, 4096, 64, 8, 128, False, False, 1),
        # the worked example's 45 rows against short, odd key lists, one of them empty
        _cross("cross_short", "fwd", 3, 10, 20, 1, 33, 2, 2, 64, False, True, 2),
        # a full packed request's rows against its text states
        _cross("cross_request_text", "fwd", 1, 58758, 58758, 558, 558, 40, 40, 128, False, False, 3),
        # audio rows of four requests against their video latents: few queries, many keys
        _cross("cross_audio_to_video", "fwd", 4, 200, 320, 12000, 14500, 24, 24, 128, False, False, 4),
        # a short training sample against a padded text batch
        _cross("cross_bwd_short", "bwd", 4, 64, 320, 40, 256, 24, 8, 64, True, True, 5),
        # training: video rows of two requests against padded text states
        _cross("cross_bwd_text", "bwd", 2, 13000, 14690, 300, 512, 24, 24, 128, True, False, 6),
        # training: both sides long (the gradient of packed self attention has this form)
        _cross("cross_bwd_long", "bwd", 1, 4096, 4096, 4096, 4096, 24, 24, 128, False, False, 7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dim = rng.choice([64, 128])
    heads_q, heads_k = rng.choice([(2, 2), (24, 24), (24, 8), (40, 40), (40, 8), (16, 1)])
    direction = rng.choice(["fwd", "bwd"])
    if rng.random() < 0.4:
        most = 58758 if direction == "fwd" else 29001
        tokens = _log_int(rng, 1, most)
        return {k: v for k, v in _norm("", direction, tokens, heads_q, heads_k, dim, rng.random() < 0.7,
                                       rng.randint(1, 4) if tokens > 4 else 1,
                                       rng.choice(["bf16", "fp32"])).items() if k != "name"}
    shape = rng.choice(["tokens", "text", "long"])
    segments = rng.randint(1, 32) if shape == "tokens" else rng.randint(1, 6)
    max_q = rng.randint(1, 3) if shape == "tokens" else _log_int(rng, 8, 14690 if shape == "text" else 4096)
    max_k = _log_int(rng, 8, 558 if shape == "text" else 4096)
    # never more than the largest listed case of the direction: score entries over all heads
    most = 58758 * 558 * 40 if direction == "fwd" else 4096 * 4096 * 24
    while segments * max_q * max_k * heads_q > most:
        if segments > 1:
            segments -= 1
        else:
            max_q = max(1, max_q // 2)
    return {k: v for k, v in _cross("", direction, segments, max(1, max_q // 2), max_q, max(1, max_k // 3), max_k,
                                    heads_q, heads_k, dim, rng.random() < 0.5, segments > 1 and rng.random() < 0.4,
                                    rng.randint(1, 1 << 20)).items() if k != "name"}


def _lengths(case):
    """(query lengths, key lengths) of the segments, fixed by the case alone."""
    rng = random.Random(case["layout"])
    lq = [rng.randint(case["min_q"], case["max_q"]) for _ in range(case["segments"])]
    lk = [rng.randint(case["min_k"], case["max_k"]) for _ in range(case["segments"])]
    if case["empty"]:
        lk[case["segments"] // 2] = 0
    return lq, lk


def work(case):
    hq, hk, d = case["heads_q"], case["heads_k"], case["dim"]
    if case["op"] == "norm":
        rows = case["tokens"] * (hq + hk)
        tokens = 13.0 * case["tokens"] if case["rotate"] else 0.0  # position and tag
        if case["direction"] == "fwd":
            return {"bytes": rows * d * 4.0 + tokens, "flops": rows * d * 7.0}
        return {"bytes": rows * d * 6.0 + tokens + 8.0 * d, "flops": rows * d * 14.0}
    lq, lk = _lengths(case)
    nq, nk, pairs = sum(lq), sum(lk), sum(a * b for a, b in zip(lq, lk))
    q, kv = nq * hq * d * 2.0, nk * hk * d * 2.0
    if case["direction"] == "fwd":
        return {"bytes": 2 * q + 2 * kv + 4.0 * nq * hq, "flops": 4.0 * hq * d * pairs}
    # q, o, do, dq and k, v, dk, dv, the log-sum-exp
    return {"bytes": 4 * q + 4 * kv + 4.0 * nq * hq, "flops": 10.0 * hq * d * pairs}


# ------------------------------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return _prepare_norm(case, gen) if case["op"] == "norm" else _prepare_cross(case, gen)


def _randn(gen, *shape, scale=1.0):
    x = torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32)
    return (x.mul_(scale) if scale != 1.0 else x).to(torch.bfloat16)


def _prepare_norm(case, gen):
    n, hq, hk, d = case["tokens"], case["heads_q"], case["heads_k"], case["dim"]
    # the projection's output: [tokens, q heads | k heads | v heads]; q and k are views of it
    qkv = _randn(gen, n, (hq + 2 * hk) * d, scale=1.5)
    state = {"case": case, "q": qkv[:, :hq * d].view(n, hq, d), "k": qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)}
    kind = torch.bfloat16 if case["weights"] == "bf16" else torch.float32
    for name in ("q_weight", "k_weight"):
        state[name] = (1.0 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(kind)
    if case["rotate"]:
        # text rows, audio rows (40 a second), then video rows of 40 x 50 frames
        text, audio = min(558, (n + 2) // 3), min(200, n // 3)
        i = torch.arange(n, device="cuda")
        v = (i - text - audio).clamp(min=0)
        video = i >= text + audio
        t = torch.where(video, v // 2000, torch.where(i < text, i, i - text))
        pos = torch.stack([t, torch.where(video, v % 2000 // 50, 0), torch.where(video, v % 50, 0)], dim=1)
        state["pos"] = pos.to(torch.float32).contiguous()
        state["tag"] = torch.where(video, 1, torch.where(i < text, 0, 2)).to(torch.uint8)
        r = case["requests"]
        cuts = [n * k // r for k in range(r + 1)]
        state["cu_requests"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        state["start_frames"] = (torch.randint(0, 4, (r,), device="cuda", generator=gen) * 119).to(torch.float32)
    if case["direction"] == "bwd":
        state["dq_out"], state["dk_out"] = _randn(gen, n, hq, d), _randn(gen, n, hk, d)
    return state


def _prepare_cross(case, gen):
    hq, hk, d = case["heads_q"], case["heads_k"], case["dim"]
    lq, lk = _lengths(case)
    nq = sum(lq)
    starts_k = [case["max_k"]] * len(lk) if case["padded"] else lk
    nk = sum(starts_k)
    kv = _randn(gen, nk, 2 * hk * d)  # the encoder's fused key/value projection
    state = {"case": case, "q": _randn(gen, nq, hq, d), "k": kv[:, :hk * d].view(nk, hk, d),
             "v": kv[:, hk * d:].view(nk, hk, d), "max_q": max(lq), "max_k": max(lk),
             "cu_q": _offsets(lq), "cu_k": _offsets(starts_k),
             "seqused_k": torch.tensor(lk, dtype=torch.int32, device="cuda") if case["padded"] else None}
    if case["direction"] == "bwd":
        state["out"], state["lse"] = _plain_cross_fwd(state)
        state["dout"] = _randn(gen, nq, hq, d)
    return state


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------
# one pass


def run(state):
    case = state["case"]
    if own:
        return _own_norm(state) if case["op"] == "norm" else _own_cross(state)
    if case["op"] == "norm":
        return _plain_norm_fwd(state) if case["direction"] == "fwd" else _plain_norm_bwd(state)
    return _plain_cross_fwd(state) if case["direction"] == "fwd" else _plain_cross_bwd(state)


def _own_norm(state):
    import packed_varlen_attention_modality_gb300 as h3

    where = dict(pos=state.get("pos"), tag=state.get("tag"), cu_requests=state.get("cu_requests"),
                 start_frames=state.get("start_frames"), eps=EPS)
    if state["case"]["direction"] == "fwd":
        return h3.qk_norm_rope(state["q"], state["k"], state["q_weight"], state["k_weight"], **where)
    return h3.qk_norm_rope_bwd(state["dq_out"], state["dk_out"], state["q"], state["k"], state["q_weight"],
                               state["k_weight"], **where)


def _own_cross(state):
    import packed_varlen_attention_modality_gb300 as h3

    lengths = dict(cu_seqlens_q=state["cu_q"], cu_seqlens_k=state["cu_k"], max_seqlen_q=state["max_q"],
                   max_seqlen_k=state["max_k"], seqused_k=state["seqused_k"])
    if state["case"]["direction"] == "fwd":
        return h3.varlen_cross_attn_fwd(state["q"], state["k"], state["v"], return_lse=True, **lengths)
    return h3.varlen_cross_attn_bwd(state["dout"], state["q"], state["k"], state["v"], state["out"], state["lse"],
                                    **lengths)


# ------------------------------------------------------------------------------------------------
# plain form: norm and rotation


def _angles(state):
    """(cos, sin) fp32 [tokens, dim / 2] of the rotation; angles in fp64."""
    d = state["case"]["dim"]
    pos, tag = state["pos"].double(), state["tag"]
    row = torch.arange(pos.shape[0], device="cuda", dtype=torch.int32)
    request = torch.searchsorted(state["cu_requests"][1:], row, right=True).clamp(max=state["start_frames"].numel() - 1)
    t = pos[:, 0] + state["start_frames"].double()[request] * HZ / FPS
    j = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    line = BASE ** (-2.0 * j / d)                       # text and audio: one band by t
    band_t = BASE ** (-2.0 * j[:d // 4] / (d // 2))     # video: half the dims by t, a quarter by h, by w
    band_hw = BASE ** (-2.0 * j[:d // 8] / (d // 4))
    flat = t[:, None] * line
    video = torch.cat([t[:, None] * band_t, pos[:, 1:2] * band_hw, pos[:, 2:3] * band_hw], dim=1)
    phi = torch.where((tag == 1)[:, None], video, flat)
    return phi.cos().float(), phi.sin().float()


def _rotate(x, cos, sin):
    a, b = x[..., 0::2], x[..., 1::2]
    c, s = cos[:, None, :], sin[:, None, :]
    return torch.stack([a * c - b * s, a * s + b * c], dim=-1).reshape(x.shape)


def _plain_norm_one(x, w, cs):
    x = x.float()
    z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    return (z if cs is None else _rotate(z, *cs)).to(torch.bfloat16)


def _plain_norm_fwd(state):
    cs = _angles(state) if state["case"]["rotate"] else None
    return _plain_norm_one(state["q"], state["q_weight"], cs), _plain_norm_one(state["k"], state["k_weight"], cs)


def _plain_norm_grad(dy, x, w, cs):
    x, dy = x.float(), dy.float()
    dz = dy if cs is None else _rotate(dy, cs[0], -cs[1])
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    g = dz * w.float()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dz * xh).sum((0, 1), dtype=torch.float64).float()


def _plain_norm_bwd(state):
    cs = _angles(state) if state["case"]["rotate"] else None
    dq, dqw = _plain_norm_grad(state["dq_out"], state["q"], state["q_weight"], cs)
    dk, dkw = _plain_norm_grad(state["dk_out"], state["k"], state["k_weight"], cs)
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------------------------------------
# plain form: cross attention, on padded batches


def _pad(x, cu, most):
    """Packed rows [n, heads, dim] -> [segments, heads, most, dim] fp32 (rows past the end: some row)."""
    at = (cu[:-1, None].long() + torch.arange(most, device="cuda")).clamp(max=x.shape[0] - 1)
    return x[at].float().transpose(1, 2)


def _unpad(x, cu, rows):
    """[segments, heads, most, ...] -> packed rows [rows, heads, ...]."""
    i = torch.arange(rows, device="cuda", dtype=torch.int32)
    g = torch.searchsorted(cu[1:], i, right=True).clamp(max=cu.numel() - 2)
    return x[g, :, (i - cu[g]).long()]


def _padded_scores(state):
    """q, k, v padded with the query heads of one key head side by side, scores, and the valid keys."""
    hq, hk, d = state["case"]["heads_q"], state["case"]["heads_k"], state["case"]["dim"]
    q = _pad(state["q"], state["cu_q"], state["max_q"])
    q = q.reshape(q.shape[0], hk, hq // hk * state["max_q"], d)
    k, v = _pad(state["k"], state["cu_k"], state["max_k"]), _pad(state["v"], state["cu_k"], state["max_k"])
    used = state["seqused_k"] if state["seqused_k"] is not None else state["cu_k"].diff()
    valid = (torch.arange(state["max_k"], device="cuda") < used[:, None])[:, None, None, :]
    s = torch.matmul(q, k.transpose(2, 3)) * (d ** -0.5)
    return q, k, v, s, valid


def _plain_cross_fwd(state):
    hq, d, most = state["case"]["heads_q"], state["case"]["dim"], state["max_q"]
    q, k, v, s, valid = _padded_scores(state)
    s = torch.where(valid, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)  # -inf for a segment without keys
    rows = state["q"].shape[0]
    b = q.shape[0]
    out = _unpad(o.reshape(b, hq, most, d), state["cu_q"], rows).to(torch.bfloat16)
    return out, _unpad(lse.reshape(b, hq, most), state["cu_q"], rows).t().contiguous()


def _plain_cross_bwd(state):
    hq, d, most = state["case"]["heads_q"], state["case"]["dim"], state["max_q"]
    q, k, v, s, valid = _padded_scores(state)
    b, nq, nk = q.shape[0], state["q"].shape[0], state["k"].shape[0]
    o = _pad(state["out"], state["cu_q"], most).reshape(q.shape)
    real = (torch.arange(most, device="cuda") < state["cu_q"].diff()[:, None])[:, None, None, :, None]
    real = real.expand(b, state["case"]["heads_k"], hq // state["case"]["heads_k"], most, 1).reshape(*q.shape[:3], 1)
    do = _pad(state["dout"], state["cu_q"], most).reshape(q.shape) * real.float()
    lse = _pad(state["lse"].t()[..., None], state["cu_q"], most).reshape(*q.shape[:3], 1)
    p = torch.where(valid & real, torch.exp(s - lse), 0.0)  # padded rows send no gradient
    ds = p * (torch.matmul(do, v.transpose(2, 3)) - (do * o).sum(-1, keepdim=True)) * (d ** -0.5)
    dq = torch.matmul(ds, k).reshape(b, hq, most, d)
    dk, dv = torch.matmul(ds.transpose(2, 3), q), torch.matmul(p.transpose(2, 3), do)
    return (_unpad(dq, state["cu_q"], nq).to(torch.bfloat16),
            _unpad_keys(dk, state, nk), _unpad_keys(dv, state, nk))


def _unpad_keys(x, state, rows):
    """As _unpad, with zero for the rows of a segment past its valid keys."""
    cu, most = state["cu_k"], state["max_k"]
    i = torch.arange(rows, device="cuda", dtype=torch.int32)
    g = torch.searchsorted(cu[1:], i, right=True).clamp(max=cu.numel() - 2)
    at = (i - cu[g]).long()
    y = x[g, :, at.clamp(max=most - 1)]
    return torch.where((at < most)[:, None, None], y, 0.0).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------
# the definition in fp64


def exact(case, seed):
    state = prepare(case, seed)
    return _exact_norm(case, state) if case["op"] == "norm" else _exact_cross(case, state)


def _exact_norm(case, state):
    d = case["dim"]
    turn = None
    if case["rotate"]:
        pos = state["pos"].double().cpu()
        tag = state["tag"].cpu()
        t = pos[:, 0].clone()
        cuts = state["cu_requests"].tolist()
        for r, s in enumerate(state["start_frames"].tolist()):
            t[cuts[r]:cuts[r + 1]] += s * 40.0 / 24.0
        phi = torch.empty(pos.shape[0], d // 2, dtype=torch.float64)
        for j in range(d // 2):
            if j < d // 4:
                video = t * 10000.0 ** (-4.0 * j / d)
            else:
                axis = 1 if j < d // 4 + d // 8 else 2
                video = pos[:, axis] * 10000.0 ** (-8.0 * (j - d // 4 - (axis - 1) * (d // 8)) / d)
            phi[:, j] = torch.where(tag == 1, video, t * 10000.0 ** (-2.0 * j / d))
        turn = torch.polar(torch.ones_like(phi), phi).cuda()[:, None, :]
    results, sums = [], []
    for x, w, dy in ((state["q"], state["q_weight"], state.get("dq_out")),
                     (state["k"], state["k_weight"], state.get("dk_out"))):
        x, w = x.double(), w.double()
        length = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        unit = x / length
        if case["direction"] == "fwd":
            z = unit * w
            if turn is not None:
                z = torch.view_as_real(torch.view_as_complex(z.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
            results.append(z)
            continue
        dz = dy.double()
        if turn is not None:
            dz = torch.view_as_real(torch.view_as_complex(dz.unflatten(-1, (-1, 2)).contiguous()) * turn.conj()).flatten(-2)
        sums.append((dz * unit).sum(1).sum(0))
        dz *= w
        results.append((dz - unit * ((dz * unit).sum(-1, keepdim=True) / d)) / length)
        del dz
    return tuple(results + sums)


def _exact_cross(case, state):
    lq, lk = _lengths(case)
    hq, hk, d = case["heads_q"], case["heads_k"], case["dim"]
    backward = case["direction"] == "bwd"
    q, k, v = state["q"], state["k"], state["v"]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(o), *(torch.zeros(k.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    a = b = 0
    for g in range(len(lq)):
        if lk[g]:
            rows, keys = slice(a, a + lq[g]), slice(b, b + lk[g])
            for h in range(hq):
                qh, kh, vh = q[rows, h].double(), k[keys, h * hk // hq].double(), v[keys, h * hk // hq].double()
                s = qh @ kh.T / math.sqrt(d)
                whole = torch.logsumexp(s, dim=1)
                p = (s - whole[:, None]).exp()
                lse[h, rows] = whole
                o[rows, h] = p @ vh
                if backward:
                    grad = state["dout"][rows, h].double()
                    dv[keys, h * hk // hq] += p.T @ grad
                    dp = grad @ vh.T
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[rows, h] = ds @ kh
                    dk[keys, h * hk // hq] += ds.T @ qh
        a += lq[g]
        b += case["max_k"] if case["padded"] else lk[g]
    return (dq, dk, dv) if backward else (o, lse)
