"""Operator benchmark cases: the step between two branches of a block (gated residual and modulated
norm, with its gradient), a paged key/value cache that is quantised as it is written and read back,
and attention of new tokens over that cache.

A case is a dict of plain values.  ``run`` takes a prepared state through one operator: in the
plain form (elementary torch operations in fp32, long sums in fp64) when ``own`` is false, through
this package's entry points when it is true.  ``exact`` is the operator's definition in fp64.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MOST = 448.0           # largest e4m3 value
SCALE_MIN, SCALE_MAX = -110, 120  # exponents of a cache row's scale

# ------------------------------------------------------------------------------------------------
# cases


def _norm(name, direction, tokens, dim, requests, norm, branch_norm, weights, modulated, stream, residual_scale):
    """tokens rows of the stream.  norm / branch_norm: "rms", "layer" or "none"; modulated: shift, scale
    and gate per request, parts of one projection; weights: of the two norms; stream: its type."""
    return {"name": name, "op": "norm", "direction": direction, "tokens": tokens, "dim": dim, "requests": requests,
            "norm": norm, "branch_norm": branch_norm, "weights": weights, "modulated": modulated, "stream": stream,
            "residual_scale": residual_scale}


def _cache(name, segments, min_rows, max_rows, max_start, heads, dim, page, kind, layout):
    """segments sequences that append rows (drawn from the range by the layout number) behind up to
    max_start cached ones, and read them back.  kind: the cache's type."""
    return {"name": name, "op": "cache", "segments": segments, "min_rows": min_rows, "max_rows": max_rows,
            "max_start": max_start, "heads": heads, "dim": dim, "page": page, "kind": kind, "layout": layout}


def _attn(name, segments, min_q, max_q, min_k, max_k, heads_q, heads_k, dim, page, kind, block, layout):
    """segments sequences of which min_k to max_k tokens are cached, the last min_q to max_q of them new.
    block: tokens of a causal block (0: every new token sees every key)."""
    return {"name": name, "op": "attn", "segments": segments, "min_q": min_q, "max_q": max_q, "min_k": min_k,
            "max_k": max_k, "heads_q": heads_q, "heads_k": heads_k, "dim": dim, "page": page, "kind": kind,
            "block": block, "layout": layout}


def listed():
    return [
        # one new token of each of four running streams: latency
        _norm("norm_tokens", "fwd", 4, 5120, 4, "layer", "none", False, True, "bf16", 1.0),
        # a full packed video request (text + audio + video) of four windows, modulated as a DiT block is
        _norm("norm_request", "fwd", 58758, 5120, 4, "layer", "none", False, True, "bf16", 1.0),
        # a short training sample: norms on both sides of the branch, residuals in fp32, odd size
        _norm("norm_bwd_short", "bwd", 317, 2560, 1, "rms", "rms", True, False, "fp32", 1.0),
        # a training step's packed batch: everything at once
        _norm("norm_bwd_batch", "bwd", 29001, 5120, 3, "rms", "rms", True, True, "bf16", 0.75),
        # 32 streams append a token each: latency
        _cache("cache_tokens", 32, 1, 1, 4096, 8, 128, 16, "e4m3", 1),
        # a denoised window of each of three requests enters the cache, and is read back
        _cache("cache_window", 3, 12001, 14690, 14690, 40, 128, 64, "e4m3", 2),
        # one token per stream, eight query heads to a key head
        _attn("paged_tokens", 32, 1, 1, 512, 4096, 64, 8, 128, 16, "bf16", 1, 3),
        # two long streams, quantised: the keys of a token are split over the GPU
        _attn("paged_tokens_long", 2, 1, 1, 90000, 100000, 40, 8, 128, 64, "e4m3", 1, 4),
        # a few new tokens per stream (an audio row's worth of a latent frame), odd lengths
        _attn("paged_few", 5, 3, 27, 2000, 9000, 40, 8, 128, 32, "bf16", 1, 5),
        # a new latent frame of 40 x 50 tokens against a request's cached rows
        _attn("paged_frame", 1, 2000, 2000, 58758, 58758, 24, 24, 128, 64, "bf16", 2000, 6),
        # chunks of two requests, causal by frames of 500 tokens, over a quantised cache
        _attn("paged_chunk", 2, 1000, 1500, 14000, 24000, 40, 40, 128, 128, "e4m3", 500, 7),
        # first chunks: nothing is cached before them, causal by token, shared key heads
        _attn("paged_first", 3, 900, 4096, 0, 0, 24, 8, 64, 64, "bf16", 1, 8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def draw(rng):
    op = rng.choice(["norm", "cache", "attn", "attn"])
    layout = rng.randint(1, 1 << 20)
    if op == "norm":
        direction = rng.choice(["fwd", "bwd"])
        tokens = _log_int(rng, 1, 58758 if direction == "fwd" else 29001)
        branch = rng.choice(["none", "rms", "layer"])
        return _unnamed(_norm("", direction, tokens, rng.choice([512, 1000, 1536, 2560, 4096, 5120]),
                              rng.randint(1, 6), rng.choice(["rms", "layer"]), branch, rng.random() < 0.5,
                              rng.random() < 0.7, rng.choice(["bf16", "bf16", "fp32"]), rng.choice([1.0, 0.75])))
    dim, page, kind = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "e4m3"])
    if op == "cache":
        rows = _log_int(rng, 1, 14690)
        segments = rng.randint(1, 32) if rows < 64 else rng.randint(1, 3)
        return _unnamed(_cache("", segments, max(1, rows // 2), rows, _log_int(rng, 1, 14690), rng.choice([2, 8, 24, 40]),
                               dim, page, kind, layout))
    heads_q, heads_k = rng.choice([(2, 2), (24, 24), (24, 8), (40, 40), (40, 8), (64, 8), (16, 1)])
    shape = rng.choice(["tokens", "few", "chunk"])
    segments = rng.randint(1, 32) if shape == "tokens" else rng.randint(1, 6)
    max_q = {"tokens": rng.randint(1, 3), "few": _log_int(rng, 4, 64), "chunk": _log_int(rng, 64, 2048)}[shape]
    max_k = _log_int(rng, 64, 100000 if shape == "tokens" else 30000)
    block = rng.choice([0, 1, 1, 50, 500])
    # never more than the largest listed cases: score entries over all heads, cached rows over key heads
    while segments * max_q * max_k * heads_q > 58758 * 2000 * 24 or segments * max_k * heads_k > 58758 * 24:
        if segments > 1:
            segments -= 1
        elif max_q > max_k // 8 and max_q > 1:
            max_q //= 2
        else:
            max_k //= 2
    return _unnamed(_attn("", segments, max(1, max_q // 2), max_q, max_k // 3, max_k, heads_q, heads_k, dim, page, kind,
                          block, layout))


def _attn_lengths(case):
    """(new tokens, all tokens) of the segments, fixed by the case alone."""
    rng = random.Random(case["layout"])
    lq = [rng.randint(case["min_q"], case["max_q"]) for _ in range(case["segments"])]
    return lq, [max(q, rng.randint(case["min_k"], case["max_k"])) for q in lq]


def _cache_lengths(case):
    """(rows appended, rows cached before) of the segments."""
    rng = random.Random(case["layout"])
    rows = [rng.randint(case["min_rows"], case["max_rows"]) for _ in range(case["segments"])]
    return rows, [rng.randint(0, case["max_start"]) for _ in range(case["segments"])]


def _limit(p, used, block):
    """Keys that the token at position p sees."""
    return used if block == 0 else min(used, (p // block + 1) * block)


def work(case):
    if case["op"] == "norm":
        n, d, r = case["tokens"], case["dim"], case["requests"]
        stream = 4.0 if case["stream"] == "fp32" else 2.0
        mod = (6.0 * r * d if case["modulated"] else 0.0) + (8.0 * d if case["weights"] else 0.0)
        if case["direction"] == "fwd":
            return {"bytes": n * d * (2 * stream + 4.0) + mod, "flops": n * d * 12.0}
        return {"bytes": n * d * (3 * stream + 6.0) + 3 * mod, "flops": n * d * 24.0}
    row = case["dim"] * 2.0 if case["kind"] == "bf16" else case["dim"] + 1.0
    if case["op"] == "cache":
        rows = sum(_cache_lengths(case)[0]) * case["heads"] * 2
        # written from bf16 and read back to bf16
        return {"bytes": rows * (2 * row + 4.0 * case["dim"]), "flops": rows * case["dim"] * 4.0}
    lq, lk = _attn_lengths(case)
    pairs = sum(sum(_limit(n - q + i, n, case["block"]) for i in range(q)) for q, n in zip(lq, lk))
    hq, hk, d = case["heads_q"], case["heads_k"], case["dim"]
    return {"bytes": sum(lq) * hq * (4.0 * d + 4) + 2 * sum(lk) * hk * row, "flops": 4.0 * hq * d * pairs}


# ------------------------------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"norm": _prepare_norm, "cache": _prepare_cache, "attn": _prepare_attn}[case["op"]](case, gen)


def _randn(gen, *shape, scale=1.0, kind=torch.bfloat16):
    x = torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32)
    return (x.mul_(scale) if scale != 1.0 else x).to(kind)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return _ints(at)


def _prepare_norm(case, gen):
    n, d, r = case["tokens"], case["dim"], case["requests"]
    stream = torch.float32 if case["stream"] == "fp32" else torch.bfloat16
    state = {"case": case, "x": _randn(gen, n, d, scale=2.0, kind=stream), "y": _randn(gen, n, d, scale=1.5),
             "cu_requests": _ints([n * k // r for k in range(r + 1)])}
    if case["modulated"]:
        mod = _randn(gen, r, 3, d, scale=0.4)  # the projection of the time embedding: shift, scale, gate
        state["shift"], state["scale"], state["gate"] = mod[:, 0], mod[:, 1], mod[:, 2]
    if case["weights"]:
        state["weight"] = 1.0 + _randn(gen, d, scale=0.2, kind=torch.float32)
        if case["branch_norm"] != "none":
            state["branch_weight"] = 1.0 + _randn(gen, d, scale=0.2, kind=torch.float32)
    if case["direction"] == "bwd":
        state["x_out"] = _plain_norm_fwd(state)[0]
        state["dx_out"], state["dh"] = _randn(gen, n, d, kind=stream), _randn(gen, n, d)
    return state


def _pages(case, lengths, gen):
    """A block table over shuffled pages for sequences of these lengths (-1 where a sequence has no page),
    and the number of pages."""
    counts = [(n + case["page"] - 1) // case["page"] for n in lengths]
    ids = torch.randperm(sum(counts) + 3, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((len(lengths), max(max(counts), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for g, c in enumerate(counts):
        table[g, :c] = ids[at:at + c]
        at += c
    return table, sum(counts) + 3


def _prepare_cache(case, gen):
    rows, start = _cache_lengths(case)
    h, d, page = case["heads"], case["dim"], case["page"]
    table, pages = _pages(case, [a + b for a, b in zip(rows, start)], gen)
    kv = _randn(gen, sum(rows), 2 * h * d, scale=1.5)  # the fused key/value projection
    state = {"case": case, "k": kv[:, :h * d].view(-1, h, d), "v": kv[:, h * d:].view(-1, h, d), "table": table,
             "cu": _offsets(rows), "start": _ints(start), "k_scale": None, "v_scale": None}
    for name in ("k", "v"):
        if case["kind"] == "bf16":
            state[name + "_cache"] = torch.zeros(pages, h, page, d, dtype=torch.bfloat16, device="cuda")
        else:
            state[name + "_cache"] = torch.zeros(pages, h, page, d, dtype=torch.float8_e4m3fn, device="cuda")
            state[name + "_scale"] = torch.zeros(pages, h, page, dtype=torch.uint8, device="cuda")
    return state


def _prepare_attn(case, gen):
    lq, lk = _attn_lengths(case)
    hq, hk, d, page = case["heads_q"], case["heads_k"], case["dim"], case["page"]
    table, pages = _pages(case, lk, gen)
    state = {"case": case, "q": _randn(gen, sum(lq), hq, d), "table": table, "cu": _offsets(lq), "used": _ints(lk),
             "max_q": max(lq), "max_k": max(lk), "k_scale": None, "v_scale": None}
    for name in ("k", "v"):
        x = _randn(gen, pages, hk, page, d)
        if case["kind"] == "bf16":
            state[name + "_cache"] = x
        else:
            state[name + "_cache"], state[name + "_scale"] = _plain_quantise(x)
    return state


# ------------------------------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "cache": _own_cache, "attn": _own_attn}[op](state)
    if op == "norm":
        return _plain_norm_fwd(state) if state["case"]["direction"] == "fwd" else _plain_norm_bwd(state)
    return _plain_cache(state) if op == "cache" else _plain_attn(state)


def _own_norm(state):
    import packed_varlen_attention_modality_gb300 as h3

    case = state["case"]
    step = dict(norm=case["norm"], weight=state.get("weight"), scale=state.get("scale"), shift=state.get("shift"),
                gate=state.get("gate"), branch_norm=case["branch_norm"], branch_weight=state.get("branch_weight"),
                residual_scale=case["residual_scale"], cu_requests=state["cu_requests"], eps=EPS)
    if case["direction"] == "fwd":
        return h3.residual_norm(state["x"], state["y"], **step)
    g = h3.residual_norm_bwd(state["dx_out"], state["dh"], state["x_out"], state["y"], **step)
    return {"dx": g.dx, "dy": g.dy, "weight": g.weight, "scale": g.scale, "shift": g.shift, "gate": g.gate,
            "branch_weight": g.branch_weight}


def _own_cache(state):
    import packed_varlen_attention_modality_gb300 as h3

    where = (state["k_cache"], state["v_cache"], state["table"], state["cu"], state["start"])
    scales = dict(k_scale=state["k_scale"], v_scale=state["v_scale"])
    h3.kv_cache_write(state["k"], state["v"], *where, **scales)
    return h3.kv_cache_read(*where, num_rows=state["k"].shape[0], **scales)


def _own_attn(state):
    import packed_varlen_attention_modality_gb300 as h3

    return h3.paged_attn_fwd(state["q"], state["k_cache"], state["v_cache"], state["table"], state["cu"],
                             state["used"], state["max_q"], state["max_k"], k_scale=state["k_scale"],
                             v_scale=state["v_scale"], causal_block=state["case"]["block"], return_lse=True)


# ------------------------------------------------------------------------------------------------
# plain form: gated residual and modulated norm


def _request(state):
    row = torch.arange(state["case"]["tokens"], device="cuda", dtype=torch.int32)
    return torch.searchsorted(state["cu_requests"][1:], row, right=True).clamp(max=state["case"]["requests"] - 1)


def _normed(x, kind):
    """(normed x, 1 / its size) of fp32 rows."""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _spread(state, name, request):
    """Modulation `name` of each token, fp32; None where there is none."""
    return state[name].float()[request] if name in state else None


def _plain_norm_fwd(state):
    case, request = state["case"], _request(state)
    u = _normed(state["y"].float(), case["branch_norm"])[0]
    for f in (state["branch_weight"].float() if "branch_weight" in state else None, _spread(state, "gate", request)):
        u = u if f is None else u * f
    x = case["residual_scale"] * state["x"].float() + u
    h = _normed(x, case["norm"])[0]
    if "weight" in state:
        h = h * state["weight"].float()
    if "scale" in state:
        h = h * (1.0 + _spread(state, "scale", request)) + _spread(state, "shift", request)
    return x.to(state["x"].dtype), h.to(torch.bfloat16)


def _norm_grad(g, xh, r, kind):
    if kind == "none":
        return g
    back = g - xh * (g * xh).mean(-1, keepdim=True)
    return r * (back - g.mean(-1, keepdim=True) if kind == "layer" else back)


def _plain_norm_bwd(state):
    case, request = state["case"], _request(state)
    n, requests = case["tokens"], case["requests"]
    mine = torch.zeros(requests, n, dtype=torch.float64, device="cuda")
    mine[request, torch.arange(n, device="cuda")] = 1.0

    def sums(x):  # over the tokens of each request
        return mine @ x.double()

    grads = {}
    xh, r = _normed(state["x_out"].float(), case["norm"])
    dh = state["dh"].float()
    if "shift" in state:
        grads["shift"] = sums(dh)
    u = sums(dh * xh)
    weight = state["weight"].float() if "weight" in state else 1.0
    one = 1.0
    if "scale" in state:
        one = 1.0 + state["scale"].float()
        grads["scale"] = u * weight
    if "weight" in state:
        grads["weight"] = (u * one).sum(0)
    g = dh * weight * (one[request] if "scale" in state else 1.0)
    total = state["dx_out"].float() + _norm_grad(g, xh, r, case["norm"])
    grads["dx"] = (case["residual_scale"] * total).to(state["x"].dtype)
    yh, r = _normed(state["y"].float(), case["branch_norm"])
    v = sums(total * yh)
    weight = state["branch_weight"].float() if "branch_weight" in state else 1.0
    gate = state["gate"].float() if "gate" in state else 1.0
    if "gate" in state:
        grads["gate"] = v * weight
    if "branch_weight" in state:
        grads["branch_weight"] = (v * gate).sum(0)
    g = total * weight * (gate[request] if "gate" in state else 1.0)
    grads["dy"] = _norm_grad(g, yh, r, case["branch_norm"]).to(torch.bfloat16)
    return {k: grads[k].float() if k in grads and k not in ("dx", "dy") else grads.get(k)
            for k in ("dx", "dy", "weight", "scale", "shift", "gate", "branch_weight")}


# ------------------------------------------------------------------------------------------------
# plain form: the cache


def _power(e):
    """2^e, fp32, exact, for int32 exponents of normal numbers."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_quantise(x):
    """Rows [..., dim] -> (e4m3 values, biased exponents of their scales).  The scale is the least power of
    two with which the row's largest value fits e4m3 (448 = 0.875 * 2^9)."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = (e - 9 + (m > 0.875).int()).clamp(SCALE_MIN, SCALE_MAX)
    return (x * _power(-e)[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_values(q, scale):
    """What a cache's entries stand for, fp32."""
    return q.float() if scale is None else q.float() * _power(scale.int() - 127)[..., None]


def _slots(state, lengths, first):
    """(page, row in it) of each of a packed batch's rows."""
    row = torch.arange(lengths, device="cuda", dtype=torch.int32)
    g = torch.searchsorted(state["cu"][1:], row, right=True).clamp(max=state["cu"].numel() - 2)
    at = (row - state["cu"][g] + first[g]).long()
    page = state["case"]["page"]
    return state["table"][g, at // page].long(), at % page


def _plain_cache(state):
    pages, rows = _slots(state, state["k"].shape[0], state["start"])
    got = []
    for name in ("k", "v"):
        x, cache, scale = state[name], state[name + "_cache"], state[name + "_scale"]
        if scale is None:
            cache[pages, :, rows] = x
            got.append(cache[pages, :, rows])
        else:
            q, s = _plain_quantise(x)
            cache.view(torch.uint8)[pages, :, rows] = q.view(torch.uint8)
            scale[pages, :, rows] = s
            back = cache.view(torch.uint8)[pages, :, rows].view(torch.float8_e4m3fn)
            got.append(_plain_values(back, scale[pages, :, rows]).to(torch.bfloat16))
    return tuple(got)


# ------------------------------------------------------------------------------------------------
# plain form: attention over the cache, on padded batches


def _gathered(state, name):
    """Keys or values of the segments, [segments, heads, max_k, dim] fp32 (past the end: some row)."""
    j = torch.arange(state["max_k"], device="cuda")
    page = state["case"]["page"]
    pages = state["table"][:, j // page].long().clamp(min=0)
    cache, scale = state[name + "_cache"], state[name + "_scale"]
    if scale is None:
        x = cache[pages, :, j % page].float()
    else:
        x = _plain_values(cache.view(torch.uint8)[pages, :, j % page].view(torch.float8_e4m3fn), scale[pages, :, j % page])
    return x.transpose(1, 2)


def _plain_attn(state):
    case, cu, most = state["case"], state["cu"], state["max_q"]
    hq, hk, d, block = case["heads_q"], case["heads_k"], case["dim"], case["block"]
    n, b = state["q"].shape[0], cu.numel() - 1
    i = torch.arange(most, device="cuda")
    q = state["q"][(cu[:-1, None] + i).clamp(max=n - 1)].float().transpose(1, 2)
    q = q.reshape(b, hk, hq // hk * most, d)  # the query heads of one key head side by side
    used = state["used"][:, None].long()
    p = used - cu.diff()[:, None] + i
    limit = torch.minimum((p // block + 1) * block, used) if block else used.expand(b, most)
    limit = limit[:, None, None].expand(b, hk, hq // hk, most).reshape(b, hk, -1, 1)
    s = torch.matmul(q, _gathered(state, "k").transpose(2, 3)).mul_(d ** -0.5)
    s.masked_fill_(torch.arange(state["max_k"], device="cuda") >= limit, -math.inf)
    top = s.amax(-1, keepdim=True)
    w = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, _gathered(state, "v")) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)  # -inf for a row that sees no key
    row = torch.arange(n, device="cuda", dtype=torch.int32)
    g = torch.searchsorted(cu[1:], row, right=True).clamp(max=b - 1)
    at = (row - cu[g]).long()
    out = o.reshape(b, hq, most, d)[g, :, at].to(torch.bfloat16)
    return out, lse.reshape(b, hq, most)[g, :, at].t().contiguous()


# ------------------------------------------------------------------------------------------------
# the definition in fp64


def exact(case, seed):
    state = prepare(case, seed)
    return {"norm": _exact_norm, "cache": _exact_cache, "attn": _exact_attn}[case["op"]](case, state)


def _exact_unit(x, kind):
    """(normed rows, their divisors), fp64."""
    if kind == "none":
        return x, None
    centre = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
    size = ((x - centre).pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    return (x - centre) / size, size


def _exact_norm(case, state):
    d, a = case["dim"], case["residual_scale"]
    ones = torch.ones(d, dtype=torch.float64, device="cuda")
    w = state["weight"].double() if "weight" in state else ones
    wb = state["branch_weight"].double() if "branch_weight" in state else ones
    cuts = state["cu_requests"].tolist()
    parts = {k: [] for k in ("x", "h", "dx", "dy", "scale", "shift", "gate", "weight", "branch_weight")}
    for r in range(case["requests"]):
        rows = slice(cuts[r], cuts[r + 1])
        scale, shift, gate = (state[k][r].double() if k in state else f * ones
                              for k, f in (("scale", 0.0), ("shift", 0.0), ("gate", 1.0)))
        unit, size = _exact_unit(state["y"][rows].double(), case["branch_norm"])
        if case["direction"] == "fwd":
            x = state["x"][rows].double() * a + unit * wb * gate
            parts["x"].append(x)
            parts["h"].append(_exact_unit(x, case["norm"])[0] * w * (scale + 1) + shift)
            continue
        normed, length = _exact_unit(state["x_out"][rows].double(), case["norm"])
        dh = state["dh"][rows].double()
        dot = (dh * normed).sum(0)
        parts["shift"].append(dh.sum(0))
        parts["scale"].append(dot * w)
        parts["weight"].append(dot * (scale + 1))

        def through(g, unit, size, kind):
            if kind == "none":
                return g
            g = g - unit * ((g * unit).sum(-1, keepdim=True) / d) - (g.sum(-1, keepdim=True) / d if kind == "layer" else 0)
            return g / size

        t = state["dx_out"][rows].double() + through(dh * (w * (scale + 1)), normed, length, case["norm"])
        parts["dx"].append(t * a)
        dot = (t * unit).sum(0)
        parts["gate"].append(dot * wb)
        parts["branch_weight"].append(dot * gate)
        parts["dy"].append(through(t * (wb * gate), unit, size, case["branch_norm"]))
    if case["direction"] == "fwd":
        return torch.cat(parts["x"]), torch.cat(parts["h"])
    grads = {"dx": torch.cat(parts["dx"]), "dy": torch.cat(parts["dy"])}
    for k in ("weight", "scale", "shift", "gate", "branch_weight"):
        summed = torch.stack(parts[k])
        grads[k] = None if k not in state else summed.sum(0) if k.endswith("weight") else summed
    return grads


def _exact_cache(case, state):
    def power(e):
        return (e + 1023 << 52).view(torch.float64)

    got = []
    for x in (state["k"].double(), state["v"].double()):
        if case["kind"] == "e4m3":
            most = x.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(most / E4M3_MOST)).clamp(SCALE_MIN, SCALE_MAX).long()
            e += (most > E4M3_MOST * power(e)).long() - (most <= E4M3_MOST * power(e - 1)).long()
            unit = power(e.clamp(SCALE_MIN, SCALE_MAX))
            z = x / unit
            # three bits behind the leading one, steps of 2^-9 below 2^-6; to even at ties
            step = power(torch.frexp(z)[1].clamp(min=-5).long() - 4)
            x = torch.round(z / step) * step * unit
        got.append(x)
    return tuple(got)


def _exact_attn(case, state):
    lq, lk = _attn_lengths(case)
    hq, hk, d, page = case["heads_q"], case["heads_k"], case["dim"], case["page"]
    o = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, o.shape[0]), -math.inf, dtype=torch.float64, device="cuda")

    def rows(name, g, h):
        pages = state["table"][g, :(lk[g] + page - 1) // page].long()
        x = state[name + "_cache"].view(torch.uint8 if case["kind"] == "e4m3" else torch.bfloat16)[pages, h]
        if case["kind"] == "e4m3":
            x = x.view(torch.float8_e4m3fn).double() * 2.0 ** (state[name + "_scale"][pages, h].double()[..., None] - 127)
        return x.double().reshape(-1, d)[:lk[g]]

    a = 0
    for g in range(len(lq)):
        limit = torch.tensor([_limit(lk[g] - lq[g] + i, lk[g], case["block"]) for i in range(lq[g])], device="cuda")
        hidden = torch.arange(lk[g], device="cuda") >= limit[:, None]
        for h in range(hk):
            k, v = rows("k", g, h), rows("v", g, h)
            for head in range(h * hq // hk, (h + 1) * hq // hk):
                s = state["q"][a:a + lq[g], head].double() @ k.T / math.sqrt(d)
                s = s.masked_fill(hidden, -math.inf)
                whole = torch.logsumexp(s, dim=1)
                lse[head, a:a + lq[g]] = whole
                o[a:a + lq[g], head] = (s - whole[:, None]).exp() @ v
        a += lq[g]
    return o, lse
