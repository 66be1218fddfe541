"""What a prompt passes through between the projections, and how its tokens are scored: the workloads and their plain forms.

Four operators, each with a plain form in elementary torch operations and the call of this library:

  rope   norm of each head and rotation by position: half and interleaved pairs, part of the head, scaled for long
         contexts (q4k_rope)
  qkv    the same for queries and keys, and the write of keys and values into the paged cache, bf16 or e4m3 with a
         scale per row (q4k_rope_kv_write)
  chunk  attention of each request's new tokens, one or many, over the paged cache (q4k_paged_attn_chunk)
  score  log-probability and rank of given tokens, entropy and the most likely alternatives (q4k_logprobs)

listed() and draw() give cases, prepare() what a program holds before the call, run() one pass through an
operator, work() its bytes and operations, exact() its result in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp32": 4, "e4m3": 1}
AMAX_FLOOR = 2.0 ** -100  # smallest row maximum that a scale is derived from
EPS = 1e-6
ROPE_BASE = 1e6
ORIGINAL = 32768  # context that the positions were trained on, where they are scaled


def listed():
    return [
        # the queries of a decode step of 16 requests, straight from the fp32 projection: latency
        {"name": "rope_decode", "op": "rope", "tokens": 16, "heads": 64, "dim": 128, "rot": 128, "pairs": "half", "norm": False, "scaled": False, "input": "fp32", "output": "bf16", "max_pos": 131071},
        # a prompt's block of odd length: wide heads, a quarter of each rotated, adjacent pairs
        {"name": "rope_prefill_part", "op": "rope", "tokens": 8191, "heads": 24, "dim": 256, "rot": 64, "pairs": "interleaved", "norm": True, "scaled": False, "input": "bf16", "output": "bf16", "max_pos": 8190},
        # a decode step of 24 requests: one fused fp32 projection, head norms, bf16 cache
        {"name": "qkv_decode", "op": "qkv", "tokens": 24, "q_heads": 64, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": "half", "norm": True, "scaled": False, "input": "fp32", "cache": "bf16", "page": 16, "max_pos": 40000},
        # a prompt's block into an 8-bit cache, positions scaled for a long context
        {"name": "qkv_prefill_e4m3", "op": "qkv", "tokens": 8191, "q_heads": 64, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": "half", "norm": True, "scaled": True, "input": "bf16", "cache": "e4m3", "page": 32, "max_pos": 131071},
        # a short question after a short conversation: latency
        {"name": "chunk_short", "op": "chunk", "requests": 1, "idle": 0, "chunks": 1, "chunk": 45, "min_len": 745, "max_len": 745, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "cache": "bf16", "window": 0, "pad": 3},
        # proposed tokens of 8 requests checked in one step, long contexts
        {"name": "chunk_verify", "op": "chunk", "requests": 8, "idle": 0, "chunks": 8, "chunk": 5, "min_len": 20001, "max_len": 60000, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "cache": "bf16", "window": 0, "pad": 0},
        # one long prompt, nothing cached before
        {"name": "chunk_prompt", "op": "chunk", "requests": 1, "idle": 0, "chunks": 1, "chunk": 8191, "min_len": 8191, "max_len": 8191, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 32, "cache": "bf16", "window": 0, "pad": 0},
        # a step of many requests: most append one token, three a piece of their prompt, two wait; 8-bit cache
        {"name": "chunk_mixed_e4m3", "op": "chunk", "requests": 60, "idle": 2, "chunks": 3, "chunk": 700, "min_len": 800, "max_len": 16001, "q_heads": 64, "kv_heads": 4, "dim": 128, "page": 64, "cache": "e4m3", "window": 0, "pad": 11},
        # pieces of four prompts, wide heads under a sliding window
        {"name": "chunk_window_256", "op": "chunk", "requests": 4, "idle": 0, "chunks": 4, "chunk": 2049, "min_len": 2049, "max_len": 9000, "q_heads": 24, "kv_heads": 4, "dim": 256, "page": 32, "cache": "bf16", "window": 4096, "pad": 0},
        # the chosen token of one request, with alternatives
        {"name": "score_one", "op": "score", "rows": 1, "vocab": 32000, "top": 20, "input": "fp32", "masked": False},
        # a decode step of 64 requests, some under a grammar
        {"name": "score_decode", "op": "score", "rows": 64, "vocab": 131072, "top": 5, "input": "fp32", "masked": True},
        # every token of a prompt
        {"name": "score_prompt", "op": "score", "rows": 2047, "vocab": 131072, "top": 1, "input": "bf16", "masked": False},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _head_shape(rng):
    dim = rng.choice([64, 128, 128, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
    return {"dim": dim, "rot": rot, "pairs": rng.choice(["half", "half", "interleaved"]), "norm": rng.random() < 0.5, "scaled": rng.random() < 0.4, "input": rng.choice(["bf16", "fp32"]),
            "max_pos": _log_int(rng, 30, 1000000)}


def draw(rng):
    op = rng.choice(["rope", "qkv", "qkv", "chunk", "chunk", "chunk", "score", "score"])
    if op == "rope":
        case = dict({"op": op}, **_head_shape(rng))
        case["dim"] = rng.choice([case["dim"], 80, 96]) if case["rot"] <= 64 else case["dim"]
        case["heads"] = rng.choice([1, 4, 5, 8, 24, 32, 64])
        return dict(case, output=rng.choice(["bf16", "bf16", "fp32"]), tokens=_log_int(rng, 1, 48000000 // (case["heads"] * case["dim"] * 4) if case["heads"] > 8 else 8191))
    if op == "qkv":
        kv = rng.choice([1, 2, 4, 8])
        return dict({"op": op, "kv_heads": kv, "q_heads": kv * rng.choice([1, 2, 3, 5, 8]), "cache": rng.choice(["bf16", "e4m3"]), "page": rng.choice([16, 32, 64, 128]), "tokens": _log_int(rng, 1, 4000)}, **_head_shape(rng))
    if op == "chunk":
        dim, kv, cache = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice(["bf16", "bf16", "e4m3"])
        heads = kv * rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        requests = _log_int(rng, 1, 64)
        idle = rng.choice([0, 0, min(2, requests - 1)])
        chunks = rng.randint(0, min(4, requests - idle))
        # a chunk and a length whose products stay within those of the long prompt
        max_len = _log_int(rng, 8, max(16, min(60000, 2.0e9 / (4 * dim * kv * requests))))
        limit = max(2, min(8000, max_len, 2.5e11 / (max(chunks, 1) * max_len * heads * dim)))
        chunk = _log_int(rng, 2, limit)
        return {"op": op, "requests": requests, "idle": idle, "chunks": chunks, "chunk": chunk, "min_len": rng.randint(1, max_len), "max_len": max_len, "q_heads": heads, "kv_heads": kv, "dim": dim,
                "page": rng.choice([16, 32, 64, 128, 256]), "cache": cache, "window": rng.choice([0, 0, 0, _log_int(rng, 1, 8192)]), "pad": rng.choice([0, 0, rng.randint(1, 40)])}
    vocab = rng.choice([_log_int(rng, 100, 131072), 32000, 65536, 100003, 131072])
    return {"op": op, "rows": _log_int(rng, 1, min(2000, 130000000 // vocab)), "vocab": vocab, "top": rng.choice([0, 1, 5, 20, rng.randint(2, 32)]), "input": rng.choice(["bf16", "fp32"]), "masked": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------ inputs


def _spread(count, low, high):
    """`count` whole numbers spread evenly over low..high, the same ones every time."""
    return [low + int((high - low) * ((i + 1) * 0.6180339887498949 % 1.0) + 0.5) for i in range(count)]


def _requests(case):
    """(cached tokens with the new ones, new tokens) of each request: idle ones append nothing."""
    n = case["requests"]
    lens = [case["max_len"]] + _spread(n - 1, case["min_len"], case["max_len"])
    new = [case["chunk"] - i % 3 if case["chunk"] > 4 else case["chunk"] for i in range(case["chunks"])] + [1] * (n - case["chunks"] - case["idle"]) + [0] * case["idle"]
    return [(max(a, b), b) for a, b in zip(lens, new)]


def _order(case):
    """The order in which the requests stand in the step: chunks among single tokens."""
    n = case["requests"]
    step = next(s for s in (7, 5, 3, 2, 1) if math.gcd(s, n) == 1)
    return [(i * step + n // 3) % n for i in range(n)]


def _freqs(case):
    """(radians per position of each pair, amplitude): scaled positions divide the slow frequencies by 4 and leave the fast
    ones, with a ramp between 32 and 1 turns over the original context."""
    rot = case["rot"]
    plain = [ROPE_BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not case["scaled"]:
        return plain, 1.0
    at = lambda turns: rot * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE))  # noqa: E731
    low, high = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
    keep = [1.0 - min(1.0, max(0.0, (i - low) / max(0.001, high - low))) for i in range(rot // 2)]
    return [f / 4.0 * (1.0 - k) + f * k for f, k in zip(plain, keep)], 1.0 + 0.1 * math.log(4.0)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rand(g, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16 if dtype == torch.bfloat16 else torch.float32, device=DEV).normal_(generator=g)
    return x.mul_(scale).to(dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    return {"rope": _prepare_rope, "qkv": _prepare_qkv, "chunk": _prepare_chunk, "score": _prepare_score}[case["op"]](case, _gen(seed))


def _angles(case, g):
    """Positions of a step's tokens, the frequencies, and these as turns of 2^-64."""
    t = case["tokens"]
    # a few requests, each with a run of positions
    first = torch.randint(0, max(1, case["max_pos"] - t // 8), (8,), generator=g, device=DEV)
    at = torch.arange(t, device=DEV)
    pos = (first[at % 8] + at // 8).clamp(max=case["max_pos"]).to(torch.int32)
    pos[0] = case["max_pos"]
    if t > 3:
        pos[torch.randint(1, t, (t // 60 + 1,), generator=g, device=DEV)] = -1  # padding tokens
    freqs, amplitude = _freqs(case)
    steps = [round(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for f in freqs]
    return {"pos": pos, "freqs": torch.tensor(freqs, dtype=torch.float64, device=DEV), "amplitude": amplitude, "steps": _ints([s - 2 ** 64 if s >= 2 ** 63 else s for s in steps], torch.int64)}


def _gamma(case, g):
    return _rand(g, (case["dim"],), torch.float32, 0.2) + 1.0 if case["norm"] else None


def _prepare_rope(case, g):
    t, h, d = case["tokens"], case["heads"], case["dim"]
    s = dict(case, **_angles(case, g), gamma=_gamma(case, g), x=_rand(g, (t, h, d), TYPES[case["input"]], 2.0))
    return dict(s, out=torch.zeros((t, h, d), dtype=TYPES[case["output"]], device=DEV))


def _prepare_qkv(case, g):
    t, hq, h, d, page = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    pages = -(-2 * t // page) + 1
    # one fused projection: a row of the step's output holds queries, keys and values
    x = _rand(g, (t, hq + 2 * h, d), TYPES[case["input"]], 2.0)
    s = dict(case, **_angles(case, g), q=x[:, :hq], k=x[:, hq:hq + h], v=x[:, hq + h:], q_gamma=_gamma(case, g), k_gamma=_gamma(case, g), pages=pages)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:t].to(torch.int32)
    s["slots"] = torch.where(s["pos"] < 0, torch.full_like(slots, -1), slots)
    s["out"] = torch.zeros((t, hq, d), dtype=torch.bfloat16, device=DEV)
    for name in ("k", "v"):
        # one page more than the calls are given: the plain form drops padding tokens there
        s[name + "_cache"] = torch.zeros((pages + 1, h, page, d), dtype=TYPES[case["cache"]], device=DEV)
        s[name + "_scale"] = torch.zeros((pages + 1, h, page), dtype=torch.float32, device=DEV) if case["cache"] == "e4m3" else None
    return s


def _prepare_chunk(case, g):
    n, page, h, d = case["requests"], case["page"], case["kv_heads"], case["dim"]
    both = [_requests(case)[i] for i in _order(case)]
    lens = _ints([a for a, _ in both])
    cu = [0]
    for _, b in both:
        cu.append(cu[-1] + b)
    width = -(-case["max_len"] // page) + 1
    have = torch.div(lens + page - 1, page, rounding_mode="floor")
    used = torch.arange(width, device=DEV)[None, :] < have[:, None]
    rank = torch.cumsum(used.flatten(), 0).view(n, width) - 1
    pages = sum(-(-a // page) for a, _ in both) + 1
    ids = (torch.randperm(pages - 1, generator=g, device=DEV) + 1).to(torch.int32)
    # page 0 is nobody's: rows past a request's pages point at it
    table = torch.where(used, ids[rank.clamp(min=0).clamp(max=pages - 2)], torch.zeros_like(rank, dtype=torch.int32)).contiguous()
    t = cu[-1] + case["pad"]  # a step's buffers may be longer than what its requests append
    s = dict(case, both=both, starts=cu, lens=lens, cu=_ints(cu, torch.int64), table=table, softmax_scale=1.0 / math.sqrt(d), tokens=t)
    s["q"] = _rand(g, (t, case["q_heads"], d), torch.bfloat16, 1.5)
    s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((t, case["q_heads"]), device=DEV)
    # what no request has written yet: the rest of a last page, and page 0
    last = table.gather(1, (have - 1)[:, None].long()).long()
    at = torch.arange(page, device=DEV)[None, :]
    stale = (have[:, None] - 1) * page + at >= lens[:, None]
    flat = torch.where(stale, last * page + at, at.expand(n, page)).flatten()
    for name in ("k", "v"):
        cache = _rand(g, (pages, h, page, d), TYPES[case["cache"]])
        if case["cache"] == "e4m3":
            cache = cache.view(torch.uint8)
            cache[flat // page, :, flat % page] = 0x7F  # NaN in e4m3
            s[name + "_cache"] = cache.view(torch.float8_e4m3fn)
            s[name + "_scale"] = torch.empty((pages, h, page), device=DEV).uniform_(0.25, 2.0, generator=g)
        else:
            cache[flat // page, :, flat % page] = float("nan")
            s[name + "_cache"], s[name + "_scale"] = cache, None
    return s


def _prepare_score(case, g):
    b, v = case["rows"], case["vocab"]
    logits = _rand(g, (b, v), torch.float32, 2.5)
    # a few likely tokens in each row, as a language model gives them
    likely = torch.randint(0, v, (b, 40), generator=g, device=DEV)
    lift = torch.empty((b, 40), device=DEV).exponential_(0.25, generator=g)
    logits.scatter_add_(1, likely, lift.clamp(max=16.0))
    row = torch.arange(b, device=DEV)
    if case["masked"]:
        logits[row % 5 == 3, : v // 2] = -math.inf  # a grammar that forbids half of the tokens
    # mostly one of the likely tokens, sometimes any, sometimes none
    token = torch.where(row % 7 == 2, torch.randint(0, v, (b,), generator=g, device=DEV), likely[:, 0])
    token = torch.where(row % 31 == 30, torch.full_like(token, -1), token).to(torch.int32)
    return dict(case, logits=logits.to(TYPES[case["input"]]), token=token)


# ------------------------------------------------------------------------------------------ the passes


def run(s):
    return {"rope": _run_rope, "qkv": _run_qkv, "chunk": _run_chunk, "score": _run_score}[s["op"]](s)


def _plain_heads(x, gamma, s):
    """fp32 heads, normed where there is a gamma, their first `rot` values rotated by the positions' angles."""
    x = x.float()
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    angle = s["pos"].double()[:, None] * s["freqs"]
    cos, sin = ((f(angle) * s["amplitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    rot = s["rot"]
    if s["pairs"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_rope(s):
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        return q4k.q4k_rope(s["x"], s["pos"], s["steps"], gamma=s["gamma"], eps=EPS, interleaved=s["pairs"] == "interleaved", amplitude=s["amplitude"], out=s["out"])
    live = (s["pos"] >= 0)[:, None, None]
    s["out"].copy_(torch.where(live, _plain_heads(s["x"], s["gamma"], s).to(s["out"].dtype), s["out"]))
    return s["out"]


def _run_qkv(s):
    n = s["pages"]
    caches = [s[k][:n] for k in ("k_cache", "v_cache", "k_scale", "v_scale") if s[k] is not None]
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        q4k.q4k_rope_kv_write(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["steps"], *caches, q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=EPS, interleaved=s["pairs"] == "interleaved",
                              amplitude=s["amplitude"], out=s["out"])
        return [s["out"]] + caches
    live = (s["pos"] >= 0)[:, None, None]
    s["out"].copy_(torch.where(live, _plain_heads(s["q"], s["q_gamma"], s).to(torch.bfloat16), s["out"]))
    page = s["page"]
    slots = torch.where(s["slots"] < 0, torch.full_like(s["slots"], n * page), s["slots"]).long()
    at, off = slots // page, slots % page
    _plain_store(_plain_heads(s["k"], s["k_gamma"], s), s["k_cache"], s["k_scale"], at, off)
    _plain_store(s["v"].float(), s["v_cache"], s["v_scale"], at, off)
    return [s["out"]] + caches


def _plain_store(x, cache, scales, at, off):
    if scales is None:
        cache[at, :, off] = x.to(cache.dtype)
        return
    amax = x.abs().amax(-1).clamp(min=AMAX_FLOOR)
    scales[at, :, off] = amax / 448.0
    cache.view(torch.uint8)[at, :, off] = (x * (448.0 / amax)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _run_chunk(s):
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        return q4k.q4k_paged_attn_chunk(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], s["softmax_scale"], s["k_scale"], s["v_scale"], window=s["window"], out=s["out"], lse=s["lse"])
    h, page, d = s["kv_heads"], s["page"], s["dim"]
    group = s["q_heads"] // h
    for r, (length, new) in enumerate(s["both"]):
        if not new:
            continue
        # the tokens that the first of the new ones may see, and what comes after them
        low = max(0, length - new + 1 - s["window"]) if s["window"] else 0
        pages = s["table"][r, low // page:-(-length // page)].long()
        begin = low // page * page
        k, v = (_plain_rows(s[x + "_cache"], s[x + "_scale"], pages)[:, low - begin:length - begin] for x in "kv")
        part = slice(s["starts"][r], s["starts"][r] + new)
        q = s["q"][part].float().view(new, h, group, d).permute(1, 0, 2, 3).reshape(h, new * group, d)
        score = torch.matmul(q, k.transpose(1, 2)).mul_(s["softmax_scale"]).view(h, new, group, length - low)
        at, pos = torch.arange(low, length, device=DEV)[None, :], torch.arange(length - new, length, device=DEV)[:, None]
        hidden = (at > pos) | ((at <= pos - s["window"]) if s["window"] else False)
        score.masked_fill_(hidden[None, :, None, :], -math.inf)
        top = score.amax(-1, keepdim=True)
        weight = score.sub_(top).exp_()
        total = weight.sum(-1, keepdim=True)
        out = torch.matmul(weight.view(h, new * group, -1), v).view(h, new, group, d) / total
        s["out"][part] = out.permute(1, 0, 2, 3).reshape(new, h * group, d).to(torch.bfloat16)
        s["lse"][part] = (top + torch.log(total)).squeeze(-1).permute(1, 0, 2).reshape(new, h * group)
    return s["out"], s["lse"]


def _plain_rows(cache, scales, pages):
    """[heads, tokens, dim] fp32 of the rows of these pages."""
    x = cache.view(torch.uint8)[pages].view(cache.dtype).float() if scales is not None else cache[pages].float()
    if scales is not None:
        x = x * scales[pages][..., None]
    return x.transpose(0, 1).flatten(1, 2)


def _run_score(s):
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        return q4k.q4k_logprobs(s["logits"], s["token"], top=s["top"])
    x = s["logits"].double()
    b, v = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x)
    high = x.max(-1, keepdim=True).values
    z = torch.where(x == high, 0.0, x - high)
    weight = torch.exp(z)
    total = weight.sum(-1, keepdim=True)
    lse = torch.log(total)
    entropy = (lse - torch.where(weight > 0, weight * z, 0.0).sum(-1, keepdim=True) / total)[:, 0]
    token = s["token"].long()[:, None]
    real = (token >= 0) & (token < v)
    index = torch.arange(v, device=DEV)[None, :]
    at = x.gather(1, token.clamp(0, v - 1))
    rank = ((x > at) | ((x == at) & (index < token))).sum(-1, keepdim=True)
    logp = torch.where(real, z.gather(1, token.clamp(0, v - 1)) - lse, -math.inf)
    n = min(s["top"], v)
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    kept = value[:, :n] > -math.inf
    tops = torch.where(kept, order[:, :n], -1).to(torch.int32)
    top_logp = torch.where(kept, z.gather(1, order[:, :n]) - lse, -math.inf).float()
    return logp[:, 0].float(), torch.where(real, rank, -1)[:, 0].to(torch.int32), entropy.float(), tops, top_logp


# ------------------------------------------------------------------------------------------ work and exact results


def work(case):
    op = case["op"]
    if op == "rope":
        values = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": values * (SIZE[case["input"]] + SIZE[case["output"]]) + 4 * case["tokens"] + 4 * case["rot"], "flops": 7.0 * values}
    if op == "qkv":
        rows = case["tokens"] * case["kv_heads"]
        values = case["tokens"] * case["q_heads"] * case["dim"]
        cache = 2 * rows * (case["dim"] * (SIZE[case["input"]] + SIZE[case["cache"]]) + (4 if case["cache"] == "e4m3" else 0))
        return {"bytes": values * (SIZE[case["input"]] + 2) + cache + 8 * case["tokens"] + 4 * case["rot"], "flops": 7.0 * (values + rows * case["dim"])}
    if op == "chunk":
        seen = pairs = new = 0
        for length, m in _requests(case):
            w = case["window"] or length
            if m:
                seen += min(length, w + m - 1)
                new += m
                # of its new tokens, those below the window see all before them, the others the window
                short = min(m, max(0, w - (length - m)))
                first = length - m + 1
                pairs += short * first + short * (short - 1) // 2 + (m - short) * w
        row = case["dim"] * SIZE[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)
        q = new * case["q_heads"]
        return {"bytes": 2 * seen * case["kv_heads"] * row + q * (4 * case["dim"] + 4) + 4 * seen // case["page"], "flops": 4.0 * pairs * case["q_heads"] * case["dim"]}
    return {"bytes": case["rows"] * (case["vocab"] * SIZE[case["input"]] + 16 + 8 * case["top"]), "flops": 6.0 * case["rows"] * case["vocab"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "qkv": _exact_qkv, "chunk": _exact_chunk, "score": _exact_score}[case["op"]](s)


def _exact_heads(x, gamma, s):
    """Each pair as a complex number times amplitude e^(i angle), in 64 bits, for the tokens that are not padding."""
    live = (s["pos"] >= 0).nonzero()[:, 0]
    y = x[live].double()
    if gamma is not None:
        y = gamma.double() * y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + EPS)
    rot = s["rot"]
    turn = torch.polar(torch.full((len(live), rot // 2), s["amplitude"], dtype=torch.float64, device=DEV), torch.outer(s["pos"][live].double(), s["freqs"]))[:, None]
    even = s["pairs"] == "interleaved"
    first = torch.arange(0, rot, 2, device=DEV) if even else torch.arange(rot // 2, device=DEV)
    second = first + (1 if even else rot // 2)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return live, y


def _exact_rope(s):
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    live, y = _exact_heads(s["x"], s["gamma"], s)
    out[live] = y
    return out


def _exact_qkv(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    live, y = _exact_heads(s["q"], s["q_gamma"], s)
    out[live] = y
    rows = {"k": _exact_heads(s["k"], s["k_gamma"], s)[1], "v": s["v"][live].double()}
    slot = s["slots"][live].long()
    caches, scales = [], []
    for name, x in rows.items():
        cache = torch.zeros((s["pages"] * s["page"], s["kv_heads"], s["dim"]), dtype=torch.float64, device=DEV)
        if s["cache"] == "e4m3":
            step = x.abs().max(-1, keepdim=True).values.clamp(min=AMAX_FLOOR) / 448
            x = x / step
            scale = torch.zeros((s["pages"] * s["page"], s["kv_heads"]), dtype=torch.float64, device=DEV)
            scale[slot] = step[..., 0]
            scales.append(scale.view(s["pages"], s["page"], s["kv_heads"]).permute(0, 2, 1).contiguous())
        cache[slot] = x
        caches.append(cache.view(s["pages"], s["page"], s["kv_heads"], s["dim"]).permute(0, 2, 1, 3).contiguous())
    return [out] + caches + scales


def _exact_chunk(s):
    group, page = s["q_heads"] // s["kv_heads"], s["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    if sum(a * b for a, b in s["both"]) * s["q_heads"] * s["dim"] > 1e12:
        return None
    for r, (length, new) in enumerate(s["both"]):
        if not new:
            continue
        pages = s["table"][r, :-(-length // page)].long()
        for j in range(s["kv_heads"]):
            rows = []
            for name in ("k", "v"):
                x = s[name + "_cache"].view(torch.uint8 if s["cache"] == "e4m3" else torch.bfloat16)[pages, j].view(TYPES[s["cache"]]).double()
                if s["cache"] == "e4m3":
                    x *= s[name + "_scale"][pages, j].double().unsqueeze(-1)
                rows.append(x.flatten(0, 1)[:length])
            step = max(1, 300000000 // (length * group))
            for i in range(0, new, step):  # some of the new tokens at a time
                count = min(step, new - i)
                part = slice(s["starts"][r] + i, s["starts"][r] + i + count)
                heads = slice(j * group, (j + 1) * group)
                age = torch.arange(length - new + i, length - new + i + count, device=DEV)[:, None] - torch.arange(length, device=DEV)[None, :]
                seen = (age >= 0) & (age < (s["window"] or length))
                z = (s["softmax_scale"] * (s["q"][part, heads].double().flatten(0, 1) @ rows[0].T)).view(count, group, length)
                z = torch.where(seen[:, None], z, -math.inf)
                norm = torch.logsumexp(z, -1)
                lse[part, heads] = norm
                out[part, heads] = (torch.exp(z - norm[..., None]).flatten(0, 1) @ rows[1]).view(count, group, -1)
    return out, lse


def _exact_score(s):
    logp, entropy, tops = [], [], []
    v, n = s["vocab"], s["top"]
    for x, token in zip(s["logits"].split(256), s["token"].long().split(256)):
        x = x.double().nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        ln = x - torch.logsumexp(x, 1, keepdim=True)
        entropy.append(-torch.xlogy(torch.exp(ln), torch.exp(ln)).sum(1))
        mine = ln.gather(1, token.clamp(0, v - 1)[:, None])[:, 0]
        logp.append(torch.where((token < 0) | (token >= v), torch.full_like(mine, -math.inf), mine))
        tops.append(torch.topk(ln, min(n, v), dim=1).values)
    return torch.cat(logp), None, torch.cat(entropy), None, torch.cat(tops)
