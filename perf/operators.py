"""What surrounds the projections in a decode step: the workloads and their plain forms.

Five operators, each with a plain form in elementary torch operations and the call of this library:

  plan   block tables and slot maps from request lengths (q4k_kv_plan)
  write  new keys and values into the paged cache, bf16 or e4m3 with a scale per row (q4k_kv_write)
  attn   attention of one new token per request over the paged cache (q4k_paged_attn)
  norm   residual addition and root-mean-square norm, bf16 or e4m3 with a scale per 128 values (q4k_add_rmsnorm)
  sample temperature, top-k, top-p and min-p sampling from given random numbers (q4k_sample)

listed() and draw() give cases, prepare() what a program holds before the call, run() one pass through an
operator, work() its bytes and operations, exact() its result in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp32": 4, "e4m3": 1}
AMAX_FLOOR = 2.0 ** -100  # smallest block maximum that a scale is derived from


def listed():
    return [
        # a decode step of 64 requests: one token each, a page of 16 now and then
        {"name": "plan_decode", "op": "plan", "requests": 64, "max_len": 8000, "page": 16, "chunk": 1, "chunked": 0, "finished": 0},
        # a large mixed step: 1000 requests, some with a prefill chunk, some done
        {"name": "plan_mixed", "op": "plan", "requests": 1000, "max_len": 16000, "page": 16, "chunk": 700, "chunked": 61, "finished": 37},
        # the new row of 16 requests, straight from the fp32 projection
        {"name": "write_decode", "op": "write", "tokens": 16, "heads": 8, "dim": 128, "page": 16, "input": "fp32", "cache": "bf16"},
        # a prefill block whose length is odd, into an 8-bit cache
        {"name": "write_prefill_e4m3", "op": "write", "tokens": 16001, "heads": 8, "dim": 128, "page": 32, "input": "bf16", "cache": "e4m3"},
        # one request, short context: latency
        {"name": "attn_one_short", "op": "attn", "requests": 1, "empty": 0, "min_len": 700, "max_len": 700, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "cache": "bf16", "window": 0},
        # a full decode batch, ragged lengths, two requests without context
        {"name": "attn_batch", "op": "attn", "requests": 128, "empty": 2, "min_len": 1, "max_len": 8191, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "cache": "bf16", "window": 0},
        # few requests, long context, 8-bit cache, 16 query heads per key head
        {"name": "attn_long_e4m3", "op": "attn", "requests": 4, "empty": 0, "min_len": 90001, "max_len": 131000, "q_heads": 64, "kv_heads": 4, "dim": 128, "page": 64, "cache": "e4m3", "window": 0},
        # wide heads under a sliding window
        {"name": "attn_window_256", "op": "attn", "requests": 24, "empty": 0, "min_len": 100, "max_len": 9000, "q_heads": 24, "kv_heads": 4, "dim": 256, "page": 32, "cache": "bf16", "window": 4096},
        # the norm before a projection of a small decode batch, input from the fp32 projection
        {"name": "norm_decode", "op": "norm", "rows": 8, "hidden": 5120, "input": "fp32", "residual": "bf16", "output": "bf16"},
        # a prefill block for an 8-bit product
        {"name": "norm_prefill_e4m3", "op": "norm", "rows": 8191, "hidden": 5120, "input": "bf16", "residual": "bf16", "output": "e4m3"},
        # one request's next token
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 32000, "input": "fp32", "mode": "filtered"},
        # a decode batch with every kind of request in it
        {"name": "sample_batch", "op": "sample", "rows": 256, "vocab": 131072, "input": "fp32", "mode": "mixed"},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["plan", "write", "attn", "attn", "attn", "norm", "sample", "sample"])
    if op == "plan":
        requests = _log_int(rng, 1, 1000)
        chunked, finished = rng.randint(0, min(40, requests)), rng.randint(0, requests // 8)
        return {"op": op, "requests": requests, "max_len": _log_int(rng, 50, 16000), "page": rng.choice([16, 32, 64, 128]), "chunk": rng.randint(1, 900),
                "chunked": min(chunked, requests - finished), "finished": finished}
    if op == "write":
        return {"op": op, "tokens": _log_int(rng, 1, 12000), "heads": rng.choice([1, 2, 4, 5, 8]), "dim": rng.choice([64, 128, 256]) if rng.random() < 0.5 else 128, "page": rng.choice([16, 32, 64, 128]),
                "input": rng.choice(["bf16", "fp32"]), "cache": rng.choice(["bf16", "e4m3"])}
    if op == "attn":
        dim, kv_heads, cache = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice(["bf16", "e4m3"])
        budget = 1.0e9 / (2 * SIZE[cache] * dim * kv_heads)  # tokens in all
        requests = _log_int(rng, 1, 128)
        max_len = _log_int(rng, 1, max(2, min(131072, budget / requests)))
        return {"op": op, "requests": requests, "empty": rng.choice([0, 0, 1]) if requests > 1 else 0, "min_len": rng.randint(1, max_len), "max_len": max_len, "q_heads": kv_heads * rng.choice([1, 2, 3, 4, 6, 8, 12, 16]),
                "kv_heads": kv_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128]), "cache": cache, "window": rng.choice([0, 0, 0, _log_int(rng, 1, 8192)])}
    if op == "norm":
        hidden = rng.choice([256, 1024, 4096, 5120, 8 * rng.randint(1, 380), 16384, 17408])
        return {"op": op, "rows": _log_int(rng, 1, max(2, 40000000 // max(hidden, 5120))), "hidden": hidden, "input": rng.choice(["bf16", "fp32"]),
                "residual": rng.choice(["bf16", "fp32", "none"]), "output": rng.choice(["bf16", "e4m3"])}
    vocab = rng.choice([_log_int(rng, 100, 131072), 32000, 65536, 100003, 131072])
    return {"op": op, "rows": _log_int(rng, 1, min(256, 33000000 // vocab)), "vocab": vocab, "input": rng.choice(["bf16", "fp32"]), "mode": rng.choice(["mixed", "filtered", "plain"])}


# ------------------------------------------------------------------------------------------ inputs


def _spread(count, low, high):
    """`count` whole numbers spread evenly over low..high, the same ones every time."""
    return [low + int((high - low) * ((i + 1) * 0.6180339887498949 % 1.0) + 0.5) for i in range(count)]


def _lengths(case):
    n = case["requests"] - case["empty"]
    return [0] * case["empty"] + ([case["max_len"]] + _spread(n - 1, case["min_len"], case["max_len"]) if n else [])


def _plan_numbers(case):
    """(lengths, added tokens): -1 for a finished request."""
    n = case["requests"]
    add = [-1] * case["finished"] + [case["chunk"] + i % 17 for i in range(case["chunked"])] + [1] * (n - case["finished"] - case["chunked"])
    return _spread(n, 1, case["max_len"]), add


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rand(g, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16 if dtype == torch.bfloat16 else torch.float32, device=DEV).normal_(generator=g)
    return x.mul_(scale).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    return {"plan": _prepare_plan, "write": _prepare_write, "attn": _prepare_attn, "norm": _prepare_norm, "sample": _prepare_sample}[case["op"]](case, _gen(seed))


def _prepare_plan(case, g):
    lens, add = _plan_numbers(case)
    n, page = case["requests"], case["page"]
    order = torch.randperm(n, generator=g, device=DEV)
    lens, add = _ints(lens)[order].contiguous(), _ints(add)[order].contiguous()
    width = -(-(case["max_len"] + case["chunk"] + 17) // page)
    pages = n * width
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    have = torch.div(lens + page - 1, page, rounding_mode="floor")
    used = torch.arange(width, device=DEV)[None, :] < have[:, None]
    rank = torch.cumsum(used.flatten(), 0).view(n, width) - 1
    table = torch.where(used, ids[rank.clamp(min=0)], torch.full_like(rank, -1, dtype=torch.int32)).contiguous()
    held = int(used.sum())
    count = pages - held
    head = pages // 3
    pool = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    pool[(head + torch.arange(count, device=DEV)) % pages] = ids[held:]
    slots = int(add.clamp(min=0).sum()) + 5  # a slot map a little longer than the step needs
    return dict(case, lens=lens, add=add, table=table, pool=pool, state=_ints([head, count]), slots=slots)


def _prepare_write(case, g):
    t, h, d, page = case["tokens"], case["heads"], case["dim"], case["page"]
    pages = -(-2 * t // page) + 1
    # keys and values of one fused projection: a row of the step's output holds both
    kv = _rand(g, (t, 2, h, d), TYPES[case["input"]], 2.0)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:t].to(torch.int32)
    if t > 3:
        slots[torch.randint(0, t, (t // 50 + 1,), generator=g, device=DEV)] = -1  # padding tokens
    s = dict(case, k=kv[:, 0], v=kv[:, 1], slots=slots, pages=pages)
    for name in ("k", "v"):
        # one page more than the calls are given: the plain form drops padding tokens there
        s[name + "_cache"] = torch.zeros((pages + 1, h, page, d), dtype=TYPES[case["cache"]], device=DEV)
        s[name + "_scale"] = torch.zeros((pages + 1, h, page), dtype=torch.float32, device=DEV) if case["cache"] == "e4m3" else None
    return s


def _prepare_attn(case, g):
    n, page, h, d = case["requests"], case["page"], case["kv_heads"], case["dim"]
    order = torch.randperm(n, generator=g, device=DEV)
    lens = _ints(_lengths(case))[order].contiguous()
    width = -(-case["max_len"] // page) + 1
    have = torch.div(lens + page - 1, page, rounding_mode="floor")
    used = torch.arange(width, device=DEV)[None, :] < have[:, None]
    rank = torch.cumsum(used.flatten(), 0).view(n, width) - 1
    pages = sum(-(-v // page) for v in _lengths(case)) + 1
    ids = (torch.randperm(pages - 1, generator=g, device=DEV) + 1).to(torch.int32)
    # page 0 is nobody's: rows past a request's pages point at it
    table = torch.where(used, ids[rank.clamp(min=0).clamp(max=max(pages - 2, 0))] if pages > 1 else torch.zeros_like(rank, dtype=torch.int32), torch.zeros_like(rank, dtype=torch.int32)).contiguous()
    s = dict(case, lens=lens, table=table, softmax_scale=1.0 / math.sqrt(d))
    s["q"] = _rand(g, (n, case["q_heads"], d), torch.bfloat16, 1.5)
    # what no request has written yet: the rest of a last page, and page 0
    last = table.gather(1, (have - 1).clamp(min=0)[:, None].long()).long()
    at = torch.arange(page, device=DEV)[None, :]
    stale = ((have[:, None] - 1) * page + at >= lens[:, None]) & (lens[:, None] > 0)
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


def _prepare_norm(case, g):
    m, h = case["rows"], case["hidden"]
    x = _rand(g, (m, h), TYPES[case["input"]], 0.7)
    res = None if case["residual"] == "none" else _rand(g, (m, h), TYPES[case["residual"]], 3.0)
    gamma = _rand(g, (h,), torch.float32, 0.1) + 1.0
    return dict(case, x=x, res=res, gamma=gamma, eps=1e-6)


def _prepare_sample(case, g):
    b, v = case["rows"], case["vocab"]
    logits = _rand(g, (b, v), torch.float32, 2.5)
    # a few likely tokens in each row, as a language model gives them
    likely = torch.randint(0, v, (b, 40), generator=g, device=DEV)
    lift = torch.empty((b, 40), device=DEV).exponential_(0.25, generator=g)
    logits.scatter_add_(1, likely, lift.clamp(max=16.0))
    row = torch.arange(b, device=DEV)
    pick = lambda values, kind: torch.tensor(values, device=DEV, dtype=kind)[torch.randint(0, len(values), (b,), generator=g, device=DEV)]  # noqa: E731
    if case["mode"] == "plain":  # temperature alone
        t, k, p, m = pick([0.7, 1.0, 1.5], torch.float32), pick([0], torch.int32), pick([1.0], torch.float32), pick([0.0], torch.float32)
    elif case["mode"] == "filtered":
        t, k, p, m = pick([0.6, 0.8, 1.0], torch.float32), pick([20, 50], torch.int32), pick([0.9, 0.95], torch.float32), pick([0.0, 0.05], torch.float32)
    else:
        t, k = pick([0.0, 0.6, 0.8, 1.0, 1.4], torch.float32), pick([0, 1, 40, 1000], torch.int32)
        p, m = pick([1.0, 0.95, 0.9, 0.5], torch.float32), pick([0.0, 0.0, 0.02, 0.1], torch.float32)
        logits[row % 5 == 3, : v // 2] = -math.inf  # a grammar that forbids half of the tokens
    u = torch.empty(b, device=DEV).uniform_(0.0, 1.0, generator=g).clamp_(max=1.0 - 2.0 ** -24)
    return dict(case, logits=logits.to(TYPES[case["input"]]), t=t, k=k, p=p, m=m, u=u)


# ------------------------------------------------------------------------------------------ the passes


def run(s):
    return {"plan": _run_plan, "write": _run_write, "attn": _run_attn, "norm": _run_norm, "sample": _run_sample}[s["op"]](s)


def _run_plan(s):
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        lens, cu, slots, pos, status, state = q4k.q4k_kv_plan(s["lens"], s["add"], s["table"], s["pool"], s["state"], s["page"], s["slots"])
        return {"lens": lens, "cu": cu, "slots": slots, "pos": pos, "status": status, "state": state, "table": s["table"], "pool": s["pool"]}
    page, cap, table, pool = s["page"], s["slots"], s["table"], s["pool"]
    n, width, total = table.shape[0], table.shape[1], pool.numel()
    lens, add = s["lens"].long(), s["add"].long()
    head, count = s["state"][0].long() % total, s["state"][1].long().clamp(0, total)
    done = add == -1
    more = add.clamp(min=0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(more, 0)])
    bad = (lens < 0) | (add < -1) | (lens + more > width * page)
    long = ~bad & ~done & (cu[1:] > cap) & (more > 0)
    have = (lens.clamp(min=0) + page - 1) // page
    need = torch.where(bad | done | long, torch.zeros_like(have), (lens + more + page - 1) // page - have)
    upto = torch.cumsum(need, 0)
    short = (need > 0) & (upto > count)
    granted = ~bad & ~long & ~short & ~done
    status = torch.where(bad, 2, torch.where(long, 3, torch.where(short, 1, 0))).to(torch.int32)
    lens_out = torch.where(granted, lens + more, torch.where(done & ~bad, torch.zeros_like(lens), lens)).to(torch.int32)
    # pages: from the ring's head to the requests, from finished requests to its tail
    col = torch.arange(width, device=DEV)[None, :]
    fresh = granted[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    ring = (head + (upto - need - have)[:, None] + col) % total
    back = torch.where(done & ~bad, have, torch.zeros_like(have))
    first = torch.cumsum(back, 0) - back
    place = first[:, None] + col
    returned = (col < back[:, None]) & (place < total - count)
    larger = torch.cat([pool, pool.new_zeros(1)])
    larger[torch.where(returned, (head + count + place) % total, torch.full_like(place, total)).flatten()] = table.flatten()
    table.copy_(torch.where(fresh, pool[ring], table))
    pool.copy_(larger[:total])
    taken = torch.where(granted, need, torch.zeros_like(need)).sum()
    state = torch.stack([(head + taken) % total, count - taken + torch.minimum(back.sum(), total - count)]).to(torch.int32)
    # tokens
    at = torch.arange(cap, device=DEV)
    who = torch.searchsorted(cu[1:].contiguous(), at, right=True).clamp(max=n - 1)
    live = (at < cu[-1]) & granted[who]
    pos = torch.where(live, lens[who] + at - cu[who], torch.zeros_like(at))
    slot = table[who, pos // page].long() * page + pos % page
    none = torch.full_like(pos, -1)
    return {"lens": lens_out, "cu": cu, "slots": torch.where(live, slot, none).to(torch.int32), "pos": torch.where(live, pos, none).to(torch.int32), "status": status, "state": state, "table": table,
            "pool": pool}


def _run_write(s):
    n = s["pages"]
    out = [s[k][:n] for k in ("k_cache", "v_cache", "k_scale", "v_scale") if s[k] is not None]
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        q4k.q4k_kv_write(s["k"], s["v"], s["slots"], *out)
        return out
    page = s["page"]
    slots = torch.where(s["slots"] < 0, torch.full_like(s["slots"], n * page), s["slots"]).long()
    at, off = slots // page, slots % page
    _plain_store(s["k"], s["k_cache"], s["k_scale"], at, off)
    _plain_store(s["v"], s["v_cache"], s["v_scale"], at, off)
    return out


def _plain_store(x, cache, scales, at, off):
    x = x.float()
    if scales is None:
        cache[at, :, off] = x.to(cache.dtype)
        return
    amax = x.abs().amax(-1).clamp(min=AMAX_FLOOR)
    scales[at, :, off] = amax / 448.0
    cache.view(torch.uint8)[at, :, off] = (x * (448.0 / amax)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _run_attn(s):
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        return q4k.q4k_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["softmax_scale"], s["k_scale"], s["v_scale"], window=s["window"])
    n, hq, d = s["q"].shape
    h, page = s["kv_heads"], s["page"]
    table = s["table"].long()
    at = torch.arange(table.shape[1] * page, device=DEV)[None, :]
    lens = s["lens"].long()[:, None]
    seen = (at < lens) & ((at >= lens - s["window"]) if s["window"] else True)  # [requests, tokens]
    k, v = _plain_rows(s["k_cache"], s["k_scale"], table, seen), _plain_rows(s["v_cache"], s["v_scale"], table, seen)
    q = s["q"].float().view(n, h, hq // h, d)
    score = torch.matmul(q, k.transpose(2, 3)) * s["softmax_scale"]
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight, v) / torch.where(total > 0, total, torch.ones_like(total))
    return out.reshape(n, hq, d).to(torch.bfloat16), (top + torch.log(total)).reshape(n, hq)


def _plain_rows(cache, scales, table, seen):
    """[requests, heads, tokens, dim] fp32 of the cache rows that a table lists; zeros where nothing is seen."""
    x = cache.view(torch.uint8)[table].view(cache.dtype).float() if scales is not None else cache[table].float()
    if scales is not None:
        x = x * scales[table][..., None]
    n, width, h, page, d = x.shape
    x = x.permute(0, 2, 1, 3, 4).reshape(n, h, width * page, d)
    return x.masked_fill_(~seen[:, None, :, None], 0.0)


def _run_norm(s):
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        return q4k.q4k_add_rmsnorm(s["x"], s["res"], s["gamma"], s["eps"], out_dtype=TYPES[s["output"]])
    h = s["x"].float() + (0.0 if s["res"] is None else s["res"].float())
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["gamma"]
    res = (None,) if s["res"] is None else (h.to(s["res"].dtype),)
    if s["output"] == "bf16":
        return (y.to(torch.bfloat16),) + res
    m, n = y.shape
    blocks = -(-n // 128)
    wide = torch.zeros((m, blocks * 128), device=DEV)
    wide[:, :n] = y
    amax = wide.view(m, blocks, 128).abs().amax(-1).clamp(min=AMAX_FLOOR)
    q = (wide.view(m, blocks, 128) * (448.0 / amax)[..., None]).view(m, blocks * 128)[:, :n]
    return (q.to(torch.float8_e4m3fn),) + res + (amax / 448.0,)


def _run_sample(s):
    if own:
        import bit_block_quantized_q4_gb300 as q4k
        return q4k.q4k_sample(s["logits"], s["u"], s["t"], s["k"], s["p"], s["m"])
    x = s["logits"].double()
    b, v = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x)
    high = x.max(-1, keepdim=True).values
    greedy = ~(s["t"] > 0)[:, None]
    t = torch.where(greedy, 1.0, s["t"].double()[:, None])
    weight = torch.where(x == -math.inf, 0.0, torch.where(x == high, 1.0, torch.exp((x - high) / t)))
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    ranked = weight.gather(1, order)
    rank = torch.arange(v, device=DEV)[None, :]
    k = torch.where((s["k"] <= 0) | (s["k"] > v), v, s["k"])[:, None]
    kept = rank < torch.where(greedy, 1, k)
    ranked = torch.where(kept, ranked, 0.0)
    before = torch.cumsum(ranked, -1) - ranked
    p = s["p"].double()[:, None]
    kept &= (p >= 1) | torch.isnan(p) | (before < p * ranked.sum(-1, keepdim=True)) | (rank == 0)
    m = s["m"].double()[:, None]
    kept &= ~(m > 0) | (ranked >= m.clamp(max=1.0))
    weight = torch.zeros_like(weight).scatter_(1, order, torch.where(kept, ranked, 0.0))
    upto = torch.cumsum(weight, -1)
    total = upto[:, -1:]
    token = (upto <= s["u"].double()[:, None] * total).sum(-1).clamp(max=v - 1)
    logp = torch.log(weight.gather(1, token[:, None]) / total)[:, 0]
    none = high[:, 0] == -math.inf
    return torch.where(none, -1, token).to(torch.int32), torch.where(none, -math.inf, logp).float()


# ------------------------------------------------------------------------------------------ work and exact results


def work(case):
    op = case["op"]
    if op == "plan":
        lens, add = _plan_numbers(case)
        n, page = len(lens), case["page"]
        fresh = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, add) if b > 0)
        back = sum(-(-a // page) for a, b in zip(lens, add) if b < 0)
        tokens = sum(max(b, 0) for b in add)
        return {"bytes": n * (4 + 4 + 4 + 8 + 4) + 8 * (fresh + back) + 8 * tokens + 16, "flops": 0}
    if op == "write":
        rows = 2 * case["tokens"] * case["heads"]
        return {"bytes": rows * (case["dim"] * (SIZE[case["input"]] + SIZE[case["cache"]]) + (4 if case["cache"] == "e4m3" else 0)) + 4 * case["tokens"], "flops": 0}
    if op == "attn":
        tokens = sum(min(v, case["window"]) if case["window"] else v for v in _lengths(case))
        row = case["dim"] * SIZE[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)
        q = case["requests"] * case["q_heads"]
        return {"bytes": 2 * tokens * case["kv_heads"] * row + q * (4 * case["dim"] + 4) + 4 * tokens // case["page"], "flops": 4.0 * tokens * case["q_heads"] * case["dim"]}
    if op == "norm":
        res = 0 if case["residual"] == "none" else 2 * SIZE[case["residual"]]
        scales = 4 * -(-case["hidden"] // 128) if case["output"] == "e4m3" else 0
        return {"bytes": case["rows"] * (case["hidden"] * (SIZE[case["input"]] + res + SIZE[case["output"]]) + scales) + 4 * case["hidden"], "flops": 5.0 * case["rows"] * case["hidden"]}
    return {"bytes": case["rows"] * (case["vocab"] * SIZE[case["input"]] + 28), "flops": 10.0 * case["rows"] * case["vocab"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": lambda s: None, "write": _exact_write, "attn": _exact_attn, "norm": _exact_norm, "sample": _exact_sample}[case["op"]](s)


def _exact_write(s):
    caches, scales = [], []
    live = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][live].long()
    for name in ("k", "v"):
        x = s[name][live].double()
        cache = torch.zeros(s[name + "_cache"][: s["pages"]].shape, dtype=torch.float64, device=DEV)
        rows = cache.permute(0, 2, 1, 3).reshape(-1, s["heads"], s["dim"])
        if s["cache"] == "e4m3":
            step = x.abs().max(-1, keepdim=True).values.clamp(min=AMAX_FLOOR) / 448
            x = x / step
            scale = torch.zeros((s["pages"] * s["page"], s["heads"]), dtype=torch.float64, device=DEV)
            scale[slot] = step[..., 0]
            scales.append(scale.view(s["pages"], s["page"], s["heads"]).permute(0, 2, 1).contiguous())
        rows[slot] = x
        caches.append(rows.view(s["pages"], s["page"], s["heads"], s["dim"]).permute(0, 2, 1, 3).contiguous())
    return caches + scales


def _exact_attn(s):
    n, hq, d = s["q"].shape
    group, page = hq // s["kv_heads"], s["page"]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=DEV)
    for r, length in enumerate(s["lens"].tolist()):
        if not length:
            continue
        start = max(0, length - s["window"]) if s["window"] else 0
        pages = s["table"][r, start // page:-(-length // page)].long()
        part = slice(start % page, start % page + length - start)
        rows = []
        for name in ("k", "v"):
            x = (s[name + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn) if s["cache"] == "e4m3" else s[name + "_cache"][pages]).double()
            if s["cache"] == "e4m3":
                x *= s[name + "_scale"][pages].double().unsqueeze(-1)
            rows.append(x.transpose(0, 1).flatten(1, 2)[:, part])  # [heads, tokens, dim]
        for j in range(s["kv_heads"]):
            z = s["softmax_scale"] * (s["q"][r, j * group:(j + 1) * group].double() @ rows[0][j].T)
            norm = torch.logsumexp(z, 1)
            lse[r, j * group:(j + 1) * group] = norm
            out[r, j * group:(j + 1) * group] = torch.exp(z - norm[:, None]) @ rows[1][j]
    return out, lse


def _exact_norm(s):
    h = s["x"].double()
    if s["res"] is not None:
        h = h + s["res"].double()
    y = s["gamma"].double() * h / torch.sqrt(h.square().sum(1, keepdim=True) / h.shape[1] + s["eps"])
    res = [None if s["res"] is None else h]
    if s["output"] == "bf16":
        return tuple([y] + res)
    scales = torch.stack([b.abs().max(1).values for b in y.split(128, 1)], 1).clamp(min=AMAX_FLOOR) / 448
    return tuple([y / scales.repeat_interleave(128, 1)[:, : y.shape[1]]] + res + [scales])


def _exact_sample(s):
    logp = []
    for r in range(s["rows"]):
        x = s["logits"][r].double()
        x = torch.where(torch.isnan(x), -math.inf, x)
        high, t = x.max(), float(s["t"][r])
        if high == -math.inf:
            logp.append(high)
            continue
        if not t > 0:
            logp.append(torch.zeros_like(high))
            continue
        z = (x - high) / t
        z, at = torch.sort(z, descending=True, stable=True)
        k = int(s["k"][r])
        n = k if 0 < k < len(z) else len(z)
        e = torch.exp(z[:n])
        c = torch.cumsum(e, 0)
        p, m = float(s["p"][r]), float(s["m"][r])
        if p < 1:
            n = min(n, max(1, int(((c - e) < p * c[-1]).sum())))
        if m > 0:
            n = min(n, int((e >= min(m, 1.0)).sum()))
        place, back = torch.sort(at[:n])
        walk = torch.cumsum(e[:n][back], 0)
        j = min(int((walk <= float(s["u"][r]) * walk[-1]).sum()), n - 1)
        logp.append(z[back[j]] - torch.log(walk[-1]))
    return None, torch.stack(logp)
