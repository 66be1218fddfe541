"""The operators around the projections against plain 64-bit forms: cache plan and write, paged attention,
residual RMS norm and sampling.

Tolerances count roundings: half a step of a type is eps / 2 relative (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4).
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from _gpu import DEV

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BAD_PAGE = 4
H16, H8, H32, HB = 2.0 ** -11, 2.0 ** -4, 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def q4k():
    from bit_block_quantized_q4_gb300 import build
    build.build()
    import bit_block_quantized_q4_gb300 as m
    assert m.q4k_get_device_error() == 0
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------------------ plan


def plain_plan(lens, add, table, pool, state, page, n_slots):
    """The definition, one request after the other."""
    lens, add, table, pool = lens.tolist(), add.tolist(), table.copy(), pool.copy()
    n, width, size = len(lens), table.shape[1], len(pool)
    head, count = int(state[0]) % size, min(max(int(state[1]), 0), size)
    old, ring = table.copy(), pool.copy()
    cu, status, out = [0], [], []
    slots, pos = np.full(n_slots, -1, np.int32), np.full(n_slots, -1, np.int32)
    asked = taken = given = 0
    flagged = False
    for r in range(n):
        more = max(add[r], 0)
        cu.append(cu[-1] + more)
        if lens[r] < 0 or add[r] < -1 or lens[r] + more > width * page:
            status.append(2), out.append(lens[r])
            continue
        have = -(-lens[r] // page)
        if add[r] == -1:
            for j in range(have):
                if given + j < size - count:
                    pool[(head + count + given + j) % size] = old[r, j]
                else:
                    flagged = True
            given += have
            status.append(0), out.append(0)
            continue
        if more and cu[-1] > n_slots:
            status.append(3), out.append(lens[r])
            continue
        need = -(-(lens[r] + more) // page) - have
        asked += need
        if need and asked > count:
            status.append(1), out.append(lens[r])
            continue
        for j in range(need):
            table[r, have + j] = ring[(head + asked - need + j) % size]
        taken += need
        status.append(0), out.append(lens[r] + more)
        for i in range(more):
            p = lens[r] + i
            pos[cu[r] + i] = p
            pg = table[r, p // page]
            if 0 <= pg < size:
                slots[cu[r] + i] = pg * page + p % page
            else:
                flagged = True
    return (np.array(out), np.array(cu), slots, pos, np.array(status), np.array([(head + taken) % size, count - taken + min(given, size - count)]),
            table, pool, flagged)


def make_plan(seed, n, page, width, scarce, finished, chunk):
    rng = np.random.RandomState(seed)
    lens = rng.randint(0, width * page * 3 // 4 + 1, n)
    add = np.where(rng.rand(n) < 0.2, rng.randint(0, chunk + 1, n), 1)
    add = np.minimum(add, width * page - lens)
    add[rng.rand(n) < finished] = -1
    have = -(-lens // page)
    size = int(have.sum()) + (max(1, n // 12) if scarce else n * width)
    ids = rng.permutation(size)
    table = np.full((n, width), -1, np.int32)
    at = 0
    for r in range(n):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    head = rng.randint(0, size)
    pool = np.full(size, -1, np.int32)
    pool[(head + np.arange(size - at)) % size] = ids[at:]
    return lens.astype(np.int32), add.astype(np.int32), table, pool, np.array([head, size - at], np.int32)


def run_plan(q4k, lens, add, table, pool, state, page, n_slots, pad=0, **kw):
    wide = torch.full((table.shape[0], table.shape[1] + pad), -7, dtype=torch.int32)
    wide[:, :table.shape[1]] = torch.from_numpy(table)
    wide = wide.to(DEV)
    t, p = wide[:, :table.shape[1]], torch.from_numpy(pool).to(DEV)
    got = q4k.q4k_kv_plan(torch.from_numpy(lens).to(DEV), torch.from_numpy(add).to(DEV), t, p, torch.from_numpy(state).to(DEV), page, n_slots, **kw)
    assert pad == 0 or bool((wide[:, table.shape[1]:] == -7).all())
    return [x.cpu().numpy() for x in got] + [t.cpu().numpy(), p.cpu().numpy()]


@pytest.mark.parametrize("seed,n,page,width,scarce,finished,chunk,slack,pad", [
    (1, 1, 16, 4, False, 0.0, 1, 0, 0), (2, 33, 16, 9, False, 0.2, 40, 5, 3), (3, 33, 16, 9, True, 0.2, 40, 5, 0), (4, 300, 1, 37, False, 0.1, 20, 0, 1),
    (5, 1025, 16, 12, True, 0.1, 90, -200, 0), (6, 2500, 64, 5, False, 0.5, 200, 9000, 0), (7, 700, 7, 30, True, 0.0, 150, -1000, 0), (8, 64, 16, 8, False, 1.0, 1, 3, 0),
    (9, 40, 32, 600, False, 0.1, 15000, 0, 0)])
def test_plan_matches_the_definition(q4k, seed, n, page, width, scarce, finished, chunk, slack, pad):
    lens, add, table, pool, state = make_plan(seed, n, page, width, scarce, finished, chunk)
    n_slots = max(0, int(np.maximum(add, 0).sum()) + slack)
    want = plain_plan(lens, add, table, pool, state, page, n_slots)
    got = run_plan(q4k, lens, add, table, pool, state, page, n_slots, pad)
    for name, g, w in zip(("lens", "cu", "slots", "pos", "status", "state", "table", "pool"), got, want):
        assert np.array_equal(g, w), name
    assert q4k.q4k_get_device_error() == (BAD_PAGE if want[-1] else 0)
    if scarce:
        assert (want[4] == 1).any()


def test_plan_bad_lengths_bad_pages_and_pages_returned_twice(q4k):
    page, width = 16, 4
    lens = np.array([-1, 65, 60, 10, 2 ** 31 - 1, 20, 64, 0, 5], np.int32)
    add = np.array([1, 1, 5, -2, 1, -1, 0, 3, 2 ** 31 - 1], np.int32)
    table = np.full((9, width), 3, np.int32)
    table[6] = [0, 1, 99, -4]
    for count, pool in ((0, [2, 1, 0, 3]), (4, [9, -1, 0, 3])):  # with 4 of 4 free, the two returned pages have no place
        state = np.array([1, count], np.int32)
        pool = np.array(pool, np.int32)
        want = plain_plan(lens, add, table, pool, state, page, 20)
        got = run_plan(q4k, lens, add, table, pool, state, page, 20)
        for g, w in zip(got, want):
            assert np.array_equal(g, w)
        assert q4k.q4k_get_device_error() == (BAD_PAGE if want[-1] else 0)
        assert want[-1] == (count == 4)
    # a head and a count outside the ring are brought into it
    state = np.array([-5, 77], np.int32)
    want = plain_plan(lens, add, table, pool, state, page, 20)
    got = run_plan(q4k, lens, add, table, pool, state, page, 20)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    q4k.q4k_get_device_error()


def test_plan_in_place_over_steps_and_pages_come_back(q4k):
    n, page, width = 1500, 16, 8
    rng = np.random.RandomState(3)
    size = 1800
    lens, table = np.zeros(n, np.int32), np.full((n, width), -1, np.int32)
    pool, state = rng.permutation(size).astype(np.int32), np.array([0, size], np.int32)
    d = {k: torch.from_numpy(v).to(DEV) for k, v in dict(lens=lens, table=table, pool=pool, state=state).items()}
    for step in range(6):
        add = rng.randint(0, 20, n).astype(np.int32)
        add[rng.rand(n) < 0.3] = -1
        n_slots = int(np.maximum(add, 0).sum())
        o = [torch.empty(k, dtype=t, device=DEV) for k, t in ((n + 1, torch.int64), (n_slots, torch.int32), (n_slots, torch.int32), (n, torch.int32))]
        q4k.q4k_kv_plan(d["lens"], torch.from_numpy(add).to(DEV), d["table"], d["pool"], d["state"], page, n_slots, out=(d["lens"], *o, d["state"]))
        want = plain_plan(lens, add, table, pool, state, page, n_slots)
        lens, state, table, pool = want[0].astype(np.int32), want[5].astype(np.int32), want[6], want[7]
        for g, w in zip((d["lens"], *o, d["state"], d["table"], d["pool"]), want):
            assert np.array_equal(g.cpu().numpy(), w), step
        used = [p for r in range(n) for p in table[r, :-(-int(lens[r]) // page)]]
        free = [pool[(state[0] + i) % size] for i in range(state[1])]
        assert sorted(used + free) == list(range(size))  # no page lost, none twice
    assert q4k.q4k_get_device_error() == 0


# ------------------------------------------------------------------------------------------ write


def cache_of(pages, heads, page, dim, kind, layout, fill=None):
    """A cache buffer [pages, heads, page, dim] in one of three layouts."""
    t = torch.uint8 if kind == E4M3 else kind
    if layout == "head-major":
        x = torch.zeros((pages, heads, page, dim), dtype=t)
    elif layout == "token-major":
        x = torch.zeros((pages, page, heads, dim), dtype=t).transpose(1, 2)
    else:  # K and V rows side by side, a page longer than it needs to be
        x = torch.zeros((pages, heads, page + 1, 2 * dim), dtype=t)[:, :, :page, :dim]
    return x


def to_dev(x, kind=None):
    """The same strides on the GPU."""
    base = x
    storage = torch.empty_strided(base.shape, base.stride(), dtype=base.dtype, device=DEV)
    storage.copy_(base)
    return storage.view(E4M3) if kind == E4M3 else storage


def quantize(x):
    """e4m3 rows with a scale, by the formula: (bytes, scales)."""
    amax = x.float().abs().amax(-1).clamp(min=2.0 ** -100)
    inv = torch.full_like(amax, 448.0) / amax  # one division: 448.0 / amax is a reciprocal and a product in torch
    return (x.float() * inv[..., None]).to(E4M3).view(torch.uint8), amax / 448.0


@pytest.mark.parametrize("layout", ["head-major", "token-major", "padded"])
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("tokens,heads,dim,page,src", [(1, 1, 64, 16, F32), (37, 3, 128, 16, BF16), (130, 8, 256, 32, F32), (5, 5, 64, 1, BF16), (600, 2, 128, 128, F32)])
def test_write(q4k, tokens, heads, dim, page, src, kind, layout):
    g = gen(tokens * 7 + dim)
    pages = 2 * tokens // page + 2
    x = torch.randn((tokens, 2, heads, dim), generator=g) * torch.exp2(torch.randint(-20, 20, (tokens, 2, heads, 1), generator=g).float())
    x[0, 0, 0] = 0.0          # a row of zeros has a scale
    x = x.to(src)
    slots = torch.randperm(pages * page, generator=g)[:tokens].to(torch.int32)
    if tokens > 3:
        slots[2] = -1
    want, scales = [], []
    for kv in range(2):
        c, s = cache_of(pages, heads, page, dim, kind, layout), torch.zeros((pages, heads, page))
        for t in range(tokens):
            if slots[t] >= 0:
                at, off = int(slots[t]) // page, int(slots[t]) % page
                if kind == BF16:
                    c[at, :, off] = x[t, kv].to(BF16)
                else:
                    c[at, :, off], s[at, :, off] = quantize(x[t, kv])
        want.append(c), scales.append(s)
    caches = [to_dev(torch.zeros_like(c) if layout == "head-major" else cache_of(pages, heads, page, dim, kind, layout), kind) for c in want]
    sc = [torch.zeros((pages, heads, page), device=DEV) for _ in range(2)] if kind == E4M3 else []
    xd = x.to(DEV)
    q4k.q4k_kv_write(xd[:, 0], xd[:, 1], slots.to(DEV), *caches, *sc)
    for kv in range(2):
        got = caches[kv].view(torch.uint8).cpu() if kind == E4M3 else caches[kv].cpu()
        assert torch.equal(got, want[kv])      # one rounding, or exact scaling arithmetic: equal bit by bit
        if kind == E4M3:
            assert torch.equal(sc[kv].cpu(), scales[kv])
    assert q4k.q4k_get_device_error() == 0


def test_write_skips_slots_outside_the_cache(q4k):
    k = torch.randn((4, 2, 64), generator=gen(1))
    caches = [torch.zeros((3, 2, 16, 64), dtype=BF16, device=DEV) for _ in range(2)]
    q4k.q4k_kv_write(k.to(DEV), k.to(DEV), torch.tensor([48, 47, -2, 2 ** 31 - 1], dtype=torch.int32, device=DEV), *caches)
    assert q4k.q4k_get_device_error() == BAD_PAGE
    for c in caches:
        assert torch.equal(c[2, :, 15].cpu(), k[1].to(BF16))
        c[2, :, 15] = 0
        assert not c.any()


def test_write_values_that_are_not_finite(q4k):
    k = torch.randn((2, 1, 64), generator=gen(2))
    k[0, 0, 5], k[1, 0, 6] = math.inf, math.nan
    for kind in (BF16, E4M3):
        caches = [torch.zeros((1, 1, 16, 64), dtype=torch.uint8 if kind == E4M3 else kind, device=DEV).view(kind) for _ in range(2)]
        sc = [torch.zeros((1, 1, 16), device=DEV) for _ in range(2)] if kind == E4M3 else []
        q4k.q4k_kv_write(k.to(DEV), k.to(DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV), *caches, *sc)
        row = caches[0][0, 0, :2].float().cpu() * (sc[0][0, 0, :2, None].cpu() if sc else 1.0)
        assert not torch.isfinite(row[0, 5]) and torch.isnan(row[1, 6])


# ------------------------------------------------------------------------------------------ attention


def make_attn(seed, lens, q_heads, kv_heads, dim, page, kind, layout="head-major", spread=1.0, extra=2):
    g = gen(seed)
    n = len(lens)
    width = max(-(-max(max(lens), 1) // page), 1) + extra
    pages = sum(-(-max(v, 0) // page) for v in lens) + 3
    ids = torch.randperm(pages - 1, generator=g) + 1
    table = torch.zeros((n, width), dtype=torch.int32)
    at = 0
    # what no token refers to holds NaN
    caches = [cache_of(pages, kv_heads, page, dim, kind, layout) for _ in range(2)]
    for c in caches:
        c.fill_(0x7F) if kind == E4M3 else c.fill_(math.nan)
    scales = [torch.full((pages, kv_heads, page), math.nan) for _ in range(2)] if kind == E4M3 else None
    dense = []
    for r, length in enumerate(lens):
        m = -(-max(length, 0) // page)
        table[r, :m] = ids[at:at + m].to(torch.int32)
        at += m
        rows = []
        for kv in range(2):
            x = torch.randn((max(length, 0), kv_heads, dim), generator=g) * spread
            if kind == E4M3:
                x = x * torch.exp2(torch.randint(-6, 7, (max(length, 0), kv_heads, 1), generator=g).float()) if kv else x
                b, s = quantize(x)
                x = b.view(E4M3).double() * s.double()[..., None]
            else:
                b = x.to(BF16)
                x = b.double()
            rows.append(x)
            for p in range(m):
                k = min(page, length - p * page)
                caches[kv][table[r, p], :, :k] = b[p * page:p * page + k].transpose(0, 1)
                if kind == E4M3:
                    scales[kv][table[r, p], :, :k] = s[p * page:p * page + k].transpose(0, 1)
        dense.append(rows)
    q = torch.randn((n, q_heads, dim), generator=g).to(BF16)
    return dict(q=q, caches=caches, scales=scales, table=table, lens=torch.tensor(lens, dtype=torch.int32), dense=dense, kind=kind, kv_heads=kv_heads)


def plain_attn(c, scale, window=0, skip=None):
    """(out, lse, bound of out, bound of lse) in 64 bits; skip(r): tokens that count as absent."""
    n, hq, d = c["q"].shape
    group = hq // c["kv_heads"]
    out, lse = torch.zeros((n, hq, d), dtype=torch.float64), torch.full((n, hq), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(n):
        length = max(int(c["lens"][r]), 0)
        keep = torch.arange(length) >= (length - window if window else 0)
        if skip is not None:
            keep &= ~skip(r, length)
        k, v = (x[:length][keep].repeat_interleave(group, 1) for x in c["dense"][r])
        if not len(k):
            continue
        q = c["q"][r].double()
        z = torch.einsum("hd,thd->ht", q, k) * scale
        size = (torch.einsum("hd,thd->ht", q.abs(), k.abs()) * abs(scale)).amax(1)
        top = z.amax(1, keepdim=True)
        e = torch.exp(z - top)
        p = e / e.sum(1, keepdim=True)
        out[r] = torch.einsum("ht,thd->hd", p, v)
        lse[r] = top[:, 0] + torch.log(e.sum(1))
        pv = torch.einsum("ht,thd->hd", p, v.abs())
        # fp32 scores: a product's rounding and d additions of up to `size` each, and the scaling; exp2
        # and its argument: 2^-20 relative; sums of t terms: t roundings; weights: two bf16 terms
        # (2^-16), or one fp16 term (half a step 2^-11, and 2^-25 of the largest weight times scale)
        dz = (d + 8) * H32 * size + 2.0 ** -20 * (1 + z.abs().amax(1) * 2 ** -2)
        rel = 2 * dz + (len(k) ** 0.5 + 40) * H32 * 2 + (2.0 ** -16 if c["kind"] == BF16 else H16)
        bo[r] = HB * out[r].abs() + rel[:, None] * pv * 1.01
        if c["kind"] == E4M3:
            bo[r] += 2.0 ** -25 * len(k) * (p.unsqueeze(-1) * v.transpose(0, 1).abs()).amax((1, 2))[:, None] * 2
        bl[r] = dz + (len(k) ** 0.5 + 40) * H32 * 2 + H32 * lse[r].abs()
    return out, lse, bo, bl


def check_attn(q4k, c, scale, window=0, skip=None, error=0, **kw):
    caches = [to_dev(x, c["kind"]) for x in c["caches"]]
    scales = [s.to(DEV) for s in c["scales"]] if c["scales"] else [None, None]
    out, lse = q4k.q4k_paged_attn(c["q"].to(DEV), *caches, c["table"].to(DEV), c["lens"].to(DEV), scale, *scales, window=window, **kw)
    assert q4k.q4k_get_device_error() == error
    want, wl, bo, bl = plain_attn(c, scale, window, skip)
    off = (out.double().cpu() - want).abs()
    assert bool((off <= bo).all()), (off - bo).max()
    lse = lse.double().cpu()
    assert torch.equal(lse == -math.inf, wl == -math.inf)
    fin = wl != -math.inf
    assert bool(((lse - wl)[fin].abs() <= bl[fin]).all()), ((lse - wl)[fin].abs() - bl[fin]).max()
    return out, lse


LENS = [1, 0, 15, 16, 17, 31, 33, 64, 100, 700, 2, 0]


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads,page", [(1, 1, 16), (8, 8, 32), (12, 4, 16), (16, 2, 64), (7, 1, 128), (32, 2, 16), (20, 1, 256), (51, 3, 32)])
def test_attn(q4k, q_heads, kv_heads, page, dim, kind):
    check_attn(q4k, make_attn(q_heads + dim, LENS, q_heads, kv_heads, dim, page, kind), dim ** -0.5)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 5000])
def test_attn_window(q4k, window, kind):
    check_attn(q4k, make_attn(window, LENS + [1500], 8, 2, 128, 16, kind), 0.1, window)
    check_attn(q4k, make_attn(window, LENS, 6, 2, 64, 128, kind), 0.1, window)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("layout", ["token-major", "padded"])
def test_attn_layouts_and_strides(q4k, layout, kind):
    c = make_attn(5, LENS, 8, 4, 128, 16, kind, layout)
    n = len(LENS)
    out = torch.full((n, 10 * 128), 7.0, dtype=BF16, device=DEV)
    o = out[:, :1024].view(n, 8, 128)
    got, _ = check_attn(q4k, c, 0.09, out=o)
    assert bool((out[:, 1024:] == 7.0).all())
    # q as a part of a fused projection's rows, the table as a part of a wider one
    wide = torch.zeros((n, 3, 16, 128), dtype=BF16)
    wide[:, 1, :16:2] = c["q"]
    table = torch.full((n, 2 * c["table"].shape[1]), 10 ** 6, dtype=torch.int32)
    table[:, :c["table"].shape[1]] = c["table"]
    scales = [s.to(DEV) for s in c["scales"]] if c["scales"] else [None, None]
    again, _ = q4k.q4k_paged_attn(wide.to(DEV)[:, 1, ::2], *[to_dev(x, kind) for x in c["caches"]], table.to(DEV)[:, :c["table"].shape[1]], c["lens"].to(DEV), 0.09, *scales)
    assert torch.equal(again, got)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("order", [(0, 2, 1, 3), (1, 0, 2, 3), (1, 2, 0, 3), (2, 0, 1, 3), (2, 1, 0, 3)])
def test_cache_dimensions_in_any_order(q4k, order, kind):
    """Cache buffers that lie heads first, tokens first and so on: the bits of a head-major one."""
    c = make_attn(17, LENS, 8, 4, 128, 32, kind)
    table, lens, q = c["table"].to(DEV), c["lens"].to(DEV), c["q"].to(DEV)
    scales = [s.to(DEV) for s in c["scales"]] if c["scales"] else []
    back = [order.index(i) for i in range(4)]
    slots = torch.tensor([3, 0, -1, 70, 64], dtype=torch.int32, device=DEV)
    rows = [torch.randn((5, 4, 128), generator=gen(18 + i)).to(DEV) for i in range(2)]

    def both(caches):
        sc = [s.clone() for s in scales]
        caches = [x.view(E4M3) for x in caches] if kind == E4M3 else caches
        first = q4k.q4k_paged_attn(q, *caches, table, lens, 0.09, *sc)
        q4k.q4k_kv_write(*rows, slots, *caches, *sc)
        return first, [x.view(torch.uint8).contiguous() if kind == E4M3 else x.contiguous() for x in caches], sc

    plain = [x.to(DEV) for x in c["caches"]]
    other = [x.permute(order).contiguous().permute(back) for x in plain]
    assert other[0].stride() != plain[0].stride()
    (o0, l0), c0, s0 = both(plain)
    (o1, l1), c1, s1 = both(other)
    assert torch.equal(o0, o1) and torch.equal(l0, l1)
    for x, y in zip(c0 + s0, c1 + s1):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # bytes: unused rows hold NaN
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_attn_long_and_many(q4k, kind):
    check_attn(q4k, make_attn(11, [20011], 16, 2, 128, 64, kind), 0.08)
    check_attn(q4k, make_attn(12, [(i * 37) % 190 for i in range(400)], 4, 2, 64, 16, kind), 0.125)
    check_attn(q4k, make_attn(13, [5000, 0, 1, 3000], 32, 1, 128, 16, kind), 0.08)


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_attn_large_scores(q4k, kind):
    """Scores of some hundreds: the weights of most tokens vanish, one token takes nearly all."""
    check_attn(q4k, make_attn(14, [300, 5, 64], 8, 2, 128, 16, kind, spread=8.0), 1.0)
    check_attn(q4k, make_attn(15, [300, 5, 64], 8, 2, 128, 16, kind, spread=8.0), -1.0)
    check_attn(q4k, make_attn(16, [300, 5, 64], 8, 2, 128, 16, kind), 0.0)


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_attn_pages_outside_the_cache_count_as_absent(q4k, kind):
    lens = [100, 40, 16, 70]
    c = make_attn(17, lens, 8, 2, 128, 16, kind)
    pages = c["caches"][0].shape[0]
    for r, p, bad in ((0, 3, pages), (0, 6, -1), (1, 0, 2 ** 31 - 1), (2, 0, -2 ** 31), (3, 4, 10 ** 6)):
        c["table"][r, p] = bad
    outside = (c["table"] < 0) | (c["table"] >= pages)
    check_attn(q4k, c, 0.1, skip=lambda r, n: outside[r][torch.arange(n) // 16], error=BAD_PAGE)
    # a length past the table: the tokens that the table covers
    c = make_attn(18, [64, 33], 8, 2, 128, 16, kind, extra=0)
    c["lens"][0] = 2 ** 31 - 1
    scales = [s.to(DEV) for s in c["scales"]] if c["scales"] else [None, None]
    out, _ = q4k.q4k_paged_attn(c["q"].to(DEV), *[to_dev(x, kind) for x in c["caches"]], c["table"].to(DEV), c["lens"].to(DEV), 0.1, *scales)
    assert q4k.q4k_get_device_error() == BAD_PAGE
    c["lens"][0] = 64
    want, _, bo, _ = plain_attn(c, 0.1)
    assert bool(((out.double().cpu() - want).abs() <= bo).all())
    # negative lengths are empty
    c["lens"][0] = -3
    check_attn(q4k, c, 0.1)


def test_attn_rows_of_zeros_and_values_that_are_not_finite(q4k):
    """Zero rows of an e4m3 cache have the smallest scale; what is not finite in a row that counts shows."""
    n, h, page, d = 3000, 2, 64, 128
    x = torch.zeros((n, 2, h, d))
    x[:, 0] = torch.randn((n, h, d), generator=gen(1))
    caches = [torch.zeros((n // page + 1, h, page, d), dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    sc = [torch.zeros((n // page + 1, h, page), device=DEV) for _ in range(2)]
    q4k.q4k_kv_write(x[:, 0].to(DEV), x[:, 1].to(DEV), torch.arange(n, dtype=torch.int32, device=DEV), *caches, *sc)
    table = torch.arange(n // page + 1, dtype=torch.int32, device=DEV)[None]
    q = torch.randn((1, 4, d), generator=gen(2)).to(BF16)
    out, lse = q4k.q4k_paged_attn(q.to(DEV), *caches, table, torch.tensor([n], dtype=torch.int32, device=DEV), 0.1, *sc)
    assert not out.any()
    k = caches[0].double().cpu().transpose(1, 2).reshape(-1, h, d)[:n] * sc[0].double().cpu().transpose(1, 2).reshape(-1, h)[:n, :, None]
    want = torch.logsumexp(torch.einsum("hd,thd->ht", q[0].double(), k.repeat_interleave(2, 1)) * 0.1, 1)
    assert bool(((lse[0].double().cpu() - want).abs() <= 2.0 ** -16).all())  # scores of some units in fp32, 3000 terms
    c = make_attn(3, [40, 1, 33, 20], 4, 2, 64, 16, BF16)
    for r, kv, t, v in ((0, 0, 7, math.nan), (1, 0, 0, math.nan), (2, 1, 32, math.inf), (3, 0, 3, -math.inf)):
        c["caches"][kv][c["table"][r, t // 16], 1, t % 16, 5] = v
    out, lse = q4k.q4k_paged_attn(c["q"].to(DEV), *[to_dev(x) for x in c["caches"]], c["table"].to(DEV), c["lens"].to(DEV), 0.1)
    out, lse = out.float().cpu(), lse.cpu()
    assert bool(torch.isfinite(out[:, :2]).all()) and bool(torch.isfinite(lse[:, :2]).all())  # the other key head
    assert bool(torch.isnan(out[:2, 2:]).all()) and bool(torch.isnan(lse[:2, 2:]).all())
    # (an infinite value times a weight in two terms: an infinity or no number, as the header says)
    assert not bool(torch.isfinite(out[2, 2:, 5]).any()) and bool(torch.isfinite(out[2, 2:, :5]).all())
    qk = c["q"][3, 2:, 5].float()  # a score of -inf takes no part, one of +inf leaves no number
    for i in range(2):
        assert bool(torch.isfinite(out[3, 2 + i]).all()) if qk[i] > 0 else bool(torch.isnan(out[3, 2 + i]).all())


def test_attn_offsets_past_32_bits(q4k):
    """A cache of over 2^32 bytes, used at its end."""
    pages, heads, page, dim = 70000, 2, 128, 128
    c = make_attn(19, [300], 8, heads, dim, page, BF16)
    caches = []
    for x in c["caches"]:
        big = torch.empty((pages, heads, page, dim), dtype=BF16, device=DEV)
        big[-x.shape[0]:] = x.to(DEV)
        caches.append(big)
    assert caches[0].numel() > 2 ** 31
    table = c["table"] + (pages - c["caches"][0].shape[0])
    out, _ = q4k.q4k_paged_attn(c["q"].to(DEV), *caches, table.to(DEV), c["lens"].to(DEV), 0.09)
    want, _, bo, _ = plain_attn(c, 0.09)
    assert bool(((out.double().cpu() - want).abs() <= bo).all())
    x = torch.randn((3, heads, dim), generator=gen(3))
    slots = torch.tensor([pages * page - 1, 5, pages * page - page], dtype=torch.int32)
    q4k.q4k_kv_write(x.to(DEV), x.to(DEV), slots.to(DEV), *caches)
    assert torch.equal(caches[1][-1, :, -1].cpu(), x[0].to(BF16)) and torch.equal(caches[0][-1, :, 0].cpu(), x[2].to(BF16))
    assert q4k.q4k_get_device_error() == 0


def test_attn_same_result_every_time_and_on_another_stream(q4k):
    c = make_attn(20, [700, 33, 4000, 1], 16, 2, 128, 16, BF16)
    args = [c["q"].to(DEV), *[to_dev(x) for x in c["caches"]], c["table"].to(DEV), c["lens"].to(DEV), 0.09]
    first = q4k.q4k_paged_attn(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        again = q4k.q4k_paged_attn(*args, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------------------------------ norm


@pytest.mark.parametrize("out", [BF16, E4M3])
@pytest.mark.parametrize("src,res", [(F32, BF16), (BF16, BF16), (BF16, F32), (F32, F32), (BF16, None)])
@pytest.mark.parametrize("m,h", [(1, 8), (3, 128), (5, 136), (2, 1000), (9, 4096), (4, 5120), (3, 8200), (2, 17408), (1, 32768)])
def test_norm(q4k, m, h, src, res, out):
    g = gen(m * h)
    x = (torch.randn((m, h + 8), generator=g) * 3).to(src)[:, :h]
    r = None if res is None else (torch.randn((m, h + 16), generator=g) * 5).to(res)[:, 8:8 + h]
    gamma = 1 + 0.2 * torch.randn(h, generator=g)
    eps = 1e-5
    xd = torch.empty((m, h + 8), dtype=src, device=DEV)[:, :h].copy_(x)
    rd = None if r is None else torch.empty((m, h + 16), dtype=res, device=DEV)[:, 8:8 + h].copy_(r)
    if rd is not None:
        assert rd.data_ptr() % 16 == 0
    got = q4k.q4k_add_rmsnorm(xd, rd, gamma.to(DEV), eps, out_dtype=out)
    hh = x.double() if r is None else x.double() + r.double()
    y = hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + eps) * gamma.double()
    # h: one fp32 rounding; the sum of squares: h / 32 + 12 additions at most in a row, halved by the square
    # root; rsqrt, two products
    rel = (h / 32 + 24) * H32 + 8 * H32
    size = (x.double().abs() + (0 if r is None else r.double().abs())) / torch.sqrt((hh * hh).mean(-1, keepdim=True) + eps) * gamma.double().abs()
    slip = rel * y.abs() + H32 * size
    if res is None:
        assert got[1] is None
    else:
        off = (got[1].double().cpu() - hh).abs()
        assert got[1].dtype == res and bool((off <= (HB if res == BF16 else 0) * hh.abs() * 1.001 + 2 * H32 * (hh.abs() + size * 0)).all())
    if out == BF16:
        assert bool(((got[0].double().cpu() - y).abs() <= HB * y.abs() + 1.01 * slip).all())
        return
    s = got[2].double().cpu()
    assert s.shape == (m, -(-h // 128))
    for b in range(s.shape[1]):
        block, part = y[:, b * 128:(b + 1) * 128], slice(b * 128, (b + 1) * 128)
        want = block.abs().amax(1).clamp(min=2.0 ** -100) / 448
        assert bool(((s[:, b] - want).abs() <= (rel + 4 * H32) * want + H32 * size[:, part].amax(1) / 448).all())
        back = got[0][:, part].double().cpu() * s[:, b, None]
        assert bool(((back - block).abs() <= H8 * block.abs() * 1.001 + 2.0 ** -10 * s[:, b, None] + 1.2 * slip[:, part]).all())


@pytest.mark.parametrize("out", [BF16, E4M3])
@pytest.mark.parametrize("m,h,src,res", [(700, 5120, BF16, BF16), (611, 8200, F32, BF16), (1300, 4104, BF16, None), (650, 17408, BF16, BF16), (640, 16384, F32, F32)])
def test_norm_many_rows(q4k, m, h, src, res, out):
    """More rows than the GPU holds at once, of more values than a block keeps in registers: against the same rows in
    calls of a few."""
    g = torch.Generator(device=DEV).manual_seed(h)
    x = torch.randn((m, h), generator=g, device=DEV).to(src)
    r = None if res is None else torch.randn((m, h), generator=g, device=DEV).to(res)
    gamma = torch.rand(h, generator=g, device=DEV) + 0.5
    got = q4k.q4k_add_rmsnorm(x, r, gamma, 1e-6, out_dtype=out)
    assert q4k.q4k_get_device_error() == 0
    hh = x.double() if r is None else x.double() + r.double()
    y = hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + 1e-6) * gamma.double()
    rel = (h / 32 + 24) * H32 + 8 * H32
    if res is not None:
        size = x.double().abs() + r.double().abs()
        assert bool(((got[1].double() - hh).abs() <= (HB if res == BF16 else 0) * hh.abs() * 1.001 + 2 * H32 * size).all())
    slip = rel * y.abs() + H32 * (x.double().abs() + (0 if r is None else r.double().abs())) / torch.sqrt((hh * hh).mean(-1, keepdim=True) + 1e-6) * gamma.double()
    if out == BF16:
        assert bool(((got[0].double() - y).abs() <= HB * y.abs() + 1.01 * slip).all())
        return
    s = got[2].double().repeat_interleave(128, 1)[:, :h]
    assert bool(((got[0].double() * s - y).abs() <= H8 * y.abs() * 1.001 + 2.0 ** -10 * s + 1.2 * slip).all())
    top = torch.nn.functional.pad(y.abs(), (0, -h % 128)).view(m, -1, 128).amax(-1) / 448
    assert bool(((got[2].double() - top).abs() <= (2 * rel + 16 * H32) * top + 1e-6 * top).all())
    again = q4k.q4k_add_rmsnorm(x[3:9], None if r is None else r[3:9], gamma, 1e-6, out_dtype=out)
    off = (again[0].float() - got[0][3:9].float()).abs()
    assert float((off > 0).float().mean()) < 0.01  # another order of the sums: a rounding here and there


def test_norm_in_place_zero_rows_and_streams(q4k):
    g = gen(9)
    x, r, gamma = torch.randn((6, 512), generator=g), torch.randn((6, 512), generator=g).to(BF16), torch.ones(512)
    x[2], r[2] = 0, 0
    xd, rd, gd = x.to(DEV), r.to(DEV), gamma.to(DEV)
    y, ro = q4k.q4k_add_rmsnorm(xd, rd, gd, 0.0)
    assert bool(torch.isnan(y[2].float()).all())          # 0 / 0 by the formula, with eps 0
    y, ro, s = q4k.q4k_add_rmsnorm(xd, rd, gd, 1e-6, out_dtype=E4M3)
    assert bool((y[2].float() == 0).all()) and bool((s[2] > 0).all()) and bool((ro[2] == 0).all())
    inplace = rd.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2, r2, s2 = q4k.q4k_add_rmsnorm(xd, inplace, gd, 1e-6, out_dtype=E4M3, residual_out=inplace, stream=st)
    torch.cuda.synchronize()
    assert r2 is inplace and torch.equal(inplace, ro) and torch.equal(s, s2) and torch.equal(y.view(torch.uint8), y2.view(torch.uint8))


# ------------------------------------------------------------------------------------------ sampling


def plain_sample(x, u, t, k, p, m):
    """(token, logp, tokens that a draw within 2^-36 of a border may give) in 64 bits."""
    x = x.astype(np.float64)
    x[np.isnan(x)] = -np.inf
    high = x.max()
    if high == -np.inf:
        return -1, -np.inf, {-1}
    if not t > 0:
        return int(x.argmax()), 0.0, {int(x.argmax())}
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(x == high, 1.0, np.where(x == -np.inf, 0.0, np.exp((x - high) / t)))
    order = np.lexsort((np.arange(len(x)), -x))
    kept = order[:k] if 0 < k < len(x) else order
    w = e[kept]
    if p < 1:
        before = np.concatenate([[0], np.cumsum(w)[:-1]])
        n = max(1, int((before < p * w.sum()).sum()))
        kept, w = kept[:n], w[:n]
    if m > 0:
        kept = kept[w >= min(m, 1.0)]
    kept = np.sort(kept)
    c = np.cumsum(e[kept])
    target = min(max(u, 0.0), 1.0) * c[-1]
    live = kept[e[kept] > 0]
    pick = lambda at: int(live[min(int((np.cumsum(e[live]) <= at).sum()), len(live) - 1)])  # noqa: E731
    token = pick(target)
    return token, math.log(e[token] / c[-1]), {token, pick(target - 2.0 ** -36 * c[-1]), pick(target + 2.0 ** -36 * c[-1])}


def check_sample(q4k, x, u, t=None, k=None, p=None, m=None):
    rows = x.shape[0]
    full = lambda v, d: torch.full((rows,), d) if v is None else v  # noqa: E731
    dev = lambda v, kind: None if v is None else v.to(kind).to(DEV)  # noqa: E731
    xd = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEV).copy_(x)
    token, logp = q4k.q4k_sample(xd, u.to(DEV), dev(t, F32), dev(k, torch.int32), dev(p, F32), dev(m, F32))
    token, logp = token.cpu(), logp.cpu().double()
    for r in range(rows):
        want, lp, near = plain_sample(x[r].float().numpy(), float(u[r]), float(full(t, 1.0)[r]), int(full(k, 0)[r]), float(full(p, 1.0)[r]), float(full(m, 0.0)[r]))
        assert int(token[r]) in near, (r, int(token[r]), want)
        if int(token[r]) == want:  # a logarithm in 64 bits of weights held to 2^-40, rounded once
            assert logp[r] == lp or abs(logp[r] - lp) <= H32 * abs(lp) + 2.0 ** -28 / math.exp(max(lp, -25.0)) * 2.0 ** -10 + 2.0 ** -30, (r, logp[r], lp)
    assert q4k.q4k_get_device_error() == 0


def peaked(rows, vocab, seed, sigma=2.5):
    g = gen(seed)
    x = torch.randn((rows, vocab), generator=g) * sigma
    x.scatter_add_(1, torch.randint(0, vocab, (rows, min(30, vocab)), generator=g), torch.rand((rows, min(30, vocab)), generator=g) * 12)
    return x, torch.rand(rows, generator=g)


@pytest.mark.parametrize("vocab", [1, 2, 31, 100, 1023, 4097, 32000, 100003, 131072, 262144])
@pytest.mark.parametrize("src", [F32, BF16])
def test_sample_mixed(q4k, vocab, src):
    rows = 12
    x, u = peaked(rows, vocab, vocab)
    i = torch.arange(rows)
    t = torch.tensor([1.0, 0.7, 0.0, 1.3])[i % 4]
    k = torch.tensor([0, 40, 1, vocab + 5, 1000])[i % 5]
    p = torch.tensor([1.0, 0.9, 0.3])[i % 3]
    m = torch.tensor([0.0, 0.1])[(i // 2) % 2]
    check_sample(q4k, x.to(src), u, t, k, p, m)
    check_sample(q4k, x.to(src), u)
    check_sample(q4k, x.to(src), u, t=torch.full((rows,), 5.0), p=torch.full((rows,), 0.8))


@pytest.mark.parametrize("rows,vocab", [(200, 3000), (160, 20011), (40, 70000)])
def test_sample_many_rows(q4k, rows, vocab):
    """Other cluster sizes than few rows take, and every way through the filters."""
    x, u = peaked(rows, vocab, rows)
    i = torch.arange(rows)
    t = torch.tensor([1.0, 0.6, 1.5, 3.0])[i % 4]
    k = torch.tensor([0, 0, 1500, 300, 2500, 12])[i % 6]
    p = torch.tensor([0.9, 0.5, 0.99, 1.0, 0.9999])[i % 5]
    m = torch.tensor([0.0, 0.0, 0.001])[i % 3]
    check_sample(q4k, x, u, t, k, p, m)
    check_sample(q4k, (x * 4).round().div(4).to(BF16), u, t, k, p, m)  # many ties


@pytest.mark.parametrize("rows,vocab", [(6, 9001), (170, 40003), (6, 131071)])
def test_sample_long_kept_sets_with_masked_tokens(q4k, rows, vocab):
    """More tokens kept than are sorted, with -inf and NaN between them."""
    x, u = peaked(rows, vocab, vocab + 1, 1.0)
    x[:, 5::11] = -math.inf
    x[:, 3::17] = math.nan
    i = torch.arange(rows)
    k = torch.tensor([0, 2100, vocab // 2, 7000])[i % 4]
    p = torch.tensor([0.97, 0.9, 0.999])[i % 3]
    for src in (F32, BF16):
        check_sample(q4k, x.to(src), u, torch.full((rows,), 3.0), k, p)
        check_sample(q4k, x.to(src), u, torch.full((rows,), 3.0), k, p, torch.full((rows,), 1e-3))


def test_sample_strided_rows_of_any_alignment(q4k):
    for src in (F32, BF16):
        x, u = peaked(5, 1111, 3)
        wide = torch.zeros((5, 1237), dtype=src)
        wide[:, 3:1114] = x.to(src)
        check_sample(q4k, wide[:, 3:1114], u, k=torch.full((5,), 50), p=torch.full((5,), 0.9))


@pytest.mark.parametrize("vocab", [7, 5000, 131072])
def test_sample_ties(q4k, vocab):
    """Equal logits: the lowest indexes are the first of the order."""
    u = torch.linspace(0, 1 - 2.0 ** -24, 16)
    x = torch.zeros((16, vocab))
    check_sample(q4k, x, u)
    check_sample(q4k, x, u, k=torch.full((16,), 5))
    check_sample(q4k, x, u, p=torch.full((16,), 0.5))
    check_sample(q4k, x, u, k=torch.full((16,), 4), p=torch.full((16,), 0.5), m=torch.full((16,), 1.0))
    check_sample(q4k, x, u, t=torch.zeros(16))
    x[:, ::3] = 1.0
    x[:, 1::3] = -0.0
    check_sample(q4k, x, u, k=torch.full((16,), vocab // 2), p=torch.full((16,), 0.95))
    x = torch.randint(-3, 4, (16, vocab), generator=gen(vocab)).float() / 2
    check_sample(q4k, x, u, k=torch.full((16,), vocab * 2 // 3 + 1), p=torch.full((16,), 0.8))


def test_sample_masks_infinities_and_nan(q4k):
    x, u = peaked(14, 3001, 8)
    low = torch.finfo(F32).min
    x[0, 10:] = -math.inf
    x[1, :-1] = -math.inf
    x[2] = -math.inf
    x[3, ::2] = math.nan
    x[4] = math.nan
    x[5, [7, 900]] = math.inf
    x[6] = low
    x[7, 5:] = low
    x[8, 100] = torch.finfo(F32).max
    x[9, :] = -math.inf
    x[9, 55] = low
    x[10] = torch.linspace(-1e38, 1e38, 3001)
    x[11, [5, 6]] = math.inf
    x[11, 8] = math.nan
    check_sample(q4k, x, u)
    check_sample(q4k, x, u, k=torch.full((14,), 20), p=torch.full((14,), 0.7), m=torch.full((14,), 0.05))
    check_sample(q4k, x, u, t=torch.zeros(14))
    check_sample(q4k, x, u, t=torch.full((14,), 1e-30))
    check_sample(q4k, x, u, t=torch.full((14,), 1e-42), p=torch.full((14,), 0.9))
    check_sample(q4k, x, u, t=torch.full((14,), 1e30), p=torch.full((14,), 0.9))


def test_sample_parameters_at_their_ends(q4k):
    x, u = peaked(10, 2000, 9)
    off = torch.tensor([0.0, -1.0, 1.0, 1.5, 2.0 ** -30, math.nan, 0.5, 0.999999, 1e-10, math.inf])
    check_sample(q4k, x, u, p=off)
    check_sample(q4k, x, u, m=off)
    check_sample(q4k, x, u, t=torch.tensor([-1.0, math.nan, -math.inf, 0.01, 100.0, 1e4, 0.5, 1e-4, 2.0, 1.0]))
    check_sample(q4k, x, u, k=torch.tensor([-5, 0, 1, 2, 1999, 2000, 2001, 2 ** 31 - 1, 3, -2 ** 31]))
    check_sample(q4k, x, torch.tensor([0.0, -0.5, 1.0, 2.0, 1 - 2.0 ** -24, 2.0 ** -149, 0.5, math.inf, -math.inf, 1e-9]), p=torch.full((10,), 0.9))


def test_sample_takes_every_token_by_its_share(q4k):
    """A sweep of u over a small row walks through the kept tokens in index order."""
    x = torch.tensor([[1.0, 3.0, 2.0, -math.inf, 2.5, 0.0]]).repeat(4000, 1)
    u = (torch.arange(4000) + 0.5) / 4000
    token, _ = q4k.q4k_sample(x.to(DEV), u.to(DEV), top_k=torch.full((4000,), 3, dtype=torch.int32, device=DEV))
    token = token.cpu()
    assert bool((token[1:] >= token[:-1]).all()) and set(token.tolist()) == {1, 2, 4}
    e = torch.exp(torch.tensor([3.0, 2.0, 2.5], dtype=torch.float64))
    for i, tok in enumerate((1, 2, 4)):
        assert abs(int((token == tok).sum()) - 4000 * float(e[i] / e.sum())) <= 1.01


# ------------------------------------------------------------------------------------------ together


def test_every_call_in_a_graph(q4k):
    """Plan, write, attention, norm and sampling captured once and replayed over changed inputs."""
    n, h, hq, d, page, vocab = 3, 2, 8, 64, 16, 1000
    g = gen(21)
    lens0 = torch.tensor([15, 0, 40], dtype=torch.int32)
    lens, add = lens0.to(DEV), torch.ones(n, dtype=torch.int32, device=DEV)
    table = torch.full((n, 6), -1, dtype=torch.int32)
    table[0, 0], table[2, :3] = 0, torch.tensor([1, 2, 3], dtype=torch.int32)
    table, pool, state = table.to(DEV), torch.arange(20, dtype=torch.int32, device=DEV), torch.tensor([4, 16], dtype=torch.int32, device=DEV)
    caches = [torch.randn((20, h, page, d), generator=g).to(BF16).to(DEV) for _ in range(2)]
    k, v, q = torch.randn((n, h, d), device=DEV), torch.randn((n, h, d), device=DEV), torch.randn((n, hq, d), device=DEV).to(BF16)
    gamma, logits, u = torch.ones(hq * d, device=DEV), torch.randn((n, vocab), device=DEV), torch.rand(n, device=DEV)

    def step():
        out = (lens, torch.empty(n + 1, dtype=torch.int64, device=DEV), *[torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(3)], state)
        _, _, slots, _, status, _ = q4k.q4k_kv_plan(lens, add, table, pool, state, page, n, out=out)
        q4k.q4k_kv_write(k, v, slots, *caches)
        o, lse = q4k.q4k_paged_attn(q, *caches, table, lens, 0.1)
        y, _ = q4k.q4k_add_rmsnorm(o.view(n, hq * d), None, gamma, 1e-6)
        token, logp = q4k.q4k_sample(logits, u)
        return slots, status, o, lse, y, token, logp

    keep = [x.clone() for x in (lens, table, pool, state, *caches)]
    eager = []
    for _ in range(4):
        k.mul_(1.5)
        eager.append([x.clone() for x in step()])
    torch.cuda.synchronize()
    after = [x.clone() for x in (lens, table, pool, state, *caches)]
    for x, y in zip((lens, table, pool, state, *caches), keep):
        x.copy_(y)
    k.div_(1.5 ** 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            static = step()
    torch.cuda.synchronize()
    for i in range(4):
        k.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(static, eager[i]):
            assert torch.equal(a, b)
    for x, y in zip((lens, table, pool, state, *caches), after):
        assert torch.equal(x, y)
    assert lens.tolist() == [19, 4, 44] and q4k.q4k_get_device_error() == 0
