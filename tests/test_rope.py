"""Norm of heads and rotation by position, with and without the cache write, against a plain 64-bit form.

Tolerances count roundings (half a step of bf16 is 2^-8, of e4m3 2^-4, of fp32 2^-24, relative).  A pair (a, b) that
turns is off, before its own rounding, by at most (|a| + |b|) amplitude times
  - the angle in fp32: pi 2^-24, and its cosine and sine 2^-22: below 2^-21;
  - the norm's factor: a sum of D squares (D 2^-24, halved by the root) and four roundings, D <= 256: 132 x 2^-24;
  - two products and a sum: 3 x 2^-24;
together below 2^-16.
"""
from __future__ import annotations

import math

import pytest
import torch

from _gpu import DEV

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BAD_PAGE = 4


@pytest.fixture(scope="module")
def q4k():
    from bit_block_quantized_q4_gb300 import build
    build.build()
    import bit_block_quantized_q4_gb300 as m
    assert m.q4k_get_device_error() == 0
    return m


def plain(x, pos, steps, gamma, eps, interleaved, amplitude):
    """(result, size of what turns) in 64 bits; steps: python integers."""
    x = x.double().cpu()
    rot = 2 * len(steps)
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double().cpu()
    turn = torch.tensor([[(p * s % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for s in steps] for p in pos.tolist()], dtype=torch.float64).reshape(len(pos), 1, len(steps))
    c, s = torch.cos(turn) * amplitude, torch.sin(turn) * amplitude
    y, size = x.clone(), x.abs()
    i = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    j = i + 1 if interleaved else i + rot // 2
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    both = (a.abs() + b.abs()) * abs(amplitude)
    size[..., i], size[..., j] = both, both
    return y, size


def ints(steps):
    return [int(s) % 2 ** 64 for s in steps.tolist()]


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF16 else 2.0 ** -24


def inputs(seed, tokens, heads, dim, dtype, top=100000):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((tokens, heads, dim), generator=g) * 2).to(dtype)
    pos = torch.randint(0, top, (tokens,), generator=g, dtype=torch.int32)
    return x, pos, 1 + 0.2 * torch.randn(dim, generator=g)


@pytest.mark.parametrize("tokens,heads,dim,rot,interleaved,norm,dtype,out", [
    (1, 1, 128, 128, False, False, F32, BF16), (16, 64, 128, 128, False, True, F32, BF16), (3, 5, 64, 64, True, True, BF16, F32), (7, 24, 256, 64, True, True, BF16, BF16),
    (9, 4, 256, 256, False, False, BF16, F32), (5, 3, 80, 32, False, True, F32, F32), (5, 3, 96, 96, True, False, BF16, BF16), (11, 2, 128, 20, False, True, F32, F32),
    (11, 2, 128, 126, False, True, BF16, BF16), (4, 2, 64, 2, False, True, F32, BF16), (4, 2, 64, 6, True, True, F32, BF16), (4, 3, 128, 0, False, True, F32, F32), (2, 1, 8, 8, False, True, F32, F32),
    (2, 2, 16, 16, True, True, BF16, BF16), (2, 2, 24, 16, False, True, F32, F32), (600, 32, 128, 64, False, True, BF16, BF16), (1999, 5, 64, 64, True, False, F32, F32), (700, 80, 256, 256, False, True, F32, BF16)])
def test_rope_matches_the_plain_form(q4k, tokens, heads, dim, rot, interleaved, norm, dtype, out):
    x, pos, gamma = inputs(1, tokens, heads, dim, dtype)
    steps, amplitude = q4k.q4k_rope_steps(rot, 10000.0, 4.0, 4096)
    got = q4k.q4k_rope(x.to(DEV), pos.to(DEV), steps.to(DEV), gamma=gamma.to(DEV) if norm else None, eps=1e-5, interleaved=interleaved, amplitude=amplitude, out_dtype=out)
    want, size = plain(x, pos, ints(steps), gamma if norm else None, 1e-5, interleaved, amplitude)
    worst = float(((got.double().cpu() - want).abs() / (half_step(out) * want.abs() + 2.0 ** -16 * size + 1e-30)).max())
    assert got.dtype == out and worst <= 1.0, worst


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 60])
def test_far_positions(q4k, interleaved, rot):
    x, _, _ = inputs(2, 6, 2, 64, F32)
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 31 - 1, 131071, 2 ** 30 + 12345], dtype=torch.int32)
    steps, _ = q4k.q4k_rope_steps(rot, 1e6)
    got = q4k.q4k_rope(x.to(DEV), pos.to(DEV), steps.to(DEV), interleaved=interleaved, out_dtype=F32)
    want, size = plain(x, pos, ints(steps), None, 0, interleaved, 1.0)
    worst = float(((got.double().cpu() - want).abs() / (2.0 ** -24 * want.abs() + 2.0 ** -20 * size)).max())  # (no norm: 2^-21 and three roundings)
    assert worst <= 1.0, worst


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (36, False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_place_strides_and_padding_tokens(q4k, rot, interleaved, dtype):
    tokens = 37
    x, pos, gamma = inputs(3, tokens, 6, 128, dtype)
    pos[::5] = -1
    pos[3] = -2 ** 31
    steps, _ = q4k.q4k_rope_steps(rot, 10000.0)
    d = lambda t: t.to(DEV)  # noqa: E731
    want = q4k.q4k_rope(d(x), d(pos), d(steps), gamma=d(gamma), interleaved=interleaved, out=torch.full_like(d(x), 7.0))
    assert bool((want[pos < 0] == 7.0).all())
    # a part of wider rows, in place; heads outermost
    wide = torch.full((tokens, 9, 136), 3.0, dtype=dtype, device=DEV)
    part = wide[:, 2:8, :128]
    part.copy_(x)
    assert q4k.q4k_rope(part, d(pos), d(steps), gamma=d(gamma), interleaved=interleaved, out=part) is part
    live = (pos >= 0)
    assert torch.equal(part[d(live)], want[d(live)]) and torch.equal(part[d(~live)], d(x[~live]))
    part.fill_(3.0)
    assert bool((wide == 3.0).all())
    turned = torch.zeros((6, tokens, 128), dtype=dtype, device=DEV).transpose(0, 1)
    q4k.q4k_rope(d(x), d(pos), d(steps), gamma=d(gamma), interleaved=interleaved, out=turned)
    assert torch.equal(turned[d(live)], want[d(live)]) and bool((turned[d(~live)] == 0).all())


def caches(pages, heads, page, dim, dtype):
    make = lambda: torch.full((pages, heads, page, dim), 1.0, device=DEV).to(dtype)  # noqa: E731
    sc = [torch.full((pages, heads, page), 5.0, device=DEV) for _ in range(2)] if dtype == E4M3 else [None, None]
    return make(), make(), sc[0], sc[1]


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,interleaved,norms,dtype,page", [
    (1, 4, 1, 128, 128, False, "qk", F32, 16), (24, 64, 8, 128, 128, False, "qk", F32, 16), (33, 6, 2, 64, 64, True, "", BF16, 32), (19, 5, 5, 256, 64, False, "q", BF16, 64), (40, 8, 2, 64, 22, False, "k", F32, 16),
    (700, 24, 8, 128, 96, True, "qk", BF16, 128)])
def test_rope_and_cache_write(q4k, cache, tokens, hq, hk, dim, rot, interleaved, norms, dtype, page):
    g = torch.Generator().manual_seed(4)
    x = (torch.randn((tokens, hq + 2 * hk, dim), generator=g) * 2).to(dtype)
    pos = torch.randint(0, 60000, (tokens,), generator=g, dtype=torch.int32)
    pages = 2 * tokens // page + 2
    slots = torch.randperm(pages * page, generator=g)[:tokens].to(torch.int32)
    if tokens > 9:
        pos[4], slots[7], pos[8], slots[8] = -1, -1, -1, -1
    gq, gk = (1 + 0.2 * torch.randn(dim, generator=g) for _ in range(2))
    steps, amplitude = q4k.q4k_rope_steps(rot, 10000.0, 2.0, 8192)
    d = lambda t: t.to(DEV)  # noqa: E731
    xd = d(x)
    q, k, v = xd[:, :hq], xd[:, hq:hq + hk], xd[:, hq + hk:]
    kc, vc, ks, vs = caches(pages, hk, page, dim, cache)
    out = torch.full((tokens, hq, dim), 7.0, dtype=BF16, device=DEV)
    use = dict(q_gamma=d(gq) if "q" in norms else None, k_gamma=d(gk) if "k" in norms else None, interleaved=interleaved, amplitude=amplitude)
    assert q4k.q4k_rope_kv_write(q, k, v, d(pos), d(slots), d(steps), kc, vc, ks, vs, out=out, **use) is out
    assert q4k.q4k_get_device_error() == 0
    # queries: what q4k_rope gives, to the bit
    same = torch.full_like(out, 7.0)
    q4k.q4k_rope(q, d(pos), d(steps), gamma=use["q_gamma"], interleaved=interleaved, amplitude=amplitude, out=same)
    assert torch.equal(out, same)
    # keys and values against the plain form
    want_k, size_k = plain(x[:, hq:hq + hk], pos.clamp(min=0), ints(steps), gk if "k" in norms else None, 1e-6, interleaved, amplitude)
    want = [want_k, x[:, hq + hk:].double()]
    sizes = [size_k, want[1].abs()]
    live = (pos >= 0) & (slots >= 0)
    rest = torch.ones((pages, page), dtype=torch.bool)
    for c, s, w, size in ((kc, ks, want[0], sizes[0]), (vc, vs, want[1], sizes[1])):
        got = c.float().double().cpu().transpose(1, 2).reshape(pages * page, hk, dim)[slots[live].long()]
        w, size = w[live], size[live]
        slack = 2.0 ** -16 * size
        if s is None:
            bound = 2.0 ** -8 * w.abs() + slack
        else:
            sc = s.double().cpu().transpose(1, 2).reshape(pages * page, hk)[slots[live].long()][..., None]
            amax = w.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
            assert bool(((sc - amax / 448).abs() <= (2.0 ** -22 * amax + slack.amax(-1, keepdim=True)) / 448).all())
            got = got * sc
            bound = 2.0 ** -4 * w.abs() * (1 + 2.0 ** -10) + 2.0 ** -10 * sc * (1 + 2.0 ** -10) + slack * 2
        worst = float(((got - w).abs() / (bound + 1e-30)).max())
        assert worst <= 1.0, worst
        # nothing else was written
        flat = rest.clone().flatten()
        flat[slots[live].long()] = False
        assert bool((c.float().cpu().transpose(1, 2).reshape(pages * page, hk, dim)[flat] == 1.0).all())
        if s is not None:
            assert bool((s.cpu().transpose(1, 2).reshape(pages * page, hk)[flat] == 5.0).all())


def test_the_fused_write_equals_the_separate_calls(q4k):
    x, pos, gamma = inputs(5, 50, 12, 128, BF16)
    steps, _ = q4k.q4k_rope_steps(128, 10000.0)
    d = lambda t: t.to(DEV)  # noqa: E731
    xd, slots = d(x), torch.arange(50, dtype=torch.int32, device=DEV)
    one, two = caches(4, 2, 16, 128, BF16), caches(4, 2, 16, 128, BF16)
    q = q4k.q4k_rope_kv_write(xd[:, :8], xd[:, 8:10], xd[:, 10:], d(pos), slots, d(steps), one[0], one[1], k_gamma=d(gamma))
    k = q4k.q4k_rope(xd[:, 8:10], d(pos), d(steps), gamma=d(gamma))
    v = xd[:, 10:].contiguous()
    q4k.q4k_kv_write(k, v, slots, two[0], two[1])
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert torch.equal(q, q4k.q4k_rope(xd[:, :8], d(pos), d(steps)))
    # in place: queries where the projection left them
    q4k.q4k_rope_kv_write(xd[:, :8], xd[:, 8:10], xd[:, 10:], d(pos), slots, d(steps), one[0], one[1], k_gamma=d(gamma), out=xd[:, :8])
    assert torch.equal(xd[:, :8], q) and torch.equal(one[0], two[0])


def test_slots_outside_the_cache_are_skipped_and_flagged(q4k):
    x, pos, _ = inputs(6, 4, 4, 64, F32)
    steps, _ = q4k.q4k_rope_steps(64, 10000.0)
    d = lambda t: t.to(DEV)  # noqa: E731
    xd = d(x)
    kc, vc, ks, vs = caches(2, 1, 16, 64, E4M3)
    slots = torch.tensor([3, 32, -2, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out = q4k.q4k_rope_kv_write(xd[:, :2], xd[:, 2:3], xd[:, 3:], d(pos), slots, d(steps), kc, vc, ks, vs)
    assert q4k.q4k_get_device_error() == BAD_PAGE
    assert torch.equal(out, q4k.q4k_rope(xd[:, :2], d(pos), d(steps)))
    changed = (vs != 5.0).nonzero().tolist()
    assert changed == [[0, 0, 3]]


def test_rows_of_zeros_and_values_that_are_not_finite(q4k):
    x = torch.zeros((4, 3, 64))
    x[1, 0, 3], x[2, 1, 40] = math.nan, math.inf
    steps, _ = q4k.q4k_rope_steps(64, 10000.0)
    pos, slots = torch.arange(4, dtype=torch.int32, device=DEV), torch.arange(4, dtype=torch.int32, device=DEV)
    xd, g = x.to(DEV), torch.ones(64, device=DEV)
    kc, vc, ks, vs = caches(1, 1, 16, 64, E4M3)
    out = q4k.q4k_rope_kv_write(xd[:, :1], xd[:, 1:2], xd[:, 2:], pos, slots, steps.to(DEV), kc, vc, ks, vs, q_gamma=g, k_gamma=g)
    assert bool((out[[0, 2, 3]] == 0).all()) and bool(torch.isnan(out[1].float()).any())
    assert bool((kc.float()[0, 0, [0, 1, 3]] == 0).all()) and bool(torch.isnan(kc.float()[0, 0, 2]).any())
    assert bool((ks[0, 0, :2] == 2.0 ** -100 / 448).all()) and bool(torch.isfinite(vs).all())


def test_streams_and_graphs(q4k):
    x, pos, gamma = inputs(7, 90, 10, 128, F32)
    steps, _ = q4k.q4k_rope_steps(128, 10000.0)
    d = lambda t: t.to(DEV)  # noqa: E731
    xd, pd, sd, gd, slots = d(x), d(pos), d(steps), d(gamma), torch.arange(90, dtype=torch.int32, device=DEV)
    kc, vc, ks, vs = caches(6, 1, 16, 128, E4M3)
    call = lambda **kw: q4k.q4k_rope_kv_write(xd[:, :8], xd[:, 8:9], xd[:, 9:], pd, slots, sd, kc, vc, ks, vs, q_gamma=gd, **kw)  # noqa: E731
    before = [t.clone() for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    want = call()
    keep = [t.clone() for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    for t, b in zip((kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), before):
        t.copy_(b)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for t, k in zip((kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), keep):
        assert torch.equal(t, k)
    empty = torch.empty((0, 8, 128), device=DEV)
    assert q4k.q4k_rope(empty, pd[:0], sd).shape == (0, 8, 128)
