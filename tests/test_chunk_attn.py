"""Attention of chunks of new tokens over the paged cache against a plain 64-bit form.

Tolerances count roundings (half a step of bf16 is 2^-8, of fp16 2^-11, relative).  An output is a weighted mean of
values; with A = sum of weight x |value|:
  - the result's own rounding: 2^-8 |out|;
  - each weight's: 2^-8 A (one bf16 term), or 2^-11 A (one fp16 term, e4m3 cache);
  - an e4m3 cache's weight times scale below 2^-14 is stored in steps of 2^-24, with a reference of 2^7 or more: off by
    2^-32 of the largest such term, which is at most max scale: 2^-32 max(scale) sum |value / scale|;
  - scores in fp32: softmax_scale sum |q||k| is at most about 12 here (dim 256: 24), so that the D additions and the
    exponential move a weight by less than 24 x 256 x 2^-24 x 1.5 < 2^-10 (as much again for the sum of weights: taken
    together below 2^-9): 2^-9 A.
The logarithm of the sum moves by no more than a score: 2^-10, and its own rounding.
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


class Step:
    """A step over a paged cache: requests of (cached tokens with the new ones, new tokens)."""

    def __init__(self, seed, both, q_heads=8, kv_heads=2, dim=128, page=16, cache=BF16, pad=0, spare=3, fill=float("nan"), width=None):
        g = torch.Generator().manual_seed(seed)
        self.both, self.page, self.cache, self.dim, self.kv_heads, self.q_heads = both, page, cache, dim, kv_heads, q_heads
        n = len(both)
        counts = [-(-max(a, 0) // page) for a, _ in both]
        pages = sum(counts) + 1
        width = width or max(counts + [1]) + spare
        ids = (torch.randperm(pages - 1, generator=g) + 1).tolist()
        self.table = torch.zeros((n, width), dtype=torch.int32)
        at = 0
        for r, c in enumerate(counts):
            use = min(c, width)
            self.table[r, :use] = torch.tensor(ids[at:at + use], dtype=torch.int32)
            at += c
        self.cu = torch.tensor([0] + [b for _, b in both]).cumsum(0)
        t = int(self.cu[-1]) + pad
        self.q = (torch.randn((t, q_heads, dim), generator=g) * 1.5).to(BF16)
        self.k, self.v, self.ks, self.vs = [], [], [], []
        shape = (pages, kv_heads, page, dim)
        make = lambda: torch.randn(shape, generator=g)  # noqa: E731
        self.k, self.v = make().to(cache), make().to(cache)
        if cache == E4M3:
            self.ks, self.vs = (torch.empty(shape[:3]).uniform_(0.25, 2.0, generator=g) for _ in range(2))
        else:
            self.ks = self.vs = None
        # what no request has written: the rest of a last page, and page 0
        for c in (self.k, self.v):
            raw = c.view(torch.uint8) if cache == E4M3 else c
            value = 0x7F if cache == E4M3 else fill
            raw[0] = value
            for r, (a, _) in enumerate(both):
                if a % page and a > 0 and a // page < width:
                    raw[self.table[r, a // page], :, a % page:] = value
        self.lens = torch.tensor([a for a, _ in both], dtype=torch.int32)

    def rows(self, r, j, length):
        """(K, V) of head j, the first `length` tokens, in 64 bits."""
        pages = self.table[r, :-(-length // self.page)].long()
        out = []
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            x = (c.view(torch.uint8)[pages, j].view(E4M3) if self.cache == E4M3 else c[pages, j]).double()
            if s is not None:
                x = x * s[pages, j].double()[..., None]
            out.append(x.flatten(0, 1)[:length])
        return out

    def plain(self, scale, window):
        group = self.q_heads // self.kv_heads
        out = torch.full(self.q.shape, 7.0, dtype=torch.float64)
        mass = torch.zeros(self.q.shape, dtype=torch.float64)
        lse = torch.full(self.q.shape[:2], 7.0, dtype=torch.float64)
        for r, (length, new) in enumerate(self.both):
            if not new:
                continue
            part = slice(int(self.cu[r]), int(self.cu[r]) + new)
            length_seen = min(max(length, 0), self.table.shape[1] * self.page)
            pos = torch.arange(max(length, 0) - new, max(length, 0))
            at = torch.arange(length_seen)
            seen = (at[None] <= pos[:, None]) & ((at[None] > pos[:, None] - window) if window else True)
            for j in range(self.kv_heads):
                heads = slice(j * group, (j + 1) * group)
                if not length_seen:
                    out[part, heads], lse[part, heads] = 0.0, -math.inf
                    continue
                k, v = self.rows(r, j, length_seen)
                z = scale * torch.einsum("tgd,ld->tgl", self.q[part, heads].double(), torch.where(torch.isnan(k), 0.0, k))
                z = torch.where(seen[:, None], z, -math.inf)
                l = torch.logsumexp(z, -1)
                w = torch.exp(z - torch.where(l == -math.inf, 0.0, l)[..., None])
                clean = torch.where(torch.isfinite(v), v, 0.0)
                out[part, heads] = torch.einsum("tgl,ld->tgd", w, clean)
                mass[part, heads] = torch.einsum("tgl,ld->tgd", w, clean.abs())
                lse[part, heads] = l
        return out, mass, lse

    def run(self, q4k, scale, window=0, **kw):
        d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        self.out = torch.full(self.q.shape, 7.0, dtype=BF16, device=DEV)
        self.lse = torch.full(self.q.shape[:2], 7.0, device=DEV)
        kw.setdefault("out", self.out)
        kw.setdefault("lse", self.lse)
        return q4k.q4k_paged_attn_chunk(d(self.q), d(self.k), d(self.v), d(self.table), d(self.lens), d(self.cu), scale, d(self.ks), d(self.vs), window=window, **kw)

    def check(self, got, scale, window=0, rows=None):
        out, mass, lse = self.plain(scale, window)
        o, l = got[0].double().cpu(), got[1].double().cpu()
        rows = slice(None) if rows is None else rows
        part = 2.0 ** -11 if self.cache == E4M3 else 2.0 ** -8
        bound = 2.0 ** -8 * out.abs() + (part + 2.0 ** -9) * mass + 1e-30
        if self.cache == E4M3:
            bound += 2.0 ** -32 * float(self.vs.max()) * torch.nan_to_num(self.v.double()).abs().sum() / self.dim
        worst = float(((o - out).abs() / bound)[rows].max())
        assert bool(torch.isfinite(o[rows]).all()) and worst <= 1.0, worst
        gone = lse == -math.inf
        assert bool(torch.equal((l == -math.inf)[rows], gone[rows]))
        worst = float(torch.where(gone, 0.0, (l - lse).abs() / (2.0 ** -10 + 2.0 ** -22 * lse.abs().clamp(max=1e30)))[rows].max())
        assert worst <= 1.0, worst


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16), (128, 256), (256, 32)])
def test_one_chunk(q4k, cache, dim, page):
    s = Step(1, [(45, 45)], dim=dim, page=page, cache=cache)
    s.check(s.run(q4k, dim ** -0.5), dim ** -0.5)
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("dim,heads,kv_heads,page,window", [
    (64, 8, 8, 16, 0), (64, 6, 2, 64, 100), (128, 8, 1, 32, 0), (128, 5, 1, 16, 37), (128, 32, 2, 128, 0), (256, 4, 2, 16, 0), (256, 12, 1, 64, 300), (128, 2, 2, 256, 1)])
def test_ragged_step(q4k, cache, dim, heads, kv_heads, page, window):
    both = [(300, 300), (1, 1), (700, 1), (129, 1), (513, 0), (1000, 77), (128, 128), (256, 3), (17, 16), (0, 0), (900, 260)]
    s = Step(2, both, heads, kv_heads, dim, page, cache, pad=5)
    s.check(s.run(q4k, dim ** -0.5, window), dim ** -0.5, window)
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("dim,both", [(64, [(6000, 9)]), (128, [(20011, 5)]), (256, [(5003, 40), (4096, 1)]), (128, [(1, 1)] * 300 + [(2500, 2)])])
def test_long_contexts_are_split_and_joined(q4k, cache, dim, both):
    s = Step(3, both, 8, 1, dim, 16, cache)
    s.check(s.run(q4k, dim ** -0.5), dim ** -0.5)
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt(q4k, cache, dim):
    s = Step(4, [(1500, 1500), (1700, 600)], 4, 2, dim, 32, cache)
    s.check(s.run(q4k, dim ** -0.5), dim ** -0.5)
    s.check(s.run(q4k, dim ** -0.5, 333), dim ** -0.5, 333)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-30])
def test_scales_that_are_not_positive(q4k, cache, scale):
    s = Step(5, [(200, 150), (40, 1)], cache=cache)
    s.check(s.run(q4k, scale), scale)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_maximum_that_grows_and_a_dominating_token(q4k, cache, dim):
    """Scores that rise by dozens of binary orders along the keys (every tile moves the reference), and fall."""
    for falling in (False, True):
        s = Step(6, [(1000, 200)], 4, 2, dim, 16, cache)
        ramp = torch.linspace(0.1, 3.0, 1000)
        ramp = ramp.flip(0) if falling else ramp
        direction = torch.where(torch.arange(dim) % 2 == 0, 1.0, -1.0)
        for i in range(1000):
            s.k[s.table[0, i // 16], :, i % 16] = (direction * ramp[i]).to(cache)
        s.q = (direction * torch.linspace(0.5, 2.0, s.q.shape[0])[:, None, None]).expand(s.q.shape).to(BF16).contiguous()
        if s.ks is not None:
            s.ks.fill_(1.0)
        # (here scores reach 2 x 3 x dim x scale: an fp32 sum of D equal-sized terms is off by D 2^-24 of it, below 2^-9)
        s.check(s.run(q4k, 0.25), 0.25)


def test_e4m3_scales_of_many_orders(q4k):
    s = Step(7, [(777, 300)], 8, 2, 128, 16, E4M3)
    g = torch.Generator().manual_seed(1)
    s.vs = torch.exp2(torch.empty(s.vs.shape).uniform_(-90.0, 60.0, generator=g))
    s.ks = torch.exp2(torch.empty(s.ks.shape).uniform_(-20.0, 1.0, generator=g))
    out, mass, lse = s.plain(0.05, 0)
    got = s.run(q4k, 0.05)
    # as elsewhere, and the least terms: 2^-32 of the largest one times a value of up to 448, for each of 777
    k, v = zip(*[s.rows(0, j, 777) for j in range(2)])
    big = torch.stack([x.abs().max() for x in v]).repeat_interleave(4)[None, :, None]
    bound = 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2.0 ** -9) * mass + 2.0 ** -32 * 777 * big
    worst = float(((got[0].double().cpu() - out).abs() / bound).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_later_tokens_that_are_not_finite_stay_out_of_earlier_results(q4k, cache, dim, which):
    both = [(150, 150), (300, 40)]
    clean, s = Step(8, both, 4, 2, dim, 16, cache), Step(8, both, 4, 2, dim, 16, cache)
    for r, at in ((0, 77), (1, 290)):
        for name in "kv" if which == "both" else which:
            row = getattr(s, name)[s.table[r, at // 16], :, at % 16]
            if cache == E4M3:
                getattr(s, name).view(torch.uint8)[s.table[r, at // 16], :, at % 16, 3] = 0x7F
            else:
                row[:, 3] = math.inf if r else math.nan
    want, got = clean.run(q4k, dim ** -0.5), s.run(q4k, dim ** -0.5)
    before = torch.cat([torch.arange(77), 150 + torch.arange(30)])
    after = torch.cat([torch.arange(77, 150), 150 + torch.arange(30, 40)])
    assert torch.equal(want[0][before], got[0][before]) and torch.equal(want[1][before], got[1][before])
    if which != "k" or cache == E4M3:
        assert bool((~torch.isfinite(got[0][after].float())).any(-1).all())
    assert q4k.q4k_get_device_error() == 0


def test_e4m3_scales_of_later_tokens_that_are_not_finite(q4k):
    clean, s = Step(9, [(150, 150)], 4, 2, 128, 16, E4M3), Step(9, [(150, 150)], 4, 2, 128, 16, E4M3)
    s.vs[s.table[0, 5], :, 1] = math.inf
    s.ks[s.table[0, 6], :, 1] = math.nan
    want, got = clean.run(q4k, 0.1), s.run(q4k, 0.1)
    assert torch.equal(want[0][:81], got[0][:81])
    assert bool(torch.isnan(got[0][81:].float()).all())


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_absent_pages_and_lengths_past_the_table(q4k, cache):
    s = Step(10, [(400, 30), (200, 7), (64, 64)], 4, 2, 128, 16, cache)
    good = s.table.clone()
    s.table[0, 3], s.table[0, 20], s.table[1, 12] = -1, 10 ** 6, s.k.shape[0]
    got = s.run(q4k, 0.1)
    assert q4k.q4k_get_device_error() == BAD_PAGE
    # the same with these tokens far below the others: an absent page has no weight
    part = s
    s.table = good
    out, mass, lse = torch.zeros(s.q.shape, dtype=torch.float64), torch.zeros(s.q.shape, dtype=torch.float64), None
    for r, (length, new) in enumerate(s.both):
        gone = {0: [3, 20], 1: [12]}.get(r, [])
        at = torch.arange(length)
        keep = ~torch.isin(at // 16, torch.tensor(gone + [-1]))
        pos = torch.arange(length - new, length)
        rows = slice(int(s.cu[r]), int(s.cu[r]) + new)
        for j in range(2):
            k, v = part.rows(r, j, length)
            z = 0.1 * torch.einsum("tgd,ld->tgl", s.q[rows, 2 * j:2 * j + 2].double(), k)
            z = torch.where(((at[None] <= pos[:, None]) & keep[None])[:, None], z, -math.inf)
            w = torch.softmax(z, -1)
            out[rows, 2 * j:2 * j + 2] = torch.einsum("tgl,ld->tgd", w, v)
            mass[rows, 2 * j:2 * j + 2] = torch.einsum("tgl,ld->tgd", w, v.abs())
    bound = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -9) * mass
    assert bool(((got[0].double().cpu() - out).abs() <= bound).all())
    # lengths past a table of 5 pages: tokens past it are absent, the window ends at the token itself
    long = Step(11, [(200, 60), (1000, 4)], 4, 2, 128, 16, cache, width=5)
    got = long.run(q4k, 0.1, 90)
    assert q4k.q4k_get_device_error() == BAD_PAGE
    long.check(got, 0.1, 90)


def test_tokens_before_the_first_position_and_bad_offsets(q4k):
    # a request that was not served: 9 tokens announced, 4 cached
    s = Step(12, [(4, 9), (100, 10)], 4, 2, 128, 16)
    got = s.run(q4k, 0.1)
    s.check(got, 0.1)
    assert bool((got[0][:5] == 0).all()) and bool((got[1][:5] == -math.inf).all())
    assert q4k.q4k_get_device_error() == 0
    for cu in ([0, -1, 19], [0, 9, 21], [-3, 9, 19], [0, 2 ** 40, 19]):
        s = Step(12, [(4, 9), (100, 10)], 4, 2, 128, 16)
        s.cu = torch.tensor(cu)
        s.run(q4k, 0.1)
        assert q4k.q4k_get_device_error() == BAD_PAGE
    s = Step(12, [(-5, 3), (100, 10)], 4, 2, 128, 16)
    got = s.run(q4k, 0.1)
    assert bool((got[0][:3] == 0).all()) and q4k.q4k_get_device_error() == 0


def test_strides_of_q_out_and_cache(q4k):
    s = Step(13, [(300, 90), (40, 1)], 4, 2, 128, 16)
    want = s.run(q4k, 0.1)
    wide = torch.zeros((s.q.shape[0], 8, 136), dtype=BF16, device=DEV)
    q = wide[:, 2:6, :128]
    q.copy_(s.q)
    out = torch.zeros((s.q.shape[0], 6 * 128), dtype=BF16, device=DEV)
    k = s.k.transpose(1, 2).contiguous().transpose(1, 2).to(DEV)
    k = torch.empty_strided(s.k.shape, (2 * 16 * 136, 136, 2 * 136, 1), dtype=BF16, device=DEV).copy_(s.k)
    v = torch.empty_strided(s.v.shape, (2 * 16 * 136, 136, 2 * 136, 1), dtype=BF16, device=DEV).copy_(s.v)
    got = q4k.q4k_paged_attn_chunk(q, k, v, s.table.to(DEV), s.lens.to(DEV), s.cu.to(DEV), 0.1, out=out[:, 128:640].unflatten(1, (4, 128)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((out[:, :128] == 0).all()) and bool((out[:, 640:] == 0).all())


def test_agrees_with_the_call_for_one_token(q4k):
    s = Step(14, [(1, 1), (500, 1), (3001, 1)], 8, 2, 128, 16)
    got = s.run(q4k, 0.1)
    one = q4k.q4k_paged_attn(s.q.to(DEV), s.k.to(DEV), s.v.to(DEV), s.table.to(DEV), s.lens.to(DEV), 0.1)
    out, mass, _ = s.plain(0.1, 0)
    bound = 2.0 ** -7 * out.abs() + (2.0 ** -8 + 2.0 ** -8) * mass  # both calls' roundings
    assert bool(((got[0].double() - one[0].double()).abs().cpu() <= bound).all())
    assert float((got[1] - one[1]).abs().max()) <= 2.0 ** -9


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_streams_graphs_and_repeated_calls_give_the_same_bits(q4k, cache):
    s = Step(15, [(700, 200), (5000, 3), (90, 90)], 8, 2, 128, 16, cache, pad=4)
    want = [x.clone() for x in s.run(q4k, 0.1)]
    for _ in range(3):
        got = s.run(q4k, 0.1)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    args = [d(x) for x in (s.q, s.k, s.v, s.table, s.lens, s.cu)]
    scales = (d(s.ks), d(s.vs))
    out, lse = torch.full_like(args[0], 7.0), torch.full(s.q.shape[:2], 7.0, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q4k.q4k_paged_attn_chunk(*args, 0.1, *scales, out=out, lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0])
    out.fill_(7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4k.q4k_paged_attn_chunk(*args, 0.1, *scales, out=out, lse=lse)
    # lengths that change between replays
    for cut in (0, 1):
        args[4].copy_(s.lens - cut * torch.tensor([30, 2500, 0], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        fresh = q4k.q4k_paged_attn_chunk(*args, 0.1, *scales, out=torch.full_like(out, 7.0))
        assert torch.equal(out, fresh[0])
        assert cut or torch.equal(out, want[0])
