"""Scores of given tokens against a plain 64-bit form.

Tolerances: a row's sum is that of up to V / 4096 + 16 additions in a row in fp32 and of exponentials good to 2^-21:
relative 2^-17 for V up to 131072 (2^-16 for twice that), which moves a logarithm by as much; besides, x - M and the
result are rounded: 2^-22 |logp|.  The entropy is ln l - w / l, where w has terms e d with |d| <= 8 + what counts, so
that w / l is off by 2^-17 (|w| / l) <= 2^-17 (entropy + 16): the reference lies within 8 of the maximum.
"""
from __future__ import annotations

import math

import pytest
import torch

from _gpu import DEV

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q4k():
    from bit_block_quantized_q4_gb300 import build
    build.build()
    import bit_block_quantized_q4_gb300 as m
    assert m.q4k_get_device_error() == 0
    return m


def plain(logits, tokens, top):
    x = logits.double().cpu()
    x = torch.where(torch.isnan(x), -math.inf, x)
    rows, v = x.shape
    high = x.amax(-1, keepdim=True)
    z = torch.where(x == high, 0.0, x - high)
    z = torch.where(high == -math.inf, -math.inf, z)
    e = torch.exp(z)
    lse = torch.log(e.sum(-1, keepdim=True))
    logp_all = torch.where(z == -math.inf, -math.inf, z - lse)
    entropy = -torch.where(e > 0, torch.exp(logp_all) * logp_all, 0.0).sum(-1)
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    place = torch.empty_like(order).scatter_(1, order, torch.arange(v).expand(rows, v))
    t = tokens.long().cpu()
    real = (t >= 0) & (t < v)
    at = t.clamp(0, v - 1)[:, None]
    logp = torch.where(real, logp_all.gather(1, at)[:, 0], -math.inf)
    rank = torch.where(real, place.gather(1, at)[:, 0], -1)
    tops, top_logp = torch.full((rows, top), -1), torch.full((rows, top), -math.inf, dtype=torch.float64)
    n = min(top, v)
    kept = value[:, :n] > -math.inf
    tops[:, :n] = torch.where(kept, order[:, :n], -1)
    top_logp[:, :n] = torch.where(kept, logp_all.gather(1, order[:, :n]), -math.inf)
    return logp, rank, entropy, tops, top_logp


def near(got, want, part):
    got = got.double().cpu()
    gone = want == -math.inf
    assert bool(torch.equal(got == -math.inf, gone))
    off = torch.where(gone, 0.0, (got - want).abs())
    worst = float((off / (part + 2.0 ** -22 * torch.where(gone, 0.0, want.abs()))).max()) if off.numel() else 0.0
    assert worst <= 1.0, worst


def check(got, logits, tokens, top):
    want = plain(logits, tokens, top)
    part = 2.0 ** -17 * max(1.0, logits.shape[1] / 131072)
    assert torch.equal(got[1].cpu().long(), want[1]) and torch.equal(got[3].cpu().long(), want[3])
    near(got[0], want[0], part)
    near(got[4], want[4], part)
    off = (got[2].double().cpu() - want[2]).abs() / (part * (want[2] + 17))
    assert float(off.max()) <= 1.0, float(off.max())


def rows_of(seed, rows, vocab, dtype, ld=None, shift=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, vocab), generator=g) * 3
    x[torch.arange(rows), torch.randint(0, vocab, (rows,), generator=g)] += 9
    tokens = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32)
    tokens[::2] = x.argmax(-1)[::2].to(torch.int32)
    if ld is None:
        return x.to(dtype).to(DEV), tokens
    wide = torch.zeros(rows * ld + shift, dtype=dtype, device=DEV)
    view = wide.as_strided((rows, vocab), (ld, 1), shift)
    view.copy_(x)
    return view, tokens


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 7, 5), (2, 33, 32), (5, 100, 20), (40, 1000, 3), (2, 2500, 20), (3, 4097, 32), (1, 32000, 20), (400, 8192, 1), (9, 32001, 5), (170, 50257, 0), (2, 131072, 32),
                                            (1, 262147, 8)])
def test_matches_the_plain_form(q4k, dtype, rows, vocab, top):
    x, tokens = rows_of(1, rows, vocab, dtype)
    check(q4k.q4k_logprobs(x, tokens.to(DEV), top=top), x, tokens, top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld,shift", [(10007, 0), (10001, 3), (10008, 1), (10003, 7)])
def test_rows_that_are_not_aligned(q4k, dtype, ld, shift):
    x, tokens = rows_of(2, 11, 10001, dtype, ld, shift)
    check(q4k.q4k_logprobs(x, tokens.to(DEV), top=6), x, tokens, 6)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab", [(2, 20000), (300, 20000), (1, 131072)])
def test_equal_logits_and_sorted_rows(q4k, dtype, rows, vocab):
    """What makes the list of candidates long: all logits equal, rising, falling, and the highest at one thread's tokens."""
    tokens = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    ramp = torch.linspace(-4, 4, vocab)
    comb = torch.where((torch.arange(vocab) // 8) % 512 == 77, 5.0, 0.0) + ramp / 100
    for base in (torch.zeros(vocab), ramp, ramp.flip(0), comb, torch.where(torch.arange(vocab) % 2 == 0, 0.0, -0.0)):
        x = base.expand(rows, vocab).to(dtype).contiguous().to(DEV)
        check(q4k.q4k_logprobs(x, tokens.to(DEV), top=32), x, tokens, 32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab", [(1, 40000), (8, 300), (350, 5000)])
def test_values_that_are_not_finite(q4k, dtype, rows, vocab):
    low = torch.finfo(dtype).min
    for seed, spoil in enumerate((
            lambda x: x.fill_(-math.inf), lambda x: x.fill_(math.nan), lambda x: x.fill_(low), lambda x: x[:, vocab // 3:].fill_(-math.inf), lambda x: x[:, ::2].fill_(math.nan),
            lambda x: x[:, 5:].fill_(low), lambda x: x[:, [3, 200]].fill_(math.inf), lambda x: x[:, 1:].fill_(math.nan), lambda x: x[:, 7:].fill_(-math.inf), lambda x: x.fill_(math.inf))):
        x, tokens = rows_of(10 + seed, rows, vocab, dtype)
        spoil(x)
        tokens[0] = 5
        check(q4k.q4k_logprobs(x, tokens.to(DEV), top=9), x, tokens, 9)


def test_large_and_small_logits(q4k):
    x, tokens = rows_of(4, 6, 9000, F32)
    for scale, shift in ((1e4, 0.0), (1.0, 1e6), (1e-6, 0.0), (1e30, 0.0), (1.0, -3e4)):
        y = x * scale + shift
        want = plain(y, tokens, 4)
        got = q4k.q4k_logprobs(y, tokens.to(DEV), top=4)
        assert torch.equal(got[1].cpu().long(), want[1]) and torch.equal(got[3].cpu().long(), want[3])
        near(got[0], want[0], 2.0 ** -17)
        near(got[4], want[4], 2.0 ** -17)


def test_tokens_outside_the_vocabulary_and_many_rows(q4k):
    x, tokens = rows_of(5, 70001, 24, F32)
    tokens[::7], tokens[1::7], tokens[2::7] = -1, 24, -2 ** 31
    check(q4k.q4k_logprobs(x, tokens.to(DEV), top=2), x, tokens, 2)
    empty = q4k.q4k_logprobs(x[:0], tokens[:0].to(DEV), top=2)
    assert [tuple(t.shape) for t in empty] == [(0,), (0,), (0,), (0, 2), (0, 2)]


def test_outputs_given_streams_graphs_and_repeated_calls(q4k):
    x, tokens = rows_of(6, 5, 131072, BF16)
    t = tokens.to(DEV)
    want = [y.clone() for y in q4k.q4k_logprobs(x, t, top=20)]
    same = lambda got: all(torch.equal(a, b) for a, b in zip(got, want))  # noqa: E731
    for _ in range(3):
        assert same(q4k.q4k_logprobs(x, t, top=20))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q4k.q4k_logprobs(x, t, top=20, stream=side)
    side.synchronize()
    assert same(got)
    out = [torch.zeros_like(y) for y in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4k.q4k_logprobs(x, t, top=20, logp=out[0], rank=out[1], entropy=out[2], top_tokens=out[3], top_logp=out[4])
    graph.replay()
    torch.cuda.synchronize()
    assert same(out)


def test_agrees_with_the_sampler(q4k):
    """The log-probability that q4k_sample gives without filters is that of its token here."""
    x, _ = rows_of(7, 20, 32000, F32)
    u = torch.rand(20, generator=torch.Generator().manual_seed(1)).to(DEV)
    token, logp = q4k.q4k_sample(x, u)
    mine = q4k.q4k_logprobs(x, token)[0]
    assert float((mine - logp).abs().max()) <= 2.0 ** -16
