"""Chunk attention over an e4m3 cache whose scales of V differ by many orders: rows of zeros as the library's own call
writes them, beside ordinary and large ones.

Tolerances count roundings.  S = softmax_scale max sum |q||k| bounds a score.
  - A score is off by (D + 8) 2^-23 S (D additions in the tensor cores, the scales' products), and so is the logarithm
    of the sum; besides, references of up to 128 binary orders and the logarithm are rounded to 2^-18 each, four times at
    most, a sum of T tiles of 128 weights good to 2^-21 to (T + 34) 2^-24 + 2^-21:
    lse within (D + 8) 2^-23 S + 2^-16 + (T + 40) 2^-24 + 2^-22 |lse|.
  - An output is a mean of values; with A = sum of weight x |value| it is rounded (2^-8 |out|), and so are weights (two
    times 2^-11), the scales' and the values' products (2^-11 each), scores and the sum: 2^-9 A + the bound of lse A.
  - What is below fp16's normal numbers: for each token that the row sees at most 2^-30 |code| of the largest scale that
    it sees (codes here are below 8).
"""
from __future__ import annotations

import math

import pytest
import torch

from _gpu import DEV
from test_chunk_attn import E4M3, Step, q4k  # noqa: F401

pytestmark = pytest.mark.gpu
ZERO_SCALE = 2.0 ** -100 / 448


def written(q4k, s, zero):  # noqa: F811
    """The requests' rows written by q4k_kv_write from random keys and values, those of `zero` [(request, first, last)]
    from values of zero."""
    g = torch.Generator().manual_seed(1)
    d = lambda x: x.to(DEV)  # noqa: E731
    k, v, ks, vs = d(s.k), d(s.v), d(s.ks), d(s.vs)
    for r, (length, _) in enumerate(s.both):
        at = torch.arange(length)
        slots = (s.table[r, at // s.page] * s.page + at % s.page).to(torch.int32)
        rows = torch.randn((2, length, s.kv_heads, s.dim), generator=g)
        for _, first, last in [z for z in zero if z[0] == r]:
            rows[1, first:last] = 0.0
        q4k.q4k_kv_write(d(rows[0]), d(rows[1]), d(slots), k, v, ks, vs)
    s.k, s.v, s.ks, s.vs = (x.cpu() for x in (k, v, ks, vs))
    for r, first, _ in zero:
        assert bool((s.vs[s.table[r, first // s.page], :, first % s.page] == torch.tensor(ZERO_SCALE)).all())


def seen_scale(s, window=0):
    """The largest scale of V that each token sees times the number of tokens that it sees, by query head."""
    group = s.q_heads // s.kv_heads
    big = torch.zeros(s.q.shape[:2], dtype=torch.float64)
    for r, (length, new) in enumerate(s.both):
        scales = s.vs[s.table[r, :-(-length // s.page)].long()].transpose(0, 1).flatten(1)[:, :length].double()
        for i in range(new):
            pos = length - new + i
            seen = scales[:, max(0, pos + 1 - window) if window else 0:pos + 1]
            big[int(s.cu[r]) + i] = seen.amax(-1).repeat_interleave(group) * seen.shape[1]
    return big


def check(s, got, scale, window=0):
    out, mass, lse = s.plain(scale, window)
    o, l = got[0].double().cpu(), got[1].double().cpu()
    size = 0.0
    for r, (length, new) in enumerate(s.both):
        for j in range(s.kv_heads):
            group = s.q_heads // s.kv_heads
            q = s.q[int(s.cu[r]):int(s.cu[r]) + new, j * group:(j + 1) * group].double().abs()
            if new:
                size = max(size, scale * float(torch.einsum("tgd,ld->tgl", q, s.rows(r, j, length)[0].abs()).max()))
    tiles = max(a for a, _ in s.both) / 64  # (of 64 or 128)
    part = (s.dim + 8) * 2.0 ** -23 * size + 2.0 ** -16 + (tiles + 40) * 2.0 ** -24
    worst = float(((l - lse).abs() / (part + 2.0 ** -22 * lse.abs())).max())
    assert worst <= 1.0, worst
    small = 2.0 ** -30 * 8 * seen_scale(s, window)[..., None]
    worst = float(((o - out).abs() / (2.0 ** -8 * out.abs() + (2.0 ** -9 + part) * mass + small)).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("zero", [[(0, 0, 128)], [(0, 0, 256)], [(0, 128, 512)], [(0, 512, 900)], [(0, 0, 900)], [(0, 0, 300), (0, 400, 420), (0, 640, 768)]])
def test_tiles_of_zero_values(q4k, dim, zero):  # noqa: F811
    """In front of, behind and between ordinary rows, and alone; weights close to each other."""
    s = Step(50, [(900, 500)], 4, 2, dim, 16, E4M3)
    written(q4k, s, zero)
    for scale in (0.005, dim ** -0.5):
        check(s, s.run(q4k, scale), scale)
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("zero", [[(0, 0, 8000)], [(0, 0, 4000)], [(0, 4000, 8000)], [(0, 1000, 7000)], [(0, 128, 7900)]])
def test_tiles_of_zero_values_in_items_that_are_split(q4k, dim, zero):  # noqa: F811
    s = Step(51, [(8000, 5)], 8, 1, dim, 16, E4M3)
    written(q4k, s, zero)
    check(s, s.run(q4k, 0.005), 0.005)
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("both", [[(1100, 600)], [(5000, 3)]])
@pytest.mark.parametrize("large", [40, 60, 100])
def test_zero_values_before_and_behind_large_ones(q4k, dim, both, large):  # noqa: F811
    """Tokens of zero values keep their weights beside values of 2^40 and far more."""
    for order in (0, 1):
        s = Step(52, both, 4, 1, dim, 16, E4M3)
        length = both[0][0]
        s.v.view(torch.uint8)[0] = 0x7F
        at = torch.arange(length)
        page, place = s.table[0, at // 16].long(), at % 16
        zero = (at < length // 2) if order == 0 else (at >= length // 2)
        s.vs[page, :, place] = torch.where(zero, ZERO_SCALE, 2.0 ** large)[:, None].float()
        s.v.view(torch.uint8)[page[zero], :, place[zero]] = 0
        check(s, s.run(q4k, 0.005), 0.005)


def steps_of(*a, change, **kw):
    """The same step twice, the second one with scales of V changed: change(vs by [request][position])."""
    clean, other = Step(*a, **kw), Step(*a, **kw)
    for r, at, value in change:
        other.vs[other.table[r, at // other.page], :, at % other.page] = value
    return clean, other


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 2), (128, 4, 2), (256, 4, 2), (64, 2, 2), (128, 2, 2), (128, 16, 1)])
@pytest.mark.parametrize("value", [2.0 ** 30, 2.0 ** 60, 2.0 ** 120, 3.4e38, 2.0 ** -100, 1e-40, 0.0, -2.0 ** 60, math.inf, -math.inf, math.nan])
def test_scales_of_later_tokens_stay_out_of_earlier_results(q4k, dim, heads, kv_heads, value):  # noqa: F811
    """Whatever a later token's scale is, earlier tokens have the same bits."""
    both = [(150, 150), (300, 40), (700, 400)]
    places = ((0, 77), (1, 290), (2, 511), (2, 650))
    clean, s = steps_of(53, both, heads, kv_heads, dim, 16, E4M3, change=[(r, at, value) for r, at in places])
    want, got = clean.run(q4k, 0.1), s.run(q4k, 0.1)
    before = torch.cat([torch.arange(77), 150 + torch.arange(30), 190 + torch.arange(211)])
    assert torch.equal(want[0][before], got[0][before]) and torch.equal(want[1][before], got[1][before])
    if 0 < value < 2.0 ** 100:
        check(s, got, 0.1)
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 2), (128, 4, 2), (256, 4, 2), (64, 2, 2), (128, 2, 2), (128, 16, 1)])
@pytest.mark.parametrize("value", [2.0 ** 30, 2.0 ** 120, 2.0 ** -100, math.inf])
def test_scales_before_the_window_stay_out(q4k, dim, heads, kv_heads, value):  # noqa: F811
    """A token's scale does not matter once the window has passed it, nor to tokens before it."""
    window = 200
    clean, s = steps_of(54, [(900, 700)], heads, kv_heads, dim, 16, E4M3, change=[(0, 333, value)])
    want, got = clean.run(q4k, 0.1, window), s.run(q4k, 0.1, window)
    pos = torch.arange(200, 900)
    rows = (pos < 333) | (pos >= 333 + window)
    assert torch.equal(want[0][rows], got[0][rows]) and torch.equal(want[1][rows], got[1][rows])
    if value < 2.0 ** 100:
        check(s, got, 0.1, window)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("both", [[(777, 600)], [(3000, 7)], [(777, 600), (3000, 7)]])
def test_scales_that_rise_and_fall_along_the_positions(q4k, dim, window, both):  # noqa: F811
    """Every row against what it sees itself."""
    for low, high in ((-60.0, 60.0), (60.0, -60.0), (-20.0, 8.0)):
        s = Step(55, both, 4, 2, dim, 16, E4M3)
        for r, (length, _) in enumerate(both):
            at = torch.arange(length)
            s.vs[s.table[r, at // 16].long(), :, at % 16] = torch.exp2(torch.linspace(low, high, length))[:, None]
        check(s, s.run(q4k, 0.1, window), 0.1, window)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_ordinary_scales_with_a_tight_bound(q4k, dim):  # noqa: F811
    both = [(300, 300), (1, 1), (700, 1), (513, 0), (1000, 77), (6000, 9)]
    s = Step(56, both, 8, 2, dim, 32, E4M3)
    check(s, s.run(q4k, dim ** -0.5), dim ** -0.5)
    check(s, s.run(q4k, dim ** -0.5, 130), dim ** -0.5, 130)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 40, 150])
@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (2, 2), (16, 1)])
def test_scales_of_many_orders_from_token_to_token(q4k, dim, window, heads, kv_heads):  # noqa: F811
    """Every row against what it sees itself, where neighbours are up to 2^200 apart; values up to 2^110 in all."""
    g = torch.Generator().manual_seed(2)
    for low, high in ((-80.0, 105.0), (-5.0, 12.0), (90.0, 108.0)):
        s = Step(57, [(500, 400), (1, 1), (40, 40)], heads, kv_heads, dim, 16, E4M3)
        s.vs = torch.exp2(torch.empty(s.vs.shape).uniform_(low, high, generator=g))
        check(s, s.run(q4k, 0.1, window), 0.1, window)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_the_largest_scales(q4k, dim):  # noqa: F811
    """Scales next to the largest number, of values that are not: 2^-9 of 2^127 each."""
    both = [(300, 250)]
    s = Step(58, both, 4, 2, dim, 16, E4M3)
    signs = torch.where(torch.rand(s.v.shape, generator=torch.Generator().manual_seed(3)) < 0.5, -1.0, 1.0)
    s.v = (signs * 2.0 ** -9).to(E4M3)
    s.vs.fill_(2.0 ** 127)
    s.vs[:, :, ::3] = 2.0 ** 100
    check(s, s.run(q4k, 0.1), 0.1)
