"""Chunk attention and the rotated cache write where they can go wrong: pages that are absent at every head size, one token
alone, two calls at once, many requests, pages beyond 4 GB."""
from __future__ import annotations

import math

import pytest
import torch

from _gpu import DEV
from test_chunk_attn import BAD_PAGE, BF16, E4M3, Step, q4k  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 64), (256, 16), (256, 64)])
def test_absent_pages_at_other_head_sizes(q4k, cache, dim, page):  # noqa: F811
    s = Step(30, [(9 * page + 5, 30), (3 * page, 7)], 4, 2, dim, page, cache)
    good = s.table.clone()
    gone = {0: [2, 7], 1: [0]}
    for r, pages in gone.items():
        s.table[r, pages] = torch.tensor([-1, 10 ** 6], dtype=torch.int32)[:len(pages)]
    got = s.run(q4k, 0.1)
    assert q4k.q4k_get_device_error() == BAD_PAGE
    s.table = good
    for r, (length, new) in enumerate(s.both):
        at, pos = torch.arange(length), torch.arange(length - new, length)
        keep = ~torch.isin(at // page, torch.tensor(gone[r]))
        rows = slice(int(s.cu[r]), int(s.cu[r]) + new)
        for j in range(2):
            k, v = s.rows(r, j, length)
            z = 0.1 * torch.einsum("tgd,ld->tgl", s.q[rows, 2 * j:2 * j + 2].double(), k)
            z = torch.where(((at[None] <= pos[:, None]) & keep[None])[:, None], z, -math.inf)
            w = torch.softmax(z, -1)
            out, mass = torch.einsum("tgl,ld->tgd", w, v), torch.einsum("tgl,ld->tgd", w, v.abs())
            # roundings of the result, of weights, and of scores, as test_chunk_attn counts them
            bound = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -9) * mass
            assert bool(((got[0][rows, 2 * j:2 * j + 2].double().cpu() - out).abs() <= bound).all()), (r, j)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_token_alone_gives_its_value(q4k, dim):  # noqa: F811
    s = Step(31, [(1, 1)] * 40, 4, 2, dim, 16)
    out, lse = s.run(q4k, 0.3)
    for r in range(40):
        k, v = (c[s.table[r, 0].long(), :, 0] for c in (s.k, s.v))
        assert torch.equal(out[r].cpu(), v.repeat_interleave(2, 0))  # a weight of exactly 1
        z = 0.3 * (s.q[r].double() * k.repeat_interleave(2, 0).double()).sum(-1)
        # dim additions in fp32 of terms whose sum of sizes is below 2^7, times 0.3, and the logarithm's rounding
        assert float((lse[r].double().cpu() - z).abs().max()) <= 2.0 ** -10


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_two_calls_at_once(q4k, cache):  # noqa: F811
    steps = [Step(32, [(3000, 700), (50, 50)], 8, 2, 128, 16, cache), Step(33, [(4000, 2), (900, 900)], 4, 4, 64, 32, cache)]
    want = [[x.clone() for x in s.run(q4k, 0.1)] for s in steps]
    d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    args = [[d(x) for x in (s.q, s.k, s.v, s.table, s.lens, s.cu)] for s in steps]
    scales = [(d(s.ks), d(s.vs)) for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    outs = [[torch.full_like(args[i][0], 7.0) for _ in range(10)] for i in range(2)]
    torch.cuda.synchronize()
    for n in range(10):
        for i in range(2):
            q4k.q4k_paged_attn_chunk(*args[i], 0.1, *scales[i], out=outs[i][n], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) for o in outs[i])
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_many_requests_with_and_without_tokens(q4k, cache):  # noqa: F811
    g = torch.Generator().manual_seed(34)
    lens = torch.randint(0, 90, (2000,), generator=g).tolist()
    both = [(n, int(n > 0 and i % 3 > 0) * min(n, 1 + i % 5)) for i, n in enumerate(lens)]
    s = Step(35, both, 4, 2, 64, 16, cache, pad=3)
    got = s.run(q4k, 0.125)
    s.check(got, 0.125)
    t = int(s.cu[-1])
    assert bool((got[0][t:] == 7).all()) and bool((got[1][t:] == 7).all())
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_pages_beyond_4_gb(q4k, cache):  # noqa: F811
    """Keys and values are rotated and written to pages of which the last lie 5 * 2^30 elements into the caches, and read
    there: the same bits as with pages side by side."""
    pages, heads, page, dim = 6, 2, 16, 128
    stride = 2 ** 30
    far = [torch.empty(5 * stride + heads * page * dim, dtype=torch.uint8 if cache == E4M3 else BF16, device=DEV)
           .as_strided((pages, heads, page, dim), (stride, page * dim, dim, 1)).view(cache) for _ in range(2)]
    near = [torch.zeros((pages, heads, page, dim), dtype=torch.uint8 if cache == E4M3 else BF16, device=DEV).view(cache) for _ in range(2)]
    tokens = 40
    g = torch.Generator().manual_seed(36)
    qkv = torch.randn((tokens, 8 + 2 * heads, dim), generator=g).to(DEV)
    table = torch.tensor([[5, 0, 4]], dtype=torch.int32, device=DEV)
    pos = torch.arange(tokens, dtype=torch.int32, device=DEV)
    slots = (table[0, (pos // page).long()] * page + pos % page).to(torch.int32)
    steps = q4k.q4k_rope_steps(dim, 1e4)[0].to(DEV)
    lens = torch.tensor([tokens], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, tokens], device=DEV)
    got = []
    for k, v in (far, near):
        scales = [torch.ones((pages, heads, page), device=DEV) for _ in range(2)] if cache == E4M3 else [None, None]
        q = q4k.q4k_rope_kv_write(qkv[:, :8], qkv[:, 8:8 + heads], qkv[:, 8 + heads:], pos, slots, steps, k, v, *scales)
        got.append((q, *q4k.q4k_paged_attn_chunk(q, k, v, table, lens, cu, 0.09, *scales)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    # and they are the rotated attention: the last token's, plainly
    x = qkv.double().cpu()
    angle = pos.double().cpu()[:, None, None] * 1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)
    turn = lambda y: torch.cat((y[..., :64] * angle.cos() - y[..., 64:] * angle.sin(), y[..., :64] * angle.sin() + y[..., 64:] * angle.cos()), -1)  # noqa: E731
    qr, kr, v = turn(x[:, :8]), turn(x[:, 8:8 + heads]), x[:, 8 + heads:]
    w = torch.softmax(0.09 * torch.einsum("hd,thd->ht", qr[-1], kr.repeat_interleave(4, 1)), -1)
    want = torch.einsum("ht,thd->hd", w, v.repeat_interleave(4, 1))
    # q, k, v and the result are rounded to bf16 (an e4m3 cache: k and v by 2^-4): of scores of size 0.09 |q||k| ~ 12
    part = 2.0 ** -8 * 4 + 2.0 ** -8 * 12 if cache == BF16 else (2.0 ** -8 + 2.0 ** -4) * 3
    assert float((got[0][1][-1].double().cpu() - want).norm() / want.norm()) <= part
    assert q4k.q4k_get_device_error() == 0


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("dim,heads,kv_heads,window", [(128, 8, 2, 200), (64, 8, 2, 200), (256, 8, 2, 200), (128, 32, 1, 0), (128, 64, 1, 0), (64, 32, 1, 130)])
def test_values_that_are_not_finite_show_in_every_token_that_sees_them(q4k, cache, dim, heads, kv_heads, window):  # noqa: F811
    """Also in those that see the whole tile of keys beside others that do not."""
    s = Step(37, [(400, 300), (257, 1)], heads, kv_heads, dim, 16, cache)
    clean = [x.clone() for x in s.run(q4k, 0.1, window)]
    for token in (5, 127, 128, 255, 399):
        s2 = Step(37, [(400, 300), (257, 1)], heads, kv_heads, dim, 16, cache)
        raw = s2.v.view(torch.uint8) if cache == E4M3 else s2.v
        raw[s2.table[0, token // 16].long(), 0, token % 16, dim // 2] = 0x7F if cache == E4M3 else math.nan
        out, lse = s2.run(q4k, 0.1, window)
        pos = torch.arange(100, 400)
        sees = (token <= pos) & ((token > pos - window) if window else True)
        group = heads // kv_heads
        mine = out[:300, :group]
        assert bool(torch.isnan(mine[sees.to(DEV)][..., dim // 2]).all()), token
        assert torch.equal(mine[~sees.to(DEV)], clean[0][:300, :group][~sees.to(DEV)]), token
        assert torch.equal(out[:, group:], clean[0][:, group:]) and torch.equal(out[300:], clean[0][300:])
    assert q4k.q4k_get_device_error() == 0
