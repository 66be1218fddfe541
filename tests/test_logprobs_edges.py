"""Scores of rows whose tokens lie beside the aligned vectors, of logits far from zero and next to the
largest number, and of the largest vocabulary.

Tolerances: as in test_logprobs: a sum good to 2^-17 per 131072 logits, a logarithm and a difference that are rounded.
"""
from __future__ import annotations

import math

import pytest
import torch

from _gpu import DEV
from test_logprobs import BF16, F32, check, near, plain, q4k  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [0.0, 100.0, -1e4, 1e6, -1e6, 4194303.0, -4194303.75, -4194304.0, 4194304.0, 1e7, -1e7])
@pytest.mark.parametrize("vocab,offset,top", [(1, 0, 1), (3, 0, 3), (5, 1, 5), (7, 3, 2), (13, 3, 4), (30, 1, 9), (2503, 1, 20), (9001, 3, 5)])
def test_tokens_beside_the_vectors_of_far_logits(q4k, vocab, offset, top, shift):  # noqa: F811
    """Differences of a few units, exact in fp32 at every shift."""
    g = torch.Generator().manual_seed(vocab)
    rows, ld = 6, vocab + offset + 4
    wide = torch.zeros(rows * ld + 8, device=DEV)
    x = wide.as_strided((rows, vocab), (ld, 1), offset)
    x.copy_(torch.randint(-16, 1, (rows, vocab), generator=g) * 0.5 + shift)
    tokens = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32)
    check(q4k.q4k_logprobs(x, tokens.to(DEV), top=top), x, tokens, top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [40, 3000, 131072])
def test_infinite_logits_behind_the_largest_finite_ones(q4k, dtype, vocab):  # noqa: F811
    """A thread's tokens: i, i + 2048, ...: the largest numbers in its first vectors, infinities in later ones and in the
    same one, beside masked tokens and NaN."""
    x = torch.randn((5, vocab), generator=torch.Generator().manual_seed(1)).to(dtype)
    large = torch.finfo(dtype).max
    x[0, :vocab // 2] = large
    x[0, -7:] = math.inf
    x[1, 8:16], x[1, vocab - 3] = large, math.inf
    x[2, 3], x[2, 4], x[2, -1] = large, math.inf, math.inf
    x[3], x[3, vocab // 2:] = -large, large
    x[3, 5], x[3, 1:9:2] = math.inf, math.nan
    x[4], x[4, ::3] = large, -math.inf
    x = x.to(DEV)
    tokens = torch.tensor([vocab - 1, 9, 3, 5, 1], dtype=torch.int32)
    check(q4k.q4k_logprobs(x, tokens.to(DEV), top=9), x, tokens, 9)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_largest_vocabulary(q4k, dtype):  # noqa: F811
    vocab = 1 << 24
    x = torch.randn((1, vocab), generator=torch.Generator().manual_seed(2)) * 3
    x = x.to(dtype).to(DEV)
    x[0, 5::7] = -math.inf
    tokens = torch.tensor([vocab - 1], dtype=torch.int32)
    got, want = q4k.q4k_logprobs(x, tokens.to(DEV), top=32), plain(x, tokens, 32)
    assert torch.equal(got[1].cpu().long(), want[1]) and torch.equal(got[3].cpu().long(), want[3])
    # each of two sums of a thread has 2^24 / 8 / 256 / 2 terms one after the other: 2^12 times 2^-24
    near(got[0], want[0], 2.0 ** -11)
    near(got[4], want[4], 2.0 ** -11)
