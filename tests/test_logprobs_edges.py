"""Scores of rows whose tokens lie beside the aligned vectors, of logits far from zero.

Tolerances: as in test_logprobs: a sum good to 2^-17 per 131072 logits, a logarithm and a difference that are rounded.
"""
from __future__ import annotations

import pytest
import torch

from _gpu import DEV
from test_logprobs import check, q4k  # noqa: F401

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
