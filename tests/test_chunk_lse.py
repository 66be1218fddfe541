"""The logarithm of the sum of weights of chunk attention over a bf16 cache, with a bound that counts what fp32 leaves.

S = softmax_scale max sum |q||k| bounds a score, which is off by (D + 8) 2^-23 S (D additions in the tensor cores, two
products); a sum of T tiles of 128 weights good to 2^-21 is off by (T + 34) 2^-24 + 2^-21; the reference, of at most 2 S
in binary orders, and the logarithm are rounded: (S + 8) 2^-22 and 2^-22 |lse|.
"""
from __future__ import annotations

import pytest
import torch

from test_chunk_attn import Step, q4k  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("both,window", [([(300, 300), (1, 1), (700, 1), (1000, 77)], 0), ([(6000, 9)], 0), ([(2000, 900)], 333), ([(1, 1)] * 50, 0)])
@pytest.mark.parametrize("scale", [0.003, 0.1])
def test_the_logarithm_of_the_sum(q4k, dim, both, window, scale):  # noqa: F811
    s = Step(60, both, 8, 2, dim, 16)
    lse = s.plain(scale, window)[2]
    size = 0.0
    for r, (length, new) in enumerate(both):
        q = s.q[int(s.cu[r]):int(s.cu[r]) + new].double().abs()
        size = max([size] + [scale * float(torch.einsum("tgd,ld->tgl", q[:, 4 * j:4 * j + 4], s.rows(r, j, length)[0].abs()).max()) for j in range(2)])
    got = s.run(q4k, scale, window)[1].double().cpu()
    tiles = max(a for a, _ in both) / 64
    bound = (dim + 8) * 2.0 ** -23 * size + (tiles + 34) * 2.0 ** -24 + 2.0 ** -21 + (size + 8) * 2.0 ** -22 + 2.0 ** -22 * lse.abs()
    worst = float(((got - lse).abs() / bound).max())
    assert worst <= 1.0, worst
