"""The table of frequencies against the formula in 60 digits, and far positions against angles computed from it."""
from __future__ import annotations

import math
from decimal import Decimal, getcontext

import pytest
import torch

from _gpu import DEV
from test_decode_ops_abi import L  # noqa: F401

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def turns(rot, base, factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0, factors=None):
    """Turns per position of each pair."""
    base, factor = Decimal(base), Decimal(factor)
    if original:
        at = lambda t: rot * (Decimal(original) / (Decimal(t) * 2 * PI)).ln() / (2 * base.ln())  # noqa: E731
        low = max(0, int(at(beta_fast).to_integral_value("ROUND_FLOOR")))
        high = min(rot - 1, int(at(beta_slow).to_integral_value("ROUND_CEILING")))
        width = max(Decimal(0.001), Decimal(high - low))
    out = []
    for i in range(rot // 2):
        g = (base.ln() * Decimal(-2 * i) / rot).exp()
        if factors is not None:
            g /= Decimal(float(factors[i]))
        keep = 1 - min(Decimal(1), max(Decimal(0), (i - low) / width)) if original else Decimal(0)
        out.append(((1 - keep) * g / factor + keep * g) / (2 * PI))
    return out


CASES = [(128, 1e4), (128, 1e6), (64, 5e5), (256, 1e4), (2, 1e4), (30, 1234.5), (256, 1e30), (254, 3e-5), (0, 10.0), (96, 1.0), (128, 1e4, 4.0), (128, 1e4, 0.3), (128, 1e4, 8.0, 4096), (64, 1e6, 4.0, 32768),
         (128, 5e5, 1.7, 8192, 16.0, 2.0), (100, 2.0, 3.0, 100)]


@pytest.mark.parametrize("case", CASES)
def test_table_is_rounded_once(L, case):  # noqa: F811
    """Each step is the formula's to half a unit of 2^-64 turn (and 2^-85 relative, of sums in twice 64 bits, where a
    frequency is many turns)."""
    import bit_block_quantized_q4_gb300 as q4k
    for factors in (None, torch.linspace(0.07, 61.0, case[0] // 2)):
        steps, _ = q4k.q4k_rope_steps(*case, factors=factors)
        for s, t in zip(steps.tolist(), turns(*case, factors=factors)):
            off = (Decimal(s) - t * 2 ** 64) % 2 ** 64
            off = min(off, 2 ** 64 - off)
            assert off <= Decimal("0.5") + t * Decimal(2) ** (64 - 85), (case, s, t)


@pytest.mark.gpu
@pytest.mark.parametrize("rot,base", [(64, 1e4), (60, 1e6), (128, 5e5)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_against_the_formula(L, rot, base, interleaved):  # noqa: F811
    """Every pair is (1, 0), which turns to the cosine and the sine of its angle: 2^-31 of a turn in the angle, fp32's
    angle, series and product: below 2^-21."""
    import bit_block_quantized_q4_gb300 as q4k
    pos = [1, 2 ** 20 + 1, 131071, 2 ** 24 - 1, 2 ** 30 + 12345, 2 ** 31 - 1]
    x = torch.zeros((len(pos), 1, 128), device=DEV)
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    x[:, 0, first] = 1.0
    steps, _ = q4k.q4k_rope_steps(rot, base)
    got = q4k.q4k_rope(x, torch.tensor(pos, dtype=torch.int32, device=DEV), steps.to(DEV), interleaved=interleaved, out_dtype=torch.float32).double().cpu()
    want = torch.zeros_like(got)
    for p, at in enumerate(pos):
        for i, t in enumerate(turns(rot, base)):
            angle = 2 * math.pi * float(t * at % 1)
            a = int(first[i])
            want[p, 0, a], want[p, 0, a + 1 if interleaved else a + rot // 2] = math.cos(angle), math.sin(angle)
    assert float((got - want).abs().max()) <= 2.0 ** -21
