"""The operators around the projections at the ends of their ranges: empty steps, lengths past the table,
weights far below the largest, pipelines that run long enough to refill every stage, and what the pointer
checks refuse.

Tolerances count roundings: half a step of a type is eps / 2 relative (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4).
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from _gpu import DEV
from test_decode_ops import BAD_PAGE, BF16, E4M3, make_attn, plain_attn, plain_plan, to_dev

gpu = pytest.mark.gpu
NULL, SHAPE, ALIGN, MEMORY = 1, 2, 3, 8


@pytest.fixture(scope="module")
def q4k():
    from bit_block_quantized_q4_gb300 import build
    build.build()
    import bit_block_quantized_q4_gb300 as m
    return m


# ------------------------------------------------------------------------------------------ plan without requests


@gpu
@pytest.mark.parametrize("n_slots", [0, 1, 37, 5000, 20000])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_of_no_requests_writes_what_is_defined(q4k, n_slots, in_place):
    """No request: the state as it is (brought into the ring), cu[0] = 0, every slot and position -1."""
    for head, count in ((3, 7), (-5, 77), (0, 0)):
        pool, table = np.arange(20, dtype=np.int32), np.zeros((0, 6), np.int32)
        none = torch.zeros(0, dtype=torch.int32, device=DEV)
        state = torch.tensor([head, count], dtype=torch.int32, device=DEV)
        dp, dt = torch.from_numpy(pool).to(DEV), torch.zeros((0, 6), dtype=torch.int32, device=DEV)
        cu = torch.full((1,), 99, dtype=torch.int64, device=DEV)
        slots, pos = (torch.full((n_slots,), 5, dtype=torch.int32, device=DEV) for _ in range(2))
        state_out = state if in_place else torch.full((2,), -7, dtype=torch.int32, device=DEV)
        q4k.q4k_kv_plan(none, none, dt, dp, state, 16, n_slots, out=(none, cu, slots, pos, none, state_out))
        want = plain_plan(np.zeros(0, np.int32), np.zeros(0, np.int32), table, pool, np.array([head, count]), 16, n_slots)
        assert cu.tolist() == want[1].tolist() == [0]
        assert bool((slots == -1).all()) and bool((pos == -1).all())
        assert state_out.tolist() == want[5].tolist()
        assert in_place or state.tolist() == [head, count]
        assert np.array_equal(dp.cpu().numpy(), pool)
        got = q4k.q4k_kv_plan(none, none, dt, dp, torch.tensor([head, count], dtype=torch.int32, device=DEV), 16, n_slots)
        for g, w in zip(got, want[:6]):
            assert np.array_equal(g.cpu().numpy(), w)
    assert q4k.q4k_get_device_error() == 0


def test_plan_of_no_requests_refusals(q4k):
    """Without requests the arrays of requests may be NULL; what is written may not, nor be host memory."""
    from test_decode_ops_abi import PLAN, _call
    L = q4k.lib()
    per_request = dict(n=0, lens=None, add=None, table=None, lens_out=None, status=None)
    for name in ("state", "cu", "state_out", "slots", "pos"):
        assert _call(L.q4k_kv_plan, PLAN, **{**per_request, name: None}) == NULL
    assert _call(L.q4k_kv_plan, PLAN, **per_request, cu=PLAN["cu"] + 4) == ALIGN
    assert _call(L.q4k_kv_plan, PLAN, **per_request, max_pages=0) == SHAPE
    for extra in ({}, dict(n_slots=0, slots=None, pos=None)):  # nothing refused before the device is asked
        assert _call(L.q4k_kv_plan, PLAN, **per_request, **extra) not in (NULL, SHAPE, ALIGN)
    none, state = torch.zeros(0, dtype=torch.int32), torch.tensor([3, 7], dtype=torch.int32)
    with pytest.raises(q4k.Q4KError) as e:  # on host tensors it would leave its outputs unwritten
        q4k.q4k_kv_plan(none, none, torch.zeros((0, 4), dtype=torch.int32), torch.zeros(9, dtype=torch.int32), state, 16, 3)
    assert e.value.status == MEMORY


# ------------------------------------------------------------------------------------------ window and lengths past the table


@gpu
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("dim,q_heads,kv_heads,page", [(128, 8, 2, 16), (64, 6, 1, 64), (256, 4, 2, 32)])
def test_attn_window_of_lengths_past_the_table(q4k, dim, q_heads, kv_heads, page, kind):
    """The window ends at the length, not at the table's end: tokens max(0, len - window) <= j < len, of which
    those past the table are absent."""
    cap = 512
    top = 2 ** 31 - 1
    for window in (0, 1, 100, 488, 489, 600, 1000, top - 500, top - 512, top):
        raw = [1000, 300, cap, top, 513, 0, 1100]
        c = make_attn(31, [min(v, cap) for v in raw], q_heads, kv_heads, dim, page, kind, extra=0)
        assert c["table"].shape[1] * page == cap
        caches = [to_dev(x, kind) for x in c["caches"]]
        scales = [s.to(DEV) for s in c["scales"]] if c["scales"] else [None, None]
        lens = torch.tensor(raw, dtype=torch.int32, device=DEV)
        out, lse = q4k.q4k_paged_attn(c["q"].to(DEV), *caches, c["table"].to(DEV), lens, dim ** -0.5, *scales, window=window)
        assert q4k.q4k_get_device_error() == BAD_PAGE
        want, wl, bo, bl = plain_attn(c, dim ** -0.5, skip=lambda r, n: torch.arange(n) < (raw[r] - window if window else 0))
        assert bool(((out.double().cpu() - want).abs() <= bo).all()), window
        lse = lse.double().cpu()
        assert torch.equal(lse == -math.inf, wl == -math.inf), window
        fin = wl != -math.inf
        assert bool(((lse - wl)[fin].abs() <= bl[fin]).all()), window
