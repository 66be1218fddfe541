"""The operators around the projections at the ends of their ranges: empty steps, lengths past the table,
weights far below the largest, pipelines that run long enough to refill every stage, and what the pointer
checks refuse.

Tolerances count roundings: half a step of a type is eps / 2 relative (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from _gpu import DEV
from test_decode_ops import plain_plan

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
