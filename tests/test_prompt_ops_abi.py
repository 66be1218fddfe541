"""Refusals of the entry points of a prompt (attention of chunks): every argument error comes back before a device
is touched, so these run without one."""
from __future__ import annotations

import pytest
import torch

from test_decode_ops_abi import ALIGN, CACHE, CACHE_REFUSALS, L, NULL, OK, ORDERS, P, SHAPE, WORKSPACE, _call, _strides  # noqa: F401

CHUNK = dict(q=P, ldq=1024, ldq_head=128, tokens=9, cu=P, n=4, q_heads=8, heads=8, dim=128, k_cache=P, v_cache=P, **CACHE, k_scale=None, v_scale=None,
             table=P, ldt=8, max_pages=8, lens=P, scale=0.1, window=0, out=P, ldo=1024, lse=None, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(page=8, page_stride=1 << 20), SHAPE), (dict(page=512, page_stride=1 << 20, head_stride=1 << 17), SHAPE), (dict(page=24, head_stride=24 * 128, page_stride=1 << 20), SHAPE),
    (dict(n=-1), SHAPE), (dict(n=65537), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 28), SHAPE), (dict(q_heads=12), SHAPE), (dict(q_heads=2048), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(max_pages=1 << 27, ldt=1 << 27), SHAPE), (dict(ldt=7), SHAPE), (dict(cache_dtype=2, k_scale=P + 8, v_scale=P), ALIGN), (dict(window=-1), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(ldq_head=64), SHAPE), (dict(ldq=-8), SHAPE), (dict(ldo=1016), SHAPE), (dict(n=0, q=None), OK), (dict(tokens=0, q=None), OK), (dict(q=None), NULL),
    (dict(cu=None), NULL), (dict(k_cache=None), NULL), (dict(v_cache=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL), (dict(cache_dtype=2, k_scale=P), NULL),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=0), WORKSPACE), (dict(q=P + 8), ALIGN), (dict(cu=P + 4), ALIGN), (dict(ldq=1028), ALIGN), (dict(ldq_head=132), ALIGN), (dict(ldo=1028), ALIGN), (dict(lens=P + 2), ALIGN),
    (dict(ws=P + 8), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_chunk_refusals(L, change, status):  # noqa: F811
    assert _call(L.q4k_paged_attn_chunk, CHUNK, **change) == status


@pytest.mark.parametrize("order", ORDERS)
def test_chunk_cache_strides_in_any_order(L, order):  # noqa: F811
    good = _strides(order)
    assert _call(L.q4k_paged_attn_chunk, CHUNK, **good) not in (OK, NULL, SHAPE, ALIGN, WORKSPACE)
    for name in good:
        assert _call(L.q4k_paged_attn_chunk, CHUNK, **{**good, name: good[name] - 8}) == SHAPE


def test_chunk_workspace_is_what_the_call_asks_for(L):  # noqa: F811
    size = L.q4k_paged_attn_chunk_workspace_size(9, 8, 8, 128)
    assert 0 < size <= L.q4k_paged_attn_chunk_workspace_size(900, 8, 8, 128) == L.q4k_paged_attn_chunk_workspace_size(1 << 20, 8, 8, 128)
    assert _call(L.q4k_paged_attn_chunk, CHUNK, ws_bytes=size - 1) == WORKSPACE
    assert _call(L.q4k_paged_attn_chunk, CHUNK, ws_bytes=size) not in (OK, NULL, SHAPE, ALIGN, WORKSPACE)
    for bad in ((-1, 8, 8, 128), (9, 0, 8, 128), (9, 8, 0, 128), (9, 8, 8, 0), (1 << 40, 8, 8, 128)):
        assert L.q4k_paged_attn_chunk_workspace_size(*bad) == 0


def test_chunk_binding_refuses_wrong_types_shapes_and_layouts(L):  # noqa: F811
    import bit_block_quantized_q4_gb300 as q4k
    z = torch.zeros
    cache = z((4, 2, 16, 64), dtype=torch.bfloat16)
    lens, cu, table, q = z(2, dtype=torch.int32), z(3, dtype=torch.int64), z((2, 3), dtype=torch.int32), z((5, 4, 64), dtype=torch.bfloat16)
    call = q4k.q4k_paged_attn_chunk
    for bad in (lambda: call(q.float(), cache, cache, table, lens, cu, 1.0), lambda: call(q, cache, cache.float(), table, lens, cu, 1.0),
                lambda: call(q, cache, cache[:, :, :, ::2], table, lens, cu, 1.0), lambda: call(q, cache, cache, table, lens, cu.int(), 1.0),
                lambda: call(q, cache, cache, table, lens, cu[:2], 1.0), lambda: call(q, cache, cache, table, lens[:1], cu, 1.0),
                lambda: call(q, cache, cache, table.long(), lens, cu, 1.0), lambda: call(q[:, :, :32], cache, cache, table, lens, cu, 1.0),
                lambda: call(q, cache, cache, table, lens, cu, 1.0, out=q[:4]), lambda: call(q, cache, cache, table, lens, cu, 1.0, lse=z((4, 5)))):
        with pytest.raises(q4k.Q4KError) as e:
            bad()
        assert e.value.status == SHAPE
