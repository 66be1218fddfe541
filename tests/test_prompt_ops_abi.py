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


ROPE = dict(x=P, x_dtype=0, ld_token=1024, ld_head=128, tokens=9, heads=8, dim=128, gamma=P, eps=1e-6, pos=P, steps=P, rot=128, interleaved=0, amplitude=1.0, y=P, y_dtype=1, ldy_token=1024, ldy_head=128, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x_dtype=2), SHAPE), (dict(y_dtype=2), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE), (dict(dim=0), SHAPE), (dict(dim=264, ld_head=264, ldy_head=264), SHAPE),
    (dict(dim=100), SHAPE), (dict(rot=-2), SHAPE), (dict(rot=130), SHAPE), (dict(rot=33), SHAPE), (dict(interleaved=2), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(amplitude=float("inf")), SHAPE),
    (dict(ld_head=64), SHAPE), (dict(ld_token=-8), SHAPE), (dict(ldy_head=64), SHAPE), (dict(ldy_token=512), SHAPE), (dict(ldy_token=64), SHAPE), (dict(ldy_token=0), SHAPE), (dict(ldy_token=128, ldy_head=1024), SHAPE), (dict(tokens=0, x=None), OK), (dict(x=None), NULL), (dict(pos=None), NULL),
    (dict(steps=None), NULL), (dict(y=None), NULL), (dict(x=P + 8), ALIGN), (dict(y=P + 8), ALIGN), (dict(gamma=P + 4), ALIGN), (dict(pos=P + 2), ALIGN), (dict(steps=P + 4), ALIGN), (dict(ld_token=1028), ALIGN), (dict(ldy_head=132, ldy_token=2048), ALIGN)])
def test_rope_refusals(L, change, status):  # noqa: F811
    assert _call(L.q4k_rope, ROPE, **change) == status


@pytest.mark.parametrize("change", [dict(steps=None, rot=0), dict(gamma=None, eps=-1.0), dict(ldy_token=128, ldy_head=1152), dict(ld_token=0), dict(tokens=1, ldy_token=0)])
def test_rope_calls_that_are_allowed(L, change):  # noqa: F811
    assert _call(L.q4k_rope, ROPE, **change) not in (OK, NULL, SHAPE, ALIGN, WORKSPACE)  # (there is no device)


FUSED = dict(q=P, ldq_token=2048, ldq_head=128, k=P, v=P, ld_token=2048, ld_head=128, dtype=0, tokens=9, q_heads=8, heads=8, dim=128, q_gamma=P, k_gamma=P, eps=1e-6, pos=P, slots=P, steps=P, rot=128, interleaved=0, amplitude=1.0,
             q_out=P, ldo_token=1024, ldo_head=128, k_cache=P, v_cache=P, **CACHE, k_scale=None, v_scale=None, stream=None)


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(dtype=2), SHAPE), (dict(tokens=-1), SHAPE), (dict(q_heads=0), SHAPE), (dict(q_heads=1025), SHAPE), (dict(rot=130), SHAPE), (dict(rot=3), SHAPE), (dict(interleaved=-1), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(amplitude=float("nan")), SHAPE), (dict(ldq_head=64), SHAPE), (dict(ld_head=64), SHAPE), (dict(ld_token=-8), SHAPE), (dict(ldo_head=64), SHAPE), (dict(ldo_token=512), SHAPE), (dict(tokens=0, q=None), OK),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(pos=None), NULL), (dict(slots=None), NULL), (dict(steps=None), NULL), (dict(q_out=None), NULL), (dict(k_cache=None), NULL), (dict(v_cache=None), NULL),
    (dict(cache_dtype=2), NULL), (dict(cache_dtype=2, k_scale=P), NULL), (dict(q=P + 8), ALIGN), (dict(k=P + 8), ALIGN), (dict(v=P + 8), ALIGN), (dict(q_gamma=P + 4), ALIGN), (dict(k_gamma=P + 4), ALIGN), (dict(pos=P + 2), ALIGN),
    (dict(slots=P + 2), ALIGN), (dict(steps=P + 4), ALIGN), (dict(q_out=P + 8), ALIGN), (dict(v_cache=P + 8), ALIGN), (dict(ldq_token=2052), ALIGN), (dict(ld_token=2052), ALIGN), (dict(ldo_token=1028), ALIGN)])
def test_rope_kv_write_refusals(L, change, status):  # noqa: F811
    assert _call(L.q4k_rope_kv_write, FUSED, **change) == status


SCORE = dict(logits=P, dtype=0, rows=2, vocab=100, ld=100, tokens=P, top=5, logp=P, rank=P, entropy=P, top_tokens=P, top_logp=P, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=(1 << 24) + 1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=(1 << 24) + 1, ld=1 << 25), SHAPE), (dict(ld=99), SHAPE), (dict(top=-1), SHAPE), (dict(top=33), SHAPE),
    (dict(rows=0, logits=None), OK), (dict(logits=None), NULL), (dict(tokens=None), NULL), (dict(logp=None), NULL), (dict(top_tokens=None), NULL), (dict(top_logp=None), NULL), (dict(logits=P + 2), ALIGN), (dict(dtype=1, logits=P + 1), ALIGN),
    (dict(tokens=P + 2), ALIGN), (dict(logp=P + 1), ALIGN), (dict(rank=P + 2), ALIGN), (dict(entropy=P + 2), ALIGN), (dict(top_tokens=P + 2), ALIGN), (dict(top_logp=P + 2), ALIGN)])
def test_logprobs_refusals(L, change, status):  # noqa: F811
    assert _call(L.q4k_logprobs, SCORE, **change) == status


def test_logprobs_outputs_that_may_be_left_out(L):  # noqa: F811
    for change in (dict(rank=None), dict(entropy=None), dict(top=0, top_tokens=None, top_logp=None)):
        assert _call(L.q4k_logprobs, SCORE, **change) not in (OK, NULL, SHAPE, ALIGN, WORKSPACE)


def test_rope_steps(L):  # noqa: F811
    import math

    import bit_block_quantized_q4_gb300 as q4k
    for rot, base in ((128, 10000.0), (64, 1e6), (2, 500000.0), (0, 10.0), (30, 1e4)):
        steps, amplitude = q4k.q4k_rope_steps(rot, base)
        assert amplitude == 1.0 and len(steps) == rot // 2 and steps.dtype == torch.int64
        for i, s in enumerate(steps.tolist()):
            f = (int(s) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi
            # a power, two products and two roundings in 64 bits; the table's own rounding is half a unit, 2^-65 turns
            assert abs(f - base ** (-2 * i / rot)) <= 2.0 ** -49 * f + 2.0 ** -65 * 2 * math.pi
    plain, _ = q4k.q4k_rope_steps(128, 10000.0)
    slow, amplitude = q4k.q4k_rope_steps(128, 10000.0, 8.0)
    assert amplitude == 1.0
    unit = lambda a: 2.0 ** -49 + 2.0 / a  # noqa: E731  (a ratio of two whole numbers that are off by half a unit)
    for a, b in zip(plain.tolist(), slow.tolist()):
        assert abs(b / a - 1 / 8) <= unit(a)
    # only slow pairs are scaled; pair i turns original / (2 pi) base^(-2 i / 128) times over 4096 positions
    mixed, amplitude = q4k.q4k_rope_steps(128, 10000.0, 8.0, 4096)
    assert abs(amplitude - (1 + 0.1 * math.log(8.0))) <= 2.0 ** -23
    turns = [4096 / (2 * math.pi) * 10000.0 ** (-2 * i / 128) for i in range(64)]
    low, high = max(i for i in range(64) if turns[i] >= 32), min(i for i in range(64) if turns[i] <= 1)
    ratio = [b / a for a, b in zip(plain.tolist(), mixed.tolist())]
    assert all(abs(r - 1) <= unit(a) for r, a in zip(ratio[:low + 1], plain.tolist())) and all(abs(r - 1 / 8) <= unit(a) for r, a in zip(ratio[high:], plain.tolist()[high:]))
    assert all(a >= b - unit(c) - unit(d) for a, b, c, d in zip(ratio, ratio[1:], plain.tolist(), plain.tolist()[1:]))
    given, _ = q4k.q4k_rope_steps(8, 100.0, factors=torch.tensor([1.0, 2.0, 4.0, 0.5]))
    base4, _ = q4k.q4k_rope_steps(8, 100.0)
    assert [round(b / a, 12) for a, b in zip(base4.tolist(), given.tolist())] == [1.0, 0.5, 0.25, 2.0]
    # a frequency of a turn and more counts modulo a turn
    fast, _ = q4k.q4k_rope_steps(2, 10.0, factors=torch.tensor([0.05]))
    assert abs((int(fast[0]) % 2 ** 64) / 2.0 ** 64 - (1 / float(torch.tensor(0.05)) / (2 * math.pi)) % 1.0) <= 2.0 ** -45
    for bad in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=258), dict(base=0.0), dict(base=float("nan")), dict(factor=0.0), dict(factor=float("inf")), dict(original=-1), dict(original=10, base=1.0),
                dict(original=10, beta_fast=0.0), dict(original=10, beta_slow=-1.0), dict(factors=torch.zeros(32)), dict(factors=torch.ones(31)), dict(factors=torch.ones(32).double())):
        with pytest.raises(q4k.Q4KError) as e:
            q4k.q4k_rope_steps(**{**dict(rot_dim=64, base=1e4), **bad})
        assert e.value.status == SHAPE


def test_rope_and_logprobs_bindings_refuse_wrong_types_shapes_and_layouts(L):  # noqa: F811
    import bit_block_quantized_q4_gb300 as q4k
    z = torch.zeros
    x, pos, steps = z((3, 4, 64)), z(3, dtype=torch.int32), z(32, dtype=torch.int64)
    cache, k = z((4, 2, 16, 64), dtype=torch.bfloat16), z((3, 2, 64))
    write = lambda *a, **kw: q4k.q4k_rope_kv_write(*a, cache, cache, **kw)  # noqa: E731
    for bad in (lambda: q4k.q4k_rope(x.half(), pos, steps), lambda: q4k.q4k_rope(x[0], pos, steps), lambda: q4k.q4k_rope(x, pos.long(), steps), lambda: q4k.q4k_rope(x, pos[:2], steps), lambda: q4k.q4k_rope(x, pos, steps.int()),
                lambda: q4k.q4k_rope(x, pos, z(33, dtype=torch.int64)), lambda: q4k.q4k_rope(x, pos, steps, gamma=z(32)), lambda: q4k.q4k_rope(x[:, :, ::2], pos, steps), lambda: q4k.q4k_rope(x, pos, steps, out=x[:2]),
                lambda: q4k.q4k_rope(x, pos, steps, out_dtype=torch.float16),
                lambda: write(x, k.bfloat16(), k, pos, pos, steps), lambda: write(x, k, k[:, :1], pos, pos, steps), lambda: write(x, x, x, pos, pos, steps), lambda: write(x, k, k, pos, pos[:2], steps),
                lambda: write(x, k, k, pos, pos, steps, out=x), lambda: write(x, k, k, pos, pos, steps, q_gamma=z(64).double()),
                lambda: q4k.q4k_logprobs(x[0].half(), pos), lambda: q4k.q4k_logprobs(x[0], pos), lambda: q4k.q4k_logprobs(x[:, 0], pos.long()), lambda: q4k.q4k_logprobs(x[:, 0], pos, top=33),
                lambda: q4k.q4k_logprobs(x[:, 0], pos, logp=z(4)), lambda: q4k.q4k_logprobs(x[:, 0], pos, top=2, top_tokens=z((3, 2)))):
        with pytest.raises(q4k.Q4KError) as e:
            bad()
        assert e.value.status == SHAPE
