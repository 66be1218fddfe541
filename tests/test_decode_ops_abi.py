"""Refusals of the entry points around the projections (cache plan and write, paged attention, norm,
sampling): every argument error comes back before a device is touched, so these run without one."""
from __future__ import annotations

import pytest
import torch

P = 0x10000  # a non-null, 64 KiB-aligned pointer value; never dereferenced
OK, NULL, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    from bit_block_quantized_q4_gb300 import build
    build.build()
    import bit_block_quantized_q4_gb300 as q4k
    return q4k.lib()


def _call(fn, base, **change):
    args = dict(base)
    for k in change:
        assert k in args, k
    args.update(change)
    return fn(*args.values())


PLAN = dict(lens=P, add=P, n=4, table=P, ldt=8, max_pages=8, page=16, pool=P, pool_size=64, state=P, lens_out=P,
            cu=P, slots=P, pos=P, n_slots=4, status=P, state_out=P, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), SHAPE), (dict(n=65537), SHAPE), (dict(max_pages=0), SHAPE), (dict(ldt=7), SHAPE), (dict(page=0), SHAPE),
    (dict(max_pages=1 << 27, ldt=1 << 27), SHAPE), (dict(pool_size=0), SHAPE), (dict(pool_size=1 << 28, page=16), SHAPE), (dict(n_slots=-1), SHAPE), (dict(n_slots=1 << 31), SHAPE),
    (dict(n=0, lens=None), OK), (dict(lens=None), NULL), (dict(add=None), NULL), (dict(table=None), NULL), (dict(pool=None), NULL),
    (dict(state=None), NULL), (dict(lens_out=None), NULL), (dict(cu=None), NULL), (dict(slots=None), NULL), (dict(pos=None), NULL),
    (dict(status=None), NULL), (dict(state_out=None), NULL), (dict(cu=P + 4), ALIGN), (dict(lens=P + 2), ALIGN), (dict(slots=P + 1), ALIGN)])
def test_plan_refusals(L, change, status):
    assert _call(L.q4k_kv_plan, PLAN, **change) == status


CACHE = dict(cache_dtype=1, n_pages=64, page=16, page_stride=16 * 8 * 128, head_stride=16 * 128, token_stride=128)
WRITE = dict(k=P, v=P, in_dtype=0, ld_token=1024, ld_head=128, slots=P, tokens=4, heads=8, dim=128, k_cache=P, v_cache=P, **CACHE,
             k_scale=None, v_scale=None, stream=None)
CACHE_REFUSALS = [
    (dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(cache_dtype=0), SHAPE), (dict(cache_dtype=3), SHAPE), (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 28), SHAPE),
    (dict(page=0), SHAPE), (dict(token_stride=120), SHAPE), (dict(head_stride=120), SHAPE),
    (dict(token_stride=136), SHAPE),               # a page's tokens run into the next head
    (dict(page_stride=16 * 8 * 128 - 8), SHAPE),   # pages overlap
    (dict(page_stride=16 * 8 * 128 + 4), ALIGN),
    (dict(cache_dtype=2, page_stride=16 * 8 * 128 + 8), ALIGN)]


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(in_dtype=2), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 30), SHAPE), (dict(ld_head=64), SHAPE), (dict(ld_token=-8), SHAPE), (dict(heads=0), SHAPE),
    (dict(tokens=0, k=None), OK), (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(k_cache=None), NULL), (dict(v_cache=None), NULL),
    (dict(cache_dtype=2), NULL), (dict(cache_dtype=2, k_scale=P), NULL), (dict(k=P + 8), ALIGN), (dict(v_cache=P + 8), ALIGN), (dict(ld_token=1028), ALIGN),
    (dict(slots=P + 2), ALIGN)])
def test_write_refusals(L, change, status):
    assert _call(L.q4k_kv_write, WRITE, **change) == status


ATTN = dict(q=P, ldq=1024, ldq_head=128, n=4, q_heads=8, heads=8, dim=128, k_cache=P, v_cache=P, **CACHE, k_scale=None, v_scale=None,
            table=P, ldt=8, max_pages=8, lens=P, scale=0.1, window=0, out=P, ldo=1024, lse=None, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(page=8, page_stride=1 << 20), SHAPE), (dict(page=512, page_stride=1 << 20, head_stride=1 << 17), SHAPE), (dict(page=24, head_stride=24 * 128, page_stride=1 << 20), SHAPE),
    (dict(n=-1), SHAPE), (dict(n=65537), SHAPE), (dict(q_heads=12), SHAPE), (dict(q_heads=2048), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 27, ldt=1 << 27), SHAPE), (dict(ldt=7), SHAPE),
    (dict(cache_dtype=2, k_scale=P + 8, v_scale=P), ALIGN), (dict(window=-1), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(ldq_head=64), SHAPE), (dict(ldo=1016), SHAPE),
    (dict(n=0, q=None), OK), (dict(q=None), NULL), (dict(k_cache=None), NULL), (dict(v_cache=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(out=None), NULL), (dict(cache_dtype=2, k_scale=P), NULL), (dict(ws=None), WORKSPACE), (dict(ws_bytes=0), WORKSPACE), (dict(q=P + 8), ALIGN), (dict(ldq=1028), ALIGN),
    (dict(ldo=1028), ALIGN), (dict(lens=P + 2), ALIGN), (dict(ws=P + 8), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_attn_refusals(L, change, status):
    assert _call(L.q4k_paged_attn, ATTN, **change) == status


def _strides(order, page=16, heads=8, pages=64, dim=128):
    """Strides of a dense cache whose dimensions lie in this order, the outermost first."""
    extent, out, at = dict(page=page, head=heads, pages=pages), {}, dim
    for name in reversed(order):
        out[{"page": "token_stride", "head": "head_stride", "pages": "page_stride"}[name]] = at
        at *= extent[name]
    return out


ORDERS = [("pages", "head", "page"), ("pages", "page", "head"), ("head", "pages", "page"), ("head", "page", "pages"), ("page", "pages", "head"), ("page", "head", "pages")]


@pytest.mark.parametrize("order", ORDERS)
def test_cache_strides_in_any_order(L, order):
    """Dense caches pass the checks of strides in every order (there is no device, or the memory is
    not a device's); eight elements less in any but the innermost stride are an overlap."""
    good = _strides(order)
    for fn, base in ((L.q4k_kv_write, WRITE), (L.q4k_paged_attn, ATTN)):
        assert _call(fn, base, **good) not in (OK, NULL, SHAPE, ALIGN, WORKSPACE)
        for name in good:
            assert _call(fn, base, **{**good, name: good[name] - 8}) == SHAPE


def test_cache_strides_whose_product_passes_64_bits(L):
    """2^24 tokens of stride 2^40 do not fit a page of 2^40, though the product is 0 in 64 bits."""
    assert _call(L.q4k_kv_write, WRITE, heads=1, page=1 << 24, n_pages=4, token_stride=1 << 40, page_stride=1 << 40) == SHAPE


NORM = dict(x=P, x_dtype=0, ldx=512, res=P, res_dtype=1, ldr=512, gamma=P, eps=1e-6, m=4, hidden=512, y=P, y_dtype=1, ldy=512, res_out=P, ldro=512,
            scales=None, lds=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x_dtype=2), SHAPE), (dict(y_dtype=0), SHAPE), (dict(res_dtype=2), SHAPE), (dict(m=-1), SHAPE), (dict(hidden=0), SHAPE), (dict(hidden=500), SHAPE),
    (dict(hidden=32776, ldx=40000, ldr=40000, ldy=40000, ldro=40000), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(ldx=504), SHAPE), (dict(ldy=504), SHAPE), (dict(ldr=504), SHAPE), (dict(ldro=504), SHAPE), (dict(y_dtype=2, scales=P, lds=3), SHAPE),
    (dict(m=0, x=None), OK), (dict(x=None), NULL), (dict(gamma=None), NULL), (dict(y=None), NULL), (dict(res_out=None), NULL), (dict(y_dtype=2, lds=4), NULL),
    (dict(x=P + 8), ALIGN), (dict(gamma=P + 4), ALIGN), (dict(ldx=516), ALIGN), (dict(ldr=516), ALIGN), (dict(res_out=P + 8), ALIGN), (dict(y_dtype=2, scales=P + 2, lds=4), ALIGN)])
def test_norm_refusals(L, change, status):
    assert _call(L.q4k_add_rmsnorm, NORM, **change) == status


SAMPLE = dict(logits=P, dtype=0, rows=2, vocab=100, ld=100, u=P, t=P, k=P, p=P, m=P, token=P, logp=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), SHAPE), (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=262145, ld=262145), SHAPE), (dict(ld=99), SHAPE),
    (dict(rows=0, logits=None), OK), (dict(logits=None), NULL), (dict(u=None), NULL), (dict(token=None), NULL), (dict(logits=P + 2), ALIGN), (dict(dtype=1, logits=P + 1), ALIGN),
    (dict(u=P + 2), ALIGN), (dict(k=P + 1), ALIGN)])
def test_sample_refusals(L, change, status):
    assert _call(L.q4k_sample, SAMPLE, **change) == status


def test_binding_refuses_wrong_types_shapes_and_layouts(L):
    import bit_block_quantized_q4_gb300 as q4k
    z = torch.zeros
    cache = z((4, 2, 16, 64), dtype=torch.bfloat16)
    lens, table, q = z(2, dtype=torch.int32), z((2, 3), dtype=torch.int32), z((2, 4, 64), dtype=torch.bfloat16)
    bad = [
        lambda: q4k.q4k_paged_attn(q.float(), cache, cache, table, lens, 1.0),
        lambda: q4k.q4k_paged_attn(q, cache, cache.float(), table, lens, 1.0),
        lambda: q4k.q4k_paged_attn(q, cache, cache[:, :, :, ::2], table, lens, 1.0),
        lambda: q4k.q4k_paged_attn(q, cache, z((4, 16, 2, 64), dtype=torch.bfloat16).transpose(1, 2), table, lens, 1.0),
        lambda: q4k.q4k_paged_attn(q, cache, cache, table.long(), lens, 1.0),
        lambda: q4k.q4k_paged_attn(q, cache, cache, table, lens[:1], 1.0),
        lambda: q4k.q4k_paged_attn(q[:, :, :32], cache, cache, table, lens, 1.0),
        lambda: q4k.q4k_kv_write(z((3, 2, 64)), z((3, 2, 64), dtype=torch.bfloat16), z(3, dtype=torch.int32), cache, cache),
        lambda: q4k.q4k_kv_write(z((3, 2, 64)), z((3, 2, 64)), z(2, dtype=torch.int32), cache, cache),
        lambda: q4k.q4k_kv_plan(lens, lens, table.t(), lens, lens, 16, 2),
        lambda: q4k.q4k_kv_plan(lens, lens.long(), table, lens, lens, 16, 2),
        lambda: q4k.q4k_add_rmsnorm(z((2, 64)), z((2, 32)), z(64), 1e-6),
        lambda: q4k.q4k_add_rmsnorm(z((2, 64)), None, z(64, dtype=torch.bfloat16), 1e-6),
        lambda: q4k.q4k_add_rmsnorm(z((2, 64)), None, z(64), 1e-6, out_dtype=torch.float32),
        lambda: q4k.q4k_sample(z((2, 10), dtype=torch.float16), z(2)),
        lambda: q4k.q4k_sample(z((2, 10)), z(3)),
        lambda: q4k.q4k_sample(z((2, 10)), z(2), top_k=z(2)),
    ]
    for call in bad:
        with pytest.raises(q4k.Q4KError) as e:
            call()
        assert e.value.status == SHAPE
