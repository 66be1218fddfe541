"""The operators around the projections at the ends of their ranges: empty steps, lengths past the table,
weights far below the largest, pipelines that run long enough to refill every stage, and what the pointer
checks refuse.

Tolerances count roundings: half a step of a type is eps / 2 relative (bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4).
"""
from __future__ import annotations

import ctypes
import glob
import math
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from _gpu import DEV
from test_decode_ops import plain_sample, BAD_PAGE, BF16, E4M3, F32, H16, H8, H32, HB, gen, make_attn, plain_attn, plain_plan, quantize, to_dev

gpu = pytest.mark.gpu
OK, NULL, SHAPE, ALIGN, MEMORY = 0, 1, 2, 3, 8


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


# ------------------------------------------------------------------------------------------ weights far below the largest


def attn_bounds(q, k, v, scale, e4m3, keep=None):
    """(out, lse, bound of out, bound of lse) in 64 bits of q [n, hq, d] over k, v [n, t, h, d], keep [n, t].

    Roundings: fp32 scores (a product's rounding and d additions of up to the sum of |q k| each, and the
    scaling), exp2 and its argument 2^-20 relative, sums of t terms, the weights: two bf16 terms (2^-16), or
    one fp16 term: half a step 2^-11 of those down to 2^-29 of the largest weight times scale, and 2^-40 of it
    below (half of fp16's smallest step 2^-24, the largest being 2^15); the output's bf16."""
    n, hq, d = q.shape
    t = k.shape[1]
    group = hq // k.shape[2]
    k, v = k.repeat_interleave(group, 2), v.repeat_interleave(group, 2)
    z = torch.einsum("nhd,nthd->nht", q, k) * scale
    size = torch.einsum("nhd,nthd->nht", q.abs(), k.abs()) * abs(scale)
    if keep is not None:
        z = z.masked_fill(~keep[:, None], -math.inf)
        size = size.masked_fill(~keep[:, None], 0.0)
        v = v.masked_fill(~keep[:, :, None, None], 0.0)
    lse = torch.logsumexp(z, 2)
    some = lse > -math.inf
    p = torch.exp(z - lse.masked_fill(~some, 0.0)[:, :, None])
    out = torch.einsum("nht,nthd->nhd", p, v)
    pv = torch.einsum("nht,nthd->nhd", p, v.abs())
    far = z.masked_fill(z == -math.inf, 0.0).abs().amax(2)
    dz = (d + 8) * H32 * size.amax(2) + 2.0 ** -20 * (1 + far * 2 ** -2)
    count = keep.sum(1).double()[:, None] if keep is not None else torch.full((n, 1), float(t), dtype=torch.float64, device=q.device)
    sums = (count.sqrt() + 40) * H32 * 2
    rel = 2 * dz + sums + (H16 if e4m3 else 2.0 ** -16)
    bo = HB * out.abs() + rel[:, :, None] * pv * 1.01
    if e4m3:
        largest = (p.unsqueeze(-1) * v.abs().permute(0, 2, 1, 3)).amax((2, 3))
        bo = bo + 2.0 ** -40 * count[:, :, None] * largest[:, :, None] * 1.01
    return out, lse, bo, dz + sums + H32 * lse.masked_fill(~some, 0.0).abs()


@gpu
@pytest.mark.parametrize("gap", [10, 14, 17, 20, 24, 27, 32])
@pytest.mark.parametrize("dim,q_heads", [(64, 2), (64, 16), (128, 4), (128, 16), (256, 8)])
def test_attn_weights_far_below_the_largest(q4k, dim, q_heads, gap):
    """One token takes nearly all the weight and the others, `gap` binary orders below it, all of the value in
    every column but the first."""
    page, h = 32, 2
    g = gen(gap + dim)
    for length in (32, 33, 700, 9000):
        k, v = torch.zeros((length, h, dim)), torch.randn((length, h, dim), generator=g).abs() + 0.5
        # scores of the others: -gap ln 2 and less, by up to one binary order
        k[:, :, 1] = -(gap + torch.rand((length, h), generator=g)) * math.log(2.0)
        v[:, :, 0] = 0.0
        sink = length * 2 // 3
        k[sink] = 0.0
        v[sink] = 0.0
        v[sink, :, 0] = 1.5
        q = torch.zeros((1, h * q_heads, dim))
        q[:, :, 1] = 1.0
        pages = -(-length // page)
        table = torch.randperm(pages, generator=g).to(torch.int32)
        caches, scales, dense = [], [], []
        for x in (k, v):
            b, s = quantize(x)
            dense.append((b.view(E4M3).double() * s.double()[..., None])[None].to(DEV))
            c, cs = torch.zeros((pages * page, h, dim), dtype=torch.uint8), torch.ones((pages * page, h))
            c[:length], cs[:length] = b, s
            c, cs = c.view(pages, page, h, dim).transpose(1, 2), cs.view(pages, page, h).transpose(1, 2)
            inv = torch.argsort(table)
            caches.append(c[inv].contiguous().to(DEV).view(E4M3)), scales.append(cs[inv].contiguous().to(DEV))
        qb = q.to(BF16).to(DEV)
        out, lse = q4k.q4k_paged_attn(qb, *caches, table[None].to(DEV), torch.tensor([length], dtype=torch.int32, device=DEV), 1.0, *scales)
        want, wl, bo, bl = attn_bounds(qb.double(), *dense, 1.0, True)
        off = (out.double() - want).abs()
        assert bool((off <= bo).all()), (length, float((off / bo).max()))
        assert bool(((lse.double() - wl).abs() <= bl).all()), length
    assert q4k.q4k_get_device_error() == 0


# ------------------------------------------------------------------------------------------ threads

THREADS = """
import sys, threading
import torch
sys.path.insert(0, sys.argv[1])
import bit_block_quantized_q4_gb300 as q4k
BF16, E4M3, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32
q4k.lib()
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(s, generator=g, device="cuda")
lens, table = torch.tensor([90, 3], dtype=I32, device="cuda"), torch.tensor([[0, 1, 2], [3, 0, 0]], dtype=I32, device="cuda")
x, res, gamma = rand(2000, 5120).to(BF16), rand(2000, 5120).to(BF16), rand(8192)
wide, logits, u = rand(1400, 8192).to(BF16), rand(4, 50000), torch.rand(4, generator=g, device="cuda")
caches = {}
for d in (64, 128, 256):
    k = [rand(4, 2, 32, d) for _ in range(2)]
    caches[d] = ([c.to(BF16) for c in k], [c.to(E4M3) for c in k], [torch.rand((4, 2, 32), generator=g, device="cuda") + 0.1 for _ in range(2)])

def calls():
    for d in (64, 128, 256):
        plain, small, scales = caches[d]
        for heads in (4, 32):
            q = torch.ones((2, heads, d), dtype=BF16, device="cuda")
            yield lambda: q4k.q4k_paged_attn(q, *plain, table, lens, 0.1)
            yield lambda: q4k.q4k_paged_attn(q, *small, table, lens, 0.1, *scales)
    for out in (BF16, E4M3):
        yield lambda: q4k.q4k_add_rmsnorm(x, res, gamma[:5120], 1e-6, out_dtype=out)
        yield lambda: q4k.q4k_add_rmsnorm(wide, None, gamma, 1e-6, out_dtype=out)
    yield lambda: q4k.q4k_sample(logits, u)
    yield lambda: q4k.q4k_sample(logits.to(BF16), u)

def bits(r):
    return [t.view(torch.uint8) if t.dtype == E4M3 else t for t in r if t is not None]

torch.cuda.synchronize()
results, errors, start = [None] * 8, [], threading.Barrier(8)

def work(i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            out = []
            for call in calls():  # every kernel's first call, in all threads at once
                start.wait(60)
                out.append(bits(call()))
            torch.cuda.current_stream().synchronize()
            results[i] = out
    except Exception as e:
        errors.append(repr(e))
        start.abort()

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
want = [bits(call()) for call in calls()]
torch.cuda.synchronize()
for r in results:
    for a, b in zip(r, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
assert q4k.q4k_get_device_error() == 0
print("threads agree")
"""


@gpu
def test_first_calls_from_several_threads(q4k):
    """A fresh process in which eight threads make every kernel's first call at the same time."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", THREADS, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "threads agree" in r.stdout, r.stdout + r.stderr


def test_launchers_keep_no_plain_state():
    """What a launcher does once per device is under std::call_once: a plain static that threads read and
    write is a data race."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    files = glob.glob(os.path.join(root, "bit_block_quantized_q4_gb300", "csrc", "*.c*"))
    assert files
    for f in files:
        with open(f) as src:
            found = re.findall(r"^\s+static (?!const|SmemLimit\b|std::once_flag\b|__)[\w:<>]+ \w+(?:\[\w+\])?(?: = [^(]*)?;", src.read(), re.M)
        assert not found, (os.path.basename(f), found)


# ------------------------------------------------------------------------------------------ what pointers are refused


class Driver:
    """Allocations straight from the driver, without a caching allocator between."""

    def __init__(self):
        self.cu = ctypes.CDLL("libcuda.so.1")

    def _ok(self, status):
        assert status == 0, status

    def device(self, size):
        p = ctypes.c_uint64()
        self._ok(self.cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(size)))
        return p.value

    def pinned(self, size):
        p = ctypes.c_void_p()
        self._ok(self.cu.cuMemAllocHost_v2(ctypes.byref(p), ctypes.c_size_t(size)))
        return p.value

    def managed(self, size):
        p = ctypes.c_uint64()
        self._ok(self.cu.cuMemAllocManaged(ctypes.byref(p), ctypes.c_size_t(size), ctypes.c_uint(1)))
        return p.value

    def free(self, p):
        self._ok(self.cu.cuMemFree_v2(ctypes.c_uint64(p)))

    def is_device(self, p):
        """Whether the driver knows the address as device memory."""
        kind = ctypes.c_uint(0)
        return self.cu.cuPointerGetAttribute(ctypes.byref(kind), 2, ctypes.c_uint64(p)) == 0 and kind.value == 2


@gpu
def test_every_pointer_of_a_call_is_checked(q4k):
    """One pointer that is not device memory is refused in any place beside others that are: freed memory and
    memory past an allocation in the 2 MB that a good pointer lies in too, pinned and managed memory.  (All
    are refused on the host: nothing is launched.)"""
    torch.zeros(1, device=DEV)
    d, L = Driver(), q4k.lib()
    size = 4096
    good = [d.device(size) for _ in range(2)]
    freed = d.device(size)
    d.free(freed)
    near = [p for p in (freed, good[0] + (1 << 20), good[0] - (1 << 20), good[0] + (1 << 19)) if p >> 21 == good[0] >> 21 and not d.is_device(p)]
    assert all(d.is_device(p) for p in good) and near, "no address of the same 2 MB that the driver does not know"
    pinned, managed = d.pinned(size), d.managed(size)
    assert L.q4k_dequant(good[0], 1, 256, good[1], 0, None) == OK
    torch.cuda.synchronize()
    sample = lambda logits, u, t, token: L.q4k_sample(logits, 0, 1, 64, 64, u, t, None, None, None, token, None, None)  # noqa: E731
    gemv = lambda w, x, y: L.q4k_gemv(w, 1, 256, x, 1, 256, y, 1, None)  # noqa: E731
    norm = lambda x, g, y: L.q4k_add_rmsnorm(x, 0, 64, None, 0, 0, g, 1e-6, 1, 64, y, 1, 64, None, 0, None, 0, None)  # noqa: E731
    plan = lambda state, cu, state_out: L.q4k_kv_plan(None, None, 0, None, 8, 8, 16, None, 64, state, None, cu, None, None, 0, None, state_out, None)  # noqa: E731
    a, b = good
    for bad in near + [pinned, managed]:
        assert not d.is_device(bad) or bad == managed
        for call, args in ((lambda w, o: L.q4k_dequant(w, 1, 256, o, 0, None), (a, b)), (sample, (a, b, a + 1024, b + 1024)), (gemv, (a, b, a + 1024)),
                           (norm, (a, b, a + 1024)), (plan, (a, b, a + 1024))):
            for i in range(len(args)):
                assert call(*args[:i], bad, *args[i + 1:]) == MEMORY
    torch.cuda.synchronize()
    assert q4k.q4k_get_device_error() == 0
    d._ok(d.cu.cuMemFreeHost(ctypes.c_void_p(pinned)))
    for p in good + [managed]:
        d.free(p)


def test_binding_refuses_a_workspace_that_is_not_contiguous(q4k):
    """An expanded tensor has more elements than memory."""
    cache = torch.zeros((4, 2, 16, 64), dtype=BF16)
    lens, table, q = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32), torch.zeros((2, 4, 64), dtype=BF16)
    size = q4k.q4k_paged_attn_workspace_size(2, 4, 2, 64)
    for workspace in (torch.zeros(1, dtype=torch.uint8).expand(size), torch.zeros(2 * size, dtype=torch.uint8)[::2]):
        with pytest.raises(q4k.Q4KError) as e:
            q4k.q4k_paged_attn(q, cache, cache, table, lens, 1.0, workspace=workspace)
        assert e.value.status == SHAPE


# ------------------------------------------------------------------------------------------ the least temperature


@gpu
def test_sample_least_temperature(q4k):
    """Logits that differ by parts of the least temperature, 2^-121, which all below it count as."""
    rows, vocab = 24, 5000
    g = gen(5)
    x = -torch.rand((rows, vocab), generator=g) * 4e-36
    u = torch.rand(rows, generator=g)
    i = torch.arange(rows)
    t = torch.tensor([1e-40, 2.0 ** -121, 1e-38, 3e-37, 2.0 ** -149, 1e-36])[i % 6]
    p, k = torch.tensor([0.9, 0.5, 1.0, 0.999])[i % 4], torch.tensor([0, 0, 3000, 40])[(i // 4) % 4]
    token, logp = (v.cpu() for v in q4k.q4k_sample(x.to(DEV), u.to(DEV), t.to(DEV), k.to(torch.int32).to(DEV), p.to(DEV)))
    for r in range(rows):
        want, lp, near = plain_sample(x[r].numpy(), float(u[r]), max(float(t[r]), 2.0 ** -121), int(k[r]), float(p[r]), 0.0)
        assert int(token[r]) in near, r
        assert int(token[r]) != want or abs(float(logp[r]) - lp) <= H32 * abs(lp) + 2.0 ** -30, r
    assert q4k.q4k_get_device_error() == 0


# ------------------------------------------------------------------------------------------ pipelines in their steady state


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


def shared_cache(seed, pages, heads, dim, page, kind):
    """Cache buffers of `pages` pages that many requests may share, on the GPU, with their values in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    caches, scales, values = [], [], []
    for kv in range(2):
        x = torch.randn((pages, heads, page, dim), generator=g, device=DEV)
        if kind == E4M3:
            x = x * torch.exp2(torch.randint(-6, 7, (pages, heads, page, 1), generator=g, device=DEV).float()) if kv else x
            b, s = quantize(x)
            caches.append(b.view(E4M3)), scales.append(s), values.append(b.view(E4M3).double() * s.double()[..., None])
        else:
            caches.append(x.to(BF16)), values.append(caches[-1].double())
    return caches, scales, values


def check_long(q4k, seed, lens, q_heads, heads, dim, page, kind, pages, window=0, absent=0.0):
    """Attention over tables into a shared cache, against 64 bits, a chunk of requests at a time."""
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    caches, scales, values = shared_cache(seed, pages, heads, dim, page, kind)
    n, width = len(lens), -(-max(lens) // page) + 3
    table = torch.randint(0, pages, (n, width), generator=g, device=DEV).to(torch.int32)
    if absent:
        out_of_range = torch.tensor([-1, pages, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
        hit = torch.rand((n, width), generator=g, device=DEV) < absent
        table = torch.where(hit, out_of_range[torch.randint(0, 3, (n, width), generator=g, device=DEV)], table)
    # entries past a request's pages: of no use to anyone
    at = torch.arange(width, device=DEV)[None]
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    table = torch.where(at * page < ln[:, None], table, torch.full_like(table, -9)).contiguous()
    q = torch.randn((n, q_heads, dim), generator=g, device=DEV).to(BF16)
    out, lse = q4k.q4k_paged_attn(q, *caches, table, ln, dim ** -0.5, *scales, window=window)
    again = q4k.q4k_paged_attn(q, *caches, table, ln, dim ** -0.5, *scales, window=window)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    seen = (at * page < ln[:, None]) & ((at + 1) * page > (ln[:, None] - window if window else 0))
    bad = bool((seen & ((table < 0) | (table >= pages))).any())
    assert q4k.q4k_get_device_error() == (BAD_PAGE if bad else 0) and (bad or not absent)
    order = torch.argsort(ln, stable=True).tolist()
    while order:
        longest = max(lens[r] for r in order[-1:])
        chunk = order[-max(1, min(len(order), int(2e7) // max(1, longest * q_heads * dim))):]
        del order[-len(chunk):]
        if not longest:
            assert not out[chunk].any() and bool((lse[chunk] == -math.inf).all())
            continue
        m = -(-longest // page)
        ids = table[chunk, :m].long()
        ok = (ids >= 0) & (ids < pages)
        k, v = (x[ids.clamp(0, pages - 1)].permute(0, 1, 3, 2, 4).reshape(len(chunk), m * page, heads, dim) for x in values)
        tok = torch.arange(m * page, device=DEV)[None]
        keep = (tok < ln[chunk, None]) & ok.repeat_interleave(page, 1)
        if window:
            keep &= tok >= ln[chunk, None] - window
        want, wl, bo, bl = attn_bounds(q[chunk].double(), k, v, dim ** -0.5, kind == E4M3, keep)
        worst = float(((out[chunk].double() - want).abs() - bo).max())
        assert worst <= 0, worst
        got = lse[chunk].double()
        assert torch.equal(got == -math.inf, wl == -math.inf)
        fin = wl != -math.inf
        assert not fin.any() or float(((got - wl).abs() - bl)[fin].max()) <= 0


# Warps per SM of a configuration, and tokens per tile: what a run of 32 tiles or more per warp needs.
WARPS = {(64, BF16): 12, (64, E4M3): 12, (128, BF16): 6, (128, E4M3): 12, (256, BF16): 6, (256, E4M3): 6}
TILE = {(256, BF16): 16}


@gpu
@pytest.mark.parametrize("window,absent,page", [(0, 0.0, 16), (3001, 0.02, 16), (0, 0.05, 64)])
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 4), (128, 16), (256, 3)])
def test_attn_many_tiles_per_warp(q4k, dim, group, kind, window, absent, page):
    """Few long requests, at least 32 tiles for every warp: each stage is refilled many times, table entries are
    fetched on the way, and pieces begin and end inside of items."""
    heads, tile = 4, TILE.get((dim, kind), 32)
    tokens = 32 * sm_count() * WARPS[dim, kind] * tile // heads
    n = 24
    per = tokens // n
    if window:  # a window's tiles only
        n = -(-tokens // (window - tile))
        per = 2 * window
    lens = [per + (i * 7919) % 97 * (per // 200 + 1) for i in range(n)] + [0, 1, 17, per // 3, 0, tile + 1]
    total = sum(-(-v // tile) - (max(0, v - window) if window else 0) // tile for v in lens) * heads
    assert total >= 32 * sm_count() * WARPS[dim, kind]
    check_long(q4k, 41 + dim, lens, heads * group, heads, dim, page, kind, 512, window, absent)


@gpu
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("dim,group,page,absent", [(64, 1, 16, 0.0), (64, 16, 32, 0.03), (128, 8, 16, 0.03), (128, 12, 256, 0.0), (256, 8, 32, 0.03), (256, 12, 16, 0.0)])
def test_attn_many_requests_per_warp(q4k, dim, group, kind, page, absent):
    """Many short requests: a warp goes through several items and requests, refills across their borders, and
    stages whose value rows were zeroed are filled again."""
    heads, tile = 8, TILE.get((dim, kind), 32)
    groups = -(-group // (8 if dim == 256 or group <= 8 else 16))
    n = 32 * sm_count() * WARPS[dim, kind] // (heads * groups * (-(-95 // tile)))
    lens = [(i * 37) % 190 for i in range(n + n // 8)]
    assert sum(-(-v // tile) for v in lens) * heads * groups >= 32 * sm_count() * WARPS[dim, kind]
    check_long(q4k, 43 + dim + group, lens, heads * group, heads, dim, page, kind, 1000, 0, absent)


@gpu
@pytest.mark.parametrize("out", [BF16, E4M3])
@pytest.mark.parametrize("h,src,res,per_sm", [(4104, BF16, None, 5), (5120, BF16, BF16, 4), (5120, F32, BF16, 3), (8200, BF16, BF16, 3), (8200, F32, F32, 1), (12288, BF16, BF16, 2), (17408, BF16, None, 2),
                                              (12800, F32, F32, 1)])
def test_norm_rows_in_the_ring(q4k, h, src, res, per_sm, out):
    """At least 16 rows for every block, so that each stage of its ring (4 at most) is filled again three times;
    with the residual's new value in a tensor of its own and in place."""
    m = 16 * per_sm * sm_count() + 37
    g = torch.Generator(device=DEV).manual_seed(h)
    x = torch.randn((m, h), generator=g, device=DEV).mul_(2).to(src)
    r = None if res is None else torch.randn((m, h), generator=g, device=DEV).mul_(3).to(res)
    gamma = torch.rand(h, generator=g, device=DEV) + 0.5
    got = q4k.q4k_add_rmsnorm(x, r, gamma, 1e-6, out_dtype=out)
    if r is not None:
        kept = r.clone()
        same = q4k.q4k_add_rmsnorm(x, kept, gamma, 1e-6, out_dtype=out, residual_out=kept)
        assert torch.equal(kept, got[1]) and torch.equal(same[0].view(torch.uint8), got[0].view(torch.uint8))
        assert out == BF16 or torch.equal(same[2], got[2])
    assert q4k.q4k_get_device_error() == 0
    # h: one fp32 rounding; the sum of squares: h / 32 + 24 additions at most in a row, halved by the square
    # root; rsqrt, the division by h, two products
    rel = (h / 32 + 24) * H32 + 8 * H32
    for part in torch.arange(m, device=DEV).split(1024):
        xx = x[part].double()
        rr = 0.0 if r is None else r[part].double()
        hh = xx + rr
        norm = torch.sqrt((hh * hh).mean(-1, keepdim=True) + 1e-6)
        y = hh / norm * gamma.double()
        size = xx.abs() + (0.0 if r is None else rr.abs())
        if r is not None:
            assert float(((got[1][part].double() - hh).abs() - (HB if res == BF16 else 0.0) * hh.abs() * 1.001 - 2 * H32 * size).max()) <= 0
        slip = rel * y.abs() + H32 * size / norm * gamma.double()
        if out == BF16:
            assert float(((got[0][part].double() - y).abs() - HB * y.abs() - 1.01 * slip).max()) <= 0
            continue
        s = got[2][part].double()
        wide = s.repeat_interleave(128, 1)[:, :h]
        # a value: half a step of e4m3 (of its smallest, 2^-9, where it is subnormal)
        assert float(((got[0][part].double() * wide - y).abs() - H8 * y.abs() * 1.001 - 2.0 ** -10 * wide - 1.2 * slip).max()) <= 0
        blocks = torch.nn.functional.pad(torch.stack([y.abs(), slip]), (0, -h % 128)).unflatten(2, (-1, 128)).amax(-1) / 448
        assert float(((s - blocks[0]).abs() - 4 * H32 * blocks[0] - 1.01 * blocks[1]).max()) <= 0
