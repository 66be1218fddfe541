"""Python binding of libq4k.so, the GB300 (sm_103a) Q4_K projection library.

The functions here carry the C entry points' names and only marshal
arguments: torch tensors in, raw device pointers, sizes and the current CUDA
stream out.  Every step of the computation runs in the library's CUDA kernels;
there is no fallback.  If libq4k.so is missing, importing works but every call
raises.  Build it with ``python -m bit_block_quantized_q4_gb300.build`` (or
``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libq4k.so")
Q4K_VALUES = 256
Q4K_BYTES = 144

STATUS = {0: "Q4K_OK", 1: "Q4K_ERR_NULL", 2: "Q4K_ERR_SHAPE", 3: "Q4K_ERR_ALIGN",
          4: "Q4K_ERR_WORKSPACE", 5: "Q4K_ERR_DEVICE", 6: "Q4K_ERR_CUDA", 7: "Q4K_ERR_DATA",
          8: "Q4K_ERR_MEMORY"}
Q4K_FLAG_OVERLAP_WEIGHTS = 1
Q4K_SEQ_MATRICES_PER_LAUNCH = 160
Q4K_MOE_WEIGHTED_DOWN = 1
EXPORTS = ("q4k_abi_version", "q4k_status_str", "q4k_dequant", "q4k_gemv", "q4k_gemv_ex",
           "q4k_gemv_glu", "q4k_gemv_seq", "q4k_gemm", "q4k_gemm_rmsnorm",
           "q4k_kq_block_bytes", "q4k_kq_dequant", "q4k_kq_gemv", "q4k_kq_gemv_seq",
           "q4k_moe_workspace_size", "q4k_moe_workspace_views", "q4k_moe_gemv",
           "q4k_moe_gemv_ex", "q4k_moe_gemv_noalloc", "q4k_moe_prefill",
           "q4k_moe_prefill_workspace_size",
           "q4k_kv_plan", "q4k_kv_write", "q4k_paged_attn", "q4k_paged_attn_workspace_size",
           "q4k_add_rmsnorm", "q4k_sample",
           "q4k_get_device_error", "q4k_selftest_wait_timeout")
Q4K_DTYPE_FP32, Q4K_DTYPE_BF16, Q4K_DTYPE_E4M3 = 0, 1, 2
Q4K_KV_OK, Q4K_KV_NO_PAGES, Q4K_KV_BAD_LENGTH, Q4K_KV_NO_SLOTS = 0, 1, 2, 3

_lock = threading.Lock()
_lib = None


class GemvOp(ctypes.Structure):
    """One entry of q4k_gemv_seq's op array (struct q4k_gemv_op); w_up is NULL
    for a plain projection, the up matrix of a fused gate/up op otherwise."""
    _fields_ = [("w", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64), ("w_up", ctypes.c_void_p)]


class Q4KError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status_str(status)})")


def lib() -> ctypes.CDLL:
    """The loaded libq4k.so with argument types declared (raises if not built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run python -m bit_block_quantized_q4_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        L.q4k_abi_version.restype = ctypes.c_int
        L.q4k_abi_version.argtypes = []
        L.q4k_status_str.restype = ctypes.c_char_p
        L.q4k_status_str.argtypes = [ctypes.c_int]
        L.q4k_dequant.restype = ctypes.c_int
        L.q4k_dequant.argtypes = [P, I64, I64, P, ctypes.c_int, P]
        L.q4k_gemv.restype = ctypes.c_int
        L.q4k_gemv.argtypes = [P, I64, I64, P, I64, I64, P, I64, P]
        L.q4k_gemv_ex.restype = ctypes.c_int
        L.q4k_gemv_ex.argtypes = [P, I64, I64, P, I64, I64, P, I64, ctypes.c_uint32, P]
        L.q4k_gemv_glu.restype = ctypes.c_int
        L.q4k_gemv_glu.argtypes = [P, P, I64, I64, P, I64, I64, P, I64, ctypes.c_uint32, P]
        L.q4k_gemv_seq.restype = ctypes.c_int
        L.q4k_gemv_seq.argtypes = [ctypes.POINTER(GemvOp), I64, I64, ctypes.c_uint32, P]
        L.q4k_gemm.restype = ctypes.c_int
        L.q4k_gemm.argtypes = [P, I64, I64, P, I64, I64, P, I64, P]
        L.q4k_kq_block_bytes.restype = ctypes.c_int
        L.q4k_kq_block_bytes.argtypes = [I32]
        L.q4k_kq_dequant.restype = ctypes.c_int
        L.q4k_kq_dequant.argtypes = [I32, P, I64, I64, P, ctypes.c_int, P]
        L.q4k_kq_gemv.restype = ctypes.c_int
        L.q4k_kq_gemv.argtypes = [I32, P, I64, I64, P, I64, I64, P, I64, P]
        L.q4k_kq_gemv_seq.restype = ctypes.c_int
        L.q4k_kq_gemv_seq.argtypes = [I32, ctypes.POINTER(GemvOp), I64, I64, ctypes.c_uint32, P]
        L.q4k_gemm_rmsnorm.restype = ctypes.c_int
        L.q4k_gemm_rmsnorm.argtypes = [P, I64, I64, P, I64, I64, P, ctypes.c_float, P, P, I64, P]
        L.q4k_moe_workspace_size.restype = SZ
        L.q4k_moe_workspace_size.argtypes = [I32, I32, I32, I64, I64]
        L.q4k_moe_workspace_views.restype = ctypes.c_int
        L.q4k_moe_workspace_views.argtypes = [I32, I32, I32, I64, I64, ctypes.POINTER(ctypes.c_uint64)]
        L.q4k_moe_gemv.restype = ctypes.c_int
        L.q4k_moe_gemv.argtypes = [P, P, P, I64, I32, I64, I64, P, I32, I64, P, P, I32, P, I64,
                                   P, SZ, P]
        L.q4k_moe_gemv_ex.restype = ctypes.c_int
        L.q4k_moe_gemv_ex.argtypes = [P, P, P, I64, I32, I64, I64, P, I32, I64, P, P, I32, P, I64,
                                      ctypes.c_uint32, P, SZ, P]
        L.q4k_moe_prefill_workspace_size.restype = SZ
        L.q4k_moe_prefill_workspace_size.argtypes = [I32, I32, I32, I64, I64]
        L.q4k_moe_prefill.restype = ctypes.c_int
        L.q4k_moe_prefill.argtypes = [P, P, P, I64, I32, I64, I64, P, I32, I64, P, P, I32, P, I64,
                                      P, SZ, P]
        L.q4k_moe_gemv_noalloc.restype = ctypes.c_int
        L.q4k_moe_gemv_noalloc.argtypes = [P, P, P, I64, I32, I64, I64, P, I32, I64, P, P, I32, P,
                                           I64, P]
        F32 = ctypes.c_float
        L.q4k_kv_plan.restype = ctypes.c_int
        L.q4k_kv_plan.argtypes = [P, P, I32, P, I64, I32, I32, P, I32, P, P, P, P, P, I64, P, P, P]
        L.q4k_kv_write.restype = ctypes.c_int
        L.q4k_kv_write.argtypes = [P, P, ctypes.c_int, I64, I64, P, I64, I32, I32, P, P, ctypes.c_int,
                                   I64, I32, I64, I64, I64, P, P, P]
        L.q4k_paged_attn_workspace_size.restype = SZ
        L.q4k_paged_attn_workspace_size.argtypes = [I32, I32, I32, I32]
        L.q4k_paged_attn.restype = ctypes.c_int
        L.q4k_paged_attn.argtypes = [P, I64, I64, I32, I32, I32, I32, P, P, ctypes.c_int, I64, I32, I64,
                                     I64, I64, P, P, P, I64, I32, P, F32, I32, P, I64, P, P, SZ, P]
        L.q4k_add_rmsnorm.restype = ctypes.c_int
        L.q4k_add_rmsnorm.argtypes = [P, ctypes.c_int, I64, P, ctypes.c_int, I64, P, F32, I64, I64, P,
                                      ctypes.c_int, I64, P, I64, P, I64, P]
        L.q4k_sample.restype = ctypes.c_int
        L.q4k_sample.argtypes = [P, ctypes.c_int, I64, I64, I64, P, P, P, P, P, P, P, P]
        L.q4k_get_device_error.restype = ctypes.c_int
        L.q4k_get_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
        L.q4k_selftest_wait_timeout.restype = ctypes.c_int
        L.q4k_selftest_wait_timeout.argtypes = [P]
        _lib = L
        return L


def status_str(status: int) -> str:
    try:
        return lib().q4k_status_str(int(status)).decode()
    except RuntimeError:
        return "library not built"


def _check(status: int, what: str) -> None:
    if status != 0:
        raise Q4KError(status, what)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def q4k_abi_version() -> int:
    return int(lib().q4k_abi_version())


def q4k_dequant(w: torch.Tensor, n: int, k: int, out_dtype=torch.float32, out=None, stream=None):
    """Dense N x K weights (fp32 or bf16) from an N x K Q4_K matrix on the GPU."""
    if out is None:
        out = torch.empty((n, k), dtype=out_dtype, device=w.device)
    code = {torch.float32: 0, torch.bfloat16: 1}[out.dtype]
    _check(lib().q4k_dequant(_ptr(w), n, k, _ptr(out), code, _stream(stream)), "q4k_dequant")
    return out


def q4k_gemv(w: torch.Tensor, n: int, k: int, x: torch.Tensor, out=None, stream=None):
    """Y[b] = W X[b] for X of shape [batch, K] (or [K]) bf16; returns fp32 [batch, N]."""
    x2 = x.unsqueeze(0) if x.dim() == 1 else x
    batch = x2.shape[0]
    if out is None:
        out = torch.empty((batch, n), dtype=torch.float32, device=x.device)
    _check(lib().q4k_gemv(_ptr(w), n, k, _ptr(x2), batch, x2.stride(0), _ptr(out), out.stride(0),
                          _stream(stream)), "q4k_gemv")
    return out[0] if x.dim() == 1 else out


def q4k_gemv_ex(w: torch.Tensor, n: int, k: int, x: torch.Tensor, flags: int, out=None,
                stream=None):
    """q4k_gemv with flags (Q4K_FLAG_OVERLAP_WEIGHTS)."""
    x2 = x.unsqueeze(0) if x.dim() == 1 else x
    batch = x2.shape[0]
    if out is None:
        out = torch.empty((batch, n), dtype=torch.float32, device=x.device)
    _check(lib().q4k_gemv_ex(_ptr(w), n, k, _ptr(x2), batch, x2.stride(0), _ptr(out),
                             out.stride(0), flags, _stream(stream)), "q4k_gemv_ex")
    return out[0] if x.dim() == 1 else out


def q4k_gemv_glu(w_gate: torch.Tensor, w_up: torch.Tensor, n: int, k: int, x: torch.Tensor,
                 flags: int = 0, out=None, stream=None):
    """H[b] = silu(Wg X[b]) * (Wu X[b]) for X [batch, K] (or [K]) bf16; fp32 [batch, N]."""
    x2 = x.unsqueeze(0) if x.dim() == 1 else x
    batch = x2.shape[0]
    if out is None:
        out = torch.empty((batch, n), dtype=torch.float32, device=x.device)
    _check(lib().q4k_gemv_glu(_ptr(w_gate), _ptr(w_up), n, k, _ptr(x2), batch, x2.stride(0),
                              _ptr(out), out.stride(0), flags, _stream(stream)), "q4k_gemv_glu")
    return out[0] if x.dim() == 1 else out


def gemv_ops(ops) -> ctypes.Array:
    """The op array of q4k_gemv_seq from (w, n, k, x, y) tuples, or
    (w_gate, n, k, x, y, w_up) for a fused gate/up op: x [batch, K] bf16 and
    y [batch, N] fp32 on the device.  The array holds raw pointers; keep the
    tensors alive while it is used.  Build it once and reuse it."""
    arr = (GemvOp * len(ops))()
    for i, op in enumerate(ops):
        w, n, k, x, y = op[:5]
        w_up = op[5] if len(op) > 5 else None
        x2 = x.unsqueeze(0) if x.dim() == 1 else x
        y2 = y.unsqueeze(0) if y.dim() == 1 else y
        arr[i] = GemvOp(_ptr(w), n, k, _ptr(x2), x2.stride(0), _ptr(y2), y2.stride(0), _ptr(w_up))
    return arr


def q4k_gemv_seq(ops, batch: int, flags: int = 0, stream=None) -> None:
    """Launch a sequence of projections in order (ops: gemv_ops(...) or a
    list of (w, n, k, x, y) tuples), as q4k_gemv_ex for each in turn."""
    arr = ops if isinstance(ops, ctypes.Array) else gemv_ops(ops)
    _check(lib().q4k_gemv_seq(arr, len(arr), batch, flags, _stream(stream)), "q4k_gemv_seq")


def q4k_gemm(w: torch.Tensor, n: int, k: int, x: torch.Tensor, out=None, stream=None):
    """Y = X W^T for X [M, K] bf16; returns bf16 [M, N]."""
    m = x.shape[0]
    if out is None:  # the C ABI wants a row stride that is a multiple of 8
        ld = (n + 7) // 8 * 8
        out = torch.empty((m, ld), dtype=torch.bfloat16, device=x.device)[:, :n]
    _check(lib().q4k_gemm(_ptr(w), n, k, _ptr(x), m, x.stride(0), _ptr(out), out.stride(0),
                          _stream(stream)), "q4k_gemm")
    return out


Q4K_FMT_Q2_K, Q4K_FMT_Q3_K, Q4K_FMT_Q4_K, Q4K_FMT_Q5_K, Q4K_FMT_Q6_K = 2, 3, 4, 5, 6


def q4k_kq_block_bytes(fmt: int) -> int:
    return int(lib().q4k_kq_block_bytes(fmt))


def q4k_kq_dequant(fmt: int, w: torch.Tensor, n: int, k: int, dtype=torch.float32, stream=None):
    """Dense weights of an n x k matrix of k-quant format fmt (fp32 or bf16)."""
    out = torch.empty((n, k), dtype=dtype, device=w.device)
    _check(lib().q4k_kq_dequant(fmt, _ptr(w), n, k, _ptr(out), 1 if dtype == torch.bfloat16 else 0,
                                _stream(stream)), "q4k_kq_dequant")
    return out


def q4k_kq_gemv(fmt: int, w: torch.Tensor, n: int, k: int, x: torch.Tensor, out=None, stream=None):
    """Y = X W^T for x [batch, k] bf16 and a k-quant matrix of format fmt; fp32 [batch, n]."""
    x2 = x if x.dim() == 2 else x.view(1, -1)
    batch = x2.shape[0]
    if out is None:
        out = torch.empty((batch, n), dtype=torch.float32, device=x.device)
    _check(lib().q4k_kq_gemv(fmt, _ptr(w), n, k, _ptr(x2), batch, x2.stride(0), _ptr(out),
                             out.stride(0), _stream(stream)), "q4k_kq_gemv")
    return out


def q4k_kq_gemv_seq(fmt: int, ops, batch: int, flags: int = 0, stream=None) -> None:
    """q4k_gemv_seq for k-quant matrices of format fmt (ops: gemv_ops(...) of
    (w, n, k, x, y) tuples, or such a list), as q4k_kq_gemv for each in turn."""
    arr = ops if isinstance(ops, ctypes.Array) else gemv_ops(ops)
    _check(lib().q4k_kq_gemv_seq(fmt, arr, len(arr), batch, flags, _stream(stream)),
           "q4k_kq_gemv_seq")


def q4k_gemm_rmsnorm(w: torch.Tensor, n: int, k: int, x: torch.Tensor, gamma: torch.Tensor,
                     eps: float, out=None, rinv=None, stream=None):
    """Y = rinv * (X (W diag(gamma))^T), rinv = 1/sqrt(mean(X^2) + eps) per token;
    returns (Y bf16 [M, N], rinv fp32 [M])."""
    m = x.shape[0]
    if out is None:
        ld = (n + 7) // 8 * 8
        out = torch.empty((m, ld), dtype=torch.bfloat16, device=x.device)[:, :n]
    if rinv is None:
        rinv = torch.empty(m, dtype=torch.float32, device=x.device)
    _check(lib().q4k_gemm_rmsnorm(_ptr(w), n, k, _ptr(x), m, x.stride(0), _ptr(gamma), float(eps),
                                  _ptr(rinv), _ptr(out), out.stride(0), _stream(stream)),
           "q4k_gemm_rmsnorm")
    return out, rinv


def q4k_moe_workspace_size(n_experts: int, n_tokens: int, top_k: int, hidden: int, ffn: int) -> int:
    return int(lib().q4k_moe_workspace_size(n_experts, n_tokens, top_k, hidden, ffn))


def q4k_moe_workspace_views(n_experts: int, n_tokens: int, top_k: int, hidden: int,
                            ffn: int) -> dict:
    """Byte offsets of the intermediate results q4k_moe_gemv leaves in its
    workspace: pair index per (token, slot), g, u, h and the down outputs."""
    arr = (ctypes.c_uint64 * 5)()
    _check(lib().q4k_moe_workspace_views(n_experts, n_tokens, top_k, hidden, ffn, arr),
           "q4k_moe_workspace_views")
    return dict(zip(("tj_pair", "g", "u", "h", "p"), (int(v) for v in arr)))


def q4k_moe_gemv(w_gate, w_up, w_down, expert_stride: int, n_experts: int, hidden: int, ffn: int,
                 x: torch.Tensor, ids: torch.Tensor, wts: torch.Tensor, out=None, workspace=None,
                 stream=None):
    """Routed-expert FFN for decode tokens; returns fp32 [T, hidden]."""
    T, top_k = ids.shape
    if out is None:
        out = torch.empty((T, hidden), dtype=torch.float32, device=x.device)
    ws_bytes = q4k_moe_workspace_size(n_experts, T, top_k, hidden, ffn)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib().q4k_moe_gemv(_ptr(w_gate), _ptr(w_up), _ptr(w_down), expert_stride, n_experts,
                              hidden, ffn, _ptr(x), T, x.stride(0), _ptr(ids), _ptr(wts), top_k,
                              _ptr(out), out.stride(0), _ptr(workspace), workspace.numel(),
                              _stream(stream)), "q4k_moe_gemv")
    return out


def q4k_moe_gemv_ex(w_gate, w_up, w_down, expert_stride: int, n_experts: int, hidden: int,
                    ffn: int, x: torch.Tensor, ids: torch.Tensor, wts: torch.Tensor, flags: int = 0,
                    out=None, workspace=None, stream=None):
    """q4k_moe_gemv with flags (Q4K_MOE_WEIGHTED_DOWN); returns fp32 [T, hidden]."""
    T, top_k = ids.shape
    if out is None:
        out = torch.empty((T, hidden), dtype=torch.float32, device=x.device)
    ws_bytes = q4k_moe_workspace_size(n_experts, T, top_k, hidden, ffn)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib().q4k_moe_gemv_ex(_ptr(w_gate), _ptr(w_up), _ptr(w_down), expert_stride, n_experts,
                                 hidden, ffn, _ptr(x), T, x.stride(0), _ptr(ids), _ptr(wts), top_k,
                                 _ptr(out), out.stride(0), flags, _ptr(workspace),
                                 workspace.numel(), _stream(stream)), "q4k_moe_gemv_ex")
    return out


def q4k_moe_prefill_workspace_size(n_experts: int, n_tokens: int, top_k: int, hidden: int,
                                   ffn: int) -> int:
    return int(lib().q4k_moe_prefill_workspace_size(n_experts, n_tokens, top_k, hidden, ffn))


def q4k_moe_prefill(w_gate, w_up, w_down, expert_stride: int, n_experts: int, hidden: int,
                    ffn: int, x: torch.Tensor, ids: torch.Tensor, wts: torch.Tensor, out=None,
                    workspace=None, stream=None):
    """Routed-expert FFN for a block of tokens (grouped tensor-core GEMMs);
    returns fp32 [T, hidden]."""
    T, top_k = ids.shape
    if out is None:
        out = torch.empty((T, hidden), dtype=torch.float32, device=x.device)
    ws_bytes = q4k_moe_prefill_workspace_size(n_experts, T, top_k, hidden, ffn)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib().q4k_moe_prefill(_ptr(w_gate), _ptr(w_up), _ptr(w_down), expert_stride, n_experts,
                                 hidden, ffn, _ptr(x), T, x.stride(0), _ptr(ids), _ptr(wts), top_k,
                                 _ptr(out), out.stride(0), _ptr(workspace), workspace.numel(),
                                 _stream(stream)), "q4k_moe_prefill")
    return out


def q4k_moe_gemv_noalloc(w_gate, w_up, w_down, expert_stride: int, n_experts: int, hidden: int,
                         ffn: int, x: torch.Tensor, ids: torch.Tensor, wts: torch.Tensor, out=None,
                         stream=None):
    """q4k_moe_gemv with the library's own fixed device workspace (no allocation)."""
    T, top_k = ids.shape
    if out is None:
        out = torch.empty((T, hidden), dtype=torch.float32, device=x.device)
    _check(lib().q4k_moe_gemv_noalloc(_ptr(w_gate), _ptr(w_up), _ptr(w_down), expert_stride,
                                      n_experts, hidden, ffn, _ptr(x), T, x.stride(0), _ptr(ids),
                                      _ptr(wts), top_k, _ptr(out), out.stride(0), _stream(stream)),
           "q4k_moe_gemv_noalloc")
    return out


# ---- Around the projections.  A decode step makes hundreds of these calls, and a call of some
# microseconds on the device should not wait for its arguments: the checks below are plain
# comparisons, and the current stream is asked for by device index (3.0 us less per call than
# torch.cuda.current_stream() on the GB300's host).

_I32, _I64, _F32, _BF16, _E4M3 = (torch.int32, torch.int64, torch.float32, torch.bfloat16,
                                  torch.float8_e4m3fn)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(what: str, t) -> None:
    raise Q4KError(2, f"{what} is {t.dtype} {tuple(t.shape)}, strides {tuple(t.stride())}"
                   if isinstance(t, torch.Tensor) else f"{what} is {type(t).__name__}, not a tensor")


def _vec(what: str, t: torch.Tensor, n: int, dtype) -> int:
    """The address of a contiguous vector of n values of this type; raises Q4KError otherwise."""
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        _refuse(what, t)
    return t.data_ptr()


def _rows(what: str, t: torch.Tensor, m: int, n: int, dtype) -> int:
    """The row stride of an m x n matrix of this type with contiguous rows.  (The stride of a single
    row is never used and may be anything in torch: n stands in for it.)"""
    if t.dtype is not dtype or t.shape != (m, n) or (n > 1 and t.stride(1) != 1):
        _refuse(what, t)
    return t.stride(0) if m != 1 else n


def _call_stream(stream, t: torch.Tensor) -> int:
    if stream is not None or _raw_stream is None or not t.is_cuda:
        return _stream(stream)
    return _raw_stream(t.get_device())


def _on(stream):
    """Outputs and workspaces that a call makes belong to the stream it runs on (the allocator may
    otherwise hand them out again while the call still uses them)."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _empty(shape, dtype, like: torch.Tensor, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def q4k_kv_plan(lens: torch.Tensor, add: torch.Tensor, table: torch.Tensor, pool: torch.Tensor,
                pool_state: torch.Tensor, page_size: int, n_slots: int, out=None, stream=None):
    """Block tables and slot maps of a step from request lengths (int32 tensors): lens, add [n] (-1:
    finished), table [n, max_pages] and pool [pages] (both updated in place), pool_state [2].
    Returns (lens_out [n], cu [n + 1] int64, slots [n_slots], pos [n_slots], status [n],
    pool_state_out [2]); out gives these six tensors (lens and pool_state may be among them)."""
    n, width, pages = lens.numel(), table.shape[-1], pool.numel()
    if n == 0 and not pool_state.is_cuda:  # (without a GPU the library's empty calls succeed and write nothing)
        raise Q4KError(8, "pool_state")
    if out is None:
        if n_slots < 0:
            raise Q4KError(2, f"n_slots is {n_slots}")
        lens_out, status = _empty(n, _I32, lens, stream), _empty(n, _I32, lens, stream)
        slots, pos = _empty(n_slots, _I32, lens, stream), _empty(n_slots, _I32, lens, stream)
        cu, state_out = _empty(n + 1, _I64, lens, stream), _empty(2, _I32, lens, stream)
        to = (lens_out.data_ptr(), cu.data_ptr(), slots.data_ptr(), pos.data_ptr(),
              status.data_ptr(), state_out.data_ptr())
    else:
        lens_out, cu, slots, pos, status, state_out = out
        to = (_vec("lens_out", lens_out, n, _I32), _vec("cu", cu, n + 1, _I64),
              _vec("slots", slots, n_slots, _I32), _vec("pos", pos, n_slots, _I32),
              _vec("status", status, n, _I32), _vec("pool_state_out", state_out, 2, _I32))
    ldt = _rows("table", table, n, width, _I32)
    _check((_lib or lib()).q4k_kv_plan(
        _vec("lens", lens, n, _I32), _vec("add", add, n, _I32), n, table.data_ptr(), ldt, width,
        page_size, _vec("pool", pool, pages, _I32), pages, _vec("pool_state", pool_state, 2, _I32),
        to[0], to[1], to[2], to[3], n_slots, to[4], to[5], _call_stream(stream, lens)), "q4k_kv_plan")
    return lens_out, cu, slots, pos, status, state_out


def _outer_strides(t: torch.Tensor):
    """Strides of all dimensions but the last (which has to be contiguous).  The stride of a dimension
    of size 1 is never used and may be anything in torch: it is given as if t were contiguous there."""
    st, shape = t.stride(), t.shape
    if st[-1] != 1 and shape[-1] > 1:
        _refuse("a tensor with a strided last dimension", t)
    if 1 not in shape:
        return st[:-1]
    out, span = list(st[:-1]), shape[-1]
    for i in range(len(out) - 1, -1, -1):
        if shape[i] == 1:
            out[i] = span
        span = max(span, out[i] * shape[i])
    return tuple(out)


def _caches(k_cache, v_cache, k_scale, v_scale):
    """(shape, strides, type code, scale addresses) of the two cache buffers, after checking them."""
    shape, dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or (dtype is not _BF16 and dtype is not _E4M3):
        _refuse("k_cache", k_cache)
    if v_cache.shape != shape or v_cache.dtype is not dtype:
        _refuse("v_cache", v_cache)
    strides = _outer_strides(k_cache)
    if v_cache.stride() != k_cache.stride() and strides != _outer_strides(v_cache):
        raise Q4KError(2, "k_cache and v_cache have different strides")
    if dtype is _BF16:
        return shape, strides, 1, None, None
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is not None and (t.dtype is not _F32 or t.shape != shape[:3] or not t.is_contiguous()):
            _refuse(name, t)
    return shape, strides, 2, _ptr(k_scale), _ptr(v_scale)


def q4k_kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, k_scale=None, v_scale=None, stream=None) -> None:
    """Write rows k, v [tokens, heads, dim] (fp32 or bf16, same strides) to the slots [tokens] int32
    (-1: skip) of the paged caches [pages, heads, page size, dim], bf16 or e4m3 (then with scales
    [pages, heads, page size] fp32)."""
    shape, strides, code, ks, vs = _caches(k_cache, v_cache, k_scale, v_scale)
    pages, heads, page, dim = shape
    tokens, dtype = slots.numel(), k.dtype
    if k.shape != (tokens, heads, dim) or (dtype is not _F32 and dtype is not _BF16):
        _refuse("k", k)
    if v.shape != k.shape or v.dtype is not dtype:
        _refuse("v", v)
    ld = _outer_strides(k)
    if v.stride() != k.stride() and ld != _outer_strides(v):
        raise Q4KError(2, "k and v have different strides")
    _check((_lib or lib()).q4k_kv_write(
        k.data_ptr(), v.data_ptr(), 1 if dtype is _BF16 else 0, ld[0], ld[1],
        _vec("slots", slots, tokens, _I32), tokens, heads, dim, k_cache.data_ptr(),
        v_cache.data_ptr(), code, pages, page, strides[0], strides[1], strides[2], ks, vs,
        _call_stream(stream, k)), "q4k_kv_write")


def q4k_paged_attn_workspace_size(n: int, q_heads: int, kv_heads: int, dim: int) -> int:
    return int(lib().q4k_paged_attn_workspace_size(n, q_heads, kv_heads, dim))


def q4k_paged_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   table: torch.Tensor, lens: torch.Tensor, softmax_scale: float, k_scale=None,
                   v_scale=None, window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per request: q [n, q_heads, dim] bf16 over the paged caches
    [pages, kv_heads, page size, dim] (bf16, or e4m3 with scales) by table [n, max_pages] and lens
    [n] int32.  Returns (out [n, q_heads, dim] bf16, lse [n, q_heads] fp32)."""
    shape, strides, code, ks, vs = _caches(k_cache, v_cache, k_scale, v_scale)
    pages, heads, page, dim = shape
    L = _lib or lib()
    if q.dtype is not _BF16 or len(q.shape) != 3 or q.shape[2] != dim:
        _refuse("q", q)
    n, q_heads = q.shape[0], q.shape[1]
    ldq = _outer_strides(q)
    width = table.shape[-1]
    ldt = _rows("table", table, n, width, _I32)
    if out is None:
        out = _empty((n, q_heads, dim), _BF16, q, stream)
        ldo = q_heads * dim
    else:
        if out.dtype is not _BF16 or out.shape != q.shape:
            _refuse("out", out)
        ldo, inner = _outer_strides(out)
        if inner != dim:
            raise Q4KError(2, f"out has head stride {inner}, not {dim}")
    if lse is None:
        lse = _empty((n, q_heads), _F32, q, stream)
    elif lse.dtype is not _F32 or lse.shape != (n, q_heads) or not lse.is_contiguous():
        _refuse("lse", lse)
    if workspace is None:
        size = L.q4k_paged_attn_workspace_size(n, q_heads, heads, dim)
        workspace = _empty(max(size, 16), torch.uint8, q, stream)
    elif not workspace.is_contiguous():  # its elements would not be bytes of memory
        _refuse("workspace", workspace)
    _check(L.q4k_paged_attn(
        q.data_ptr(), ldq[0], ldq[1], n, q_heads, heads, dim, k_cache.data_ptr(),
        v_cache.data_ptr(), code, pages, page, strides[0], strides[1], strides[2], ks, vs,
        table.data_ptr(), ldt, width, _vec("lens", lens, n, _I32), softmax_scale, window,
        out.data_ptr(), ldo, lse.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _call_stream(stream, q)), "q4k_paged_attn")
    return out, lse


def q4k_add_rmsnorm(x: torch.Tensor, residual, gamma: torch.Tensor, eps: float,
                    out_dtype=torch.bfloat16, out=None, residual_out=None, scales=None, stream=None):
    """h = x + residual; y = h * gamma / sqrt(mean(h^2) + eps) for x, residual [m, hidden] fp32 or
    bf16 (residual may be None).  Returns (y, residual_out) with y bf16, or (y, residual_out, scales)
    with y e4m3 (out_dtype torch.float8_e4m3fn) and scales [m, ceil(hidden / 128)] fp32; residual_out
    may be residual itself, and is None where residual is."""
    dtype = x.dtype
    if len(x.shape) != 2 or (dtype is not _F32 and dtype is not _BF16):
        _refuse("x", x)
    m, hidden = x.shape
    ldx = _rows("x", x, m, hidden, dtype)
    res = res_out = res_dtype = None
    ldr = ldro = 0
    if residual is not None:
        res_dtype = residual.dtype
        if res_dtype is not _F32 and res_dtype is not _BF16:
            _refuse("residual", residual)
        ldr = _rows("residual", residual, m, hidden, res_dtype)
        res = residual.data_ptr()
        if residual_out is None:
            residual_out, ldro = _empty((m, hidden), res_dtype, x, stream), hidden
        else:
            ldro = _rows("residual_out", residual_out, m, hidden, res_dtype)
        res_out = residual_out.data_ptr()
    else:
        residual_out = None
    if out is None:
        out, ldy = _empty((m, hidden), out_dtype, x, stream), hidden
    else:
        out_dtype = out.dtype
        ldy = _rows("out", out, m, hidden, out_dtype)
    if out_dtype is _BF16:
        code, sc, lds = 1, None, 0
    elif out_dtype is _E4M3:
        code, blocks = 2, (hidden + 127) // 128
        if scales is None:
            scales, lds = _empty((m, blocks), _F32, x, stream), blocks
        else:
            lds = _rows("scales", scales, m, blocks, _F32)
        sc = scales.data_ptr()
    else:
        _refuse("out", out)
    _check((_lib or lib()).q4k_add_rmsnorm(
        x.data_ptr(), 1 if dtype is _BF16 else 0, ldx, res, 1 if res_dtype is _BF16 else 0, ldr,
        _vec("gamma", gamma, hidden, _F32), eps, m, hidden, out.data_ptr(), code, ldy, res_out, ldro,
        sc, lds, _call_stream(stream, x)), "q4k_add_rmsnorm")
    return (out, residual_out) if code == 1 else (out, residual_out, scales)


def q4k_sample(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None,
               min_p=None, out=None, logp=None, stream=None):
    """Choose a token per row of logits [rows, vocab] (fp32 or bf16) from the random numbers u [rows]
    fp32 in [0, 1); temperature, top_p, min_p (fp32) and top_k (int32) are [rows] or None (1, off).
    Returns (token [rows] int32, logp [rows] fp32)."""
    dtype = logits.dtype
    if len(logits.shape) != 2 or (dtype is not _F32 and dtype is not _BF16):
        _refuse("logits", logits)
    rows, vocab = logits.shape
    ld = _rows("logits", logits, rows, vocab, dtype)
    t = None if temperature is None else _vec("temperature", temperature, rows, _F32)
    k = None if top_k is None else _vec("top_k", top_k, rows, _I32)
    p = None if top_p is None else _vec("top_p", top_p, rows, _F32)
    mp = None if min_p is None else _vec("min_p", min_p, rows, _F32)
    if out is None:
        out = _empty(rows, _I32, logits, stream)
    if logp is None:
        logp = _empty(rows, _F32, logits, stream)
    _check((_lib or lib()).q4k_sample(
        logits.data_ptr(), 1 if dtype is _BF16 else 0, rows, vocab, ld, _vec("u", u, rows, _F32), t, k,
        p, mp, _vec("out", out, rows, _I32), _vec("logp", logp, rows, _F32),
        _call_stream(stream, logits)), "q4k_sample")
    return out, logp


def q4k_get_device_error(stream=None) -> int:
    """Synchronizes the stream, returns and clears the device error word."""
    bits = ctypes.c_uint32(0)
    st = lib().q4k_get_device_error(_stream(stream), ctypes.byref(bits))
    if st not in (0, 7):
        raise Q4KError(st, "q4k_get_device_error")
    return int(bits.value)


def q4k_selftest_wait_timeout(stream=None) -> None:
    """Launch the bounded-wait self test (a wait nothing completes; ~2 s)."""
    _check(lib().q4k_selftest_wait_timeout(_stream(stream)), "q4k_selftest_wait_timeout")
