// q4k_api.cu -- the extern "C" boundary of libq4k.so (declared in
// include/q4k.h): argument checks, device checks, launch, error mapping.
//
// "spec: specialized model runtimes", section "Architecture": the runtime is
// loaded in-process behind a C ABI; section "Prototype ABI scope": every
// failure returns a clean value its caller already handles (no exceptions, no
// aborts cross this boundary); section "Correctness and control": FFI pointer,
// length and error-path behaviour is tested.
#include <cuda_runtime.h>
#include <stdint.h>
#include <algorithm>

#include <initializer_list>
#include <mutex>
#include <vector>

#include "../../include/q4k.h"
#include "q4k_device.cuh"
#include "q4k_internal.h"
#include "q4k_step.h"

namespace q4k {

__device__ unsigned int g_device_error = 0u;

namespace {

DeviceFacts g_facts[kMaxDevices];
std::once_flag g_facts_once[kMaxDevices];
unsigned *g_err_ptr[kMaxDevices];
std::once_flag g_err_once[kMaxDevices];

void resolve_error_word(int dev) {
  void *p = nullptr;
  if (cudaGetSymbolAddress(&p, g_device_error) == cudaSuccess) g_err_ptr[dev] = static_cast<unsigned *>(p);
}

void query_facts(int dev) {
  DeviceFacts &f = g_facts[dev];
  f.device = dev;
  cudaDeviceGetAttribute(&f.major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&f.minor, cudaDevAttrComputeCapabilityMinor, dev);
  cudaDeviceGetAttribute(&f.sm_count, cudaDevAttrMultiProcessorCount, dev);
  cudaDeviceGetAttribute(&f.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  cudaDeviceGetAttribute(&f.max_smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  cudaDeviceGetAttribute(&f.l2_bytes, cudaDevAttrL2CacheSize, dev);
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

void resolve_encode() {
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Device check shared by every compute entry point.
int check_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return Q4K_ERR_CUDA;
  const DeviceFacts *f = device_facts();
  if (f->major != 10 || f->minor != 3) return Q4K_ERR_DEVICE;
  return Q4K_OK;
}

// No GPU at all, so that no pointer can be device memory.
bool no_device() {
  int count = 0;
  const cudaError_t e = cudaGetDeviceCount(&count);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver || (e == cudaSuccess && count == 0);
}

int map_launch(cudaError_t e) { return e == cudaSuccess ? Q4K_OK : Q4K_ERR_CUDA; }

// Q4K_OK when every non-null pointer is memory of the current device
// (cudaMalloc'd, not host, pinned, managed or another GPU's memory).  The
// kernels' TMA copies, and the prefill GEMM's cluster-multicast copy of X, are
// built over these addresses; they must read this GPU's own memory only.
// Every pointer is asked for by itself, about half a microsecond each: that a
// neighbour in the same 2 MB is device memory says nothing about memory that is
// freed or was never allocated.
int check_device_memory(std::initializer_list<const void *> ptrs) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return Q4K_ERR_CUDA;
  for (const void *p : ptrs) {
    if (!p) continue;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      (void)cudaGetLastError();  // the failed query leaves no error behind
      return Q4K_ERR_MEMORY;
    }
    if (at.type != cudaMemoryTypeDevice || at.device != dev) return Q4K_ERR_MEMORY;
  }
  return Q4K_OK;
}

static_assert(kMoeScratchBytes == Q4K_MOE_NOALLOC_SCRATCH_BYTES,
              "the allocation-free MoE array and its documented size must agree");

}  // namespace

const DeviceFacts *device_facts() {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) dev = 0;
  std::call_once(g_facts_once[dev], query_facts, dev);
  return &g_facts[dev];
}

unsigned *device_error_word() {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  std::call_once(g_err_once[dev], resolve_error_word, dev);
  return g_err_ptr[dev];
}

CUresult encode_tiled(CUtensorMap *map, CUtensorMapDataType type, uint32_t rank, void *addr,
                      const uint64_t *dims, const uint64_t *strides_bytes, const uint32_t *box,
                      CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promo) {
  std::call_once(g_encode_once, resolve_encode);
  if (!g_encode) return CUDA_ERROR_NOT_FOUND;
  cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  return g_encode(map, type, rank, addr, reinterpret_cast<const cuuint64_t *>(dims),
                  reinterpret_cast<const cuuint64_t *>(strides_bytes),
                  reinterpret_cast<const cuuint32_t *>(box), elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, promo, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

namespace {
// One warp waits, through the same bounded wait every kernel uses, on an
// mbarrier that no thread ever arrives at.  After the wall-clock limit the wait
// gives up, sets the timeout bit of the device error word and the kernel ends.
__global__ void selftest_wait_timeout_kernel(unsigned *err) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  (void)mbar_wait(&bar, 0, err);
}
}  // namespace

}  // namespace q4k

using namespace q4k;

extern "C" {

int q4k_abi_version(void) { return Q4K_ABI_VERSION; }

const char *q4k_status_str(int status) {
  switch (status) {
    case Q4K_OK: return "ok";
    case Q4K_ERR_NULL: return "null pointer";
    case Q4K_ERR_SHAPE: return "bad shape";
    case Q4K_ERR_ALIGN: return "misaligned pointer or stride";
    case Q4K_ERR_WORKSPACE: return "workspace missing or too small";
    case Q4K_ERR_DEVICE: return "device is not sm_103";
    case Q4K_ERR_CUDA: return "CUDA error";
    case Q4K_ERR_DATA: return "a kernel reported bad data";
    case Q4K_ERR_MEMORY: return "a pointer is not device memory of the current device";
    default: return "unknown status";
  }
}

int q4k_dequant(const void *w, int64_t n, int64_t k, void *out, int out_dtype, void *stream) {
  if (n < 0 || k <= 0 || (k % kQK) != 0 || (out_dtype != 0 && out_dtype != 1)) return Q4K_ERR_SHAPE;
  if (n == 0) return Q4K_OK;
  if (!w || !out) return Q4K_ERR_NULL;
  if (!aligned(w, 16) || !aligned(out, 16)) return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w, out});
  if (st != Q4K_OK) return st;
  return map_launch(launch_dequant(w, n, k, out, out_dtype, static_cast<cudaStream_t>(stream)));
}

namespace {
// Argument checks of one projection; Q4K_OK with *empty set when there is
// nothing to compute.
int check_gemv(const void *w, int64_t n, int64_t k, const void *x, int64_t batch, int64_t ldx,
               const float *y, int64_t ldy, uint32_t flags, bool *empty) {
  *empty = false;
  if (n < 0 || k <= 0 || (k % kQK) != 0 || batch < 0 || batch > 16) return Q4K_ERR_SHAPE;
  if (n > INT32_MAX / 2 || k / kQK > INT32_MAX / kBlockBytes) return Q4K_ERR_SHAPE;
  if (flags & ~(uint32_t)Q4K_FLAG_OVERLAP_WEIGHTS) return Q4K_ERR_SHAPE;
  if (n == 0 || batch == 0) {
    *empty = true;
    return Q4K_OK;
  }
  if (ldx < k || ldy < n) return Q4K_ERR_SHAPE;
  if (!w || !x || !y) return Q4K_ERR_NULL;
  if (!aligned(w, 16) || !aligned(x, 16) || !aligned(y, 4) || (ldx % 8) != 0) return Q4K_ERR_ALIGN;
  return Q4K_OK;
}
}  // namespace

namespace {
// Batch sizes the stream kernel takes (its batch-row strides are 32-bit; at
// batch 1 they are not used).
bool stream_batch(int64_t batch, int64_t ldx, int64_t ldy) {
  return batch == 1 || (batch <= stream_max_batch() && ldx <= INT32_MAX && ldy <= INT32_MAX);
}
int64_t stream_stride(int64_t batch, int64_t ld) { return batch == 1 ? 0 : ld; }

// One projection (plain, or fused gate/up when w_up is set) after its
// arguments were checked: batch 1..4 runs in the stream kernel; 5..16 in the
// 64-row tile kernel when the op has enough tiles to occupy the GPU, else in
// the per-op batched kernel.
int run_gemv(const void *w, const void *w_up, int64_t n, int64_t k, const void *x, int64_t batch,
             int64_t ldx, float *y, int64_t ldy, uint32_t flags, void *stream) {
  const bool overlap = (flags & Q4K_FLAG_OVERLAP_WEIGHTS) != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const StreamOpDesc d = {w, w_up, x, y, n, k, stream_stride(batch, ldx), stream_stride(batch, ldy)};
  if (stream_batch(batch, ldx, ldy)) return map_launch(launch_stream(&d, 1, (int)batch, overlap, s));
  if (ldx <= INT32_MAX && ldy <= INT32_MAX && wide_worth_it(&d, 1, (int)batch))
    return map_launch(launch_wide(&d, 1, (int)batch, overlap, s));
  return map_launch(launch_gemv(w, w_up, n, k, x, batch, ldx, y, ldy, overlap, s));
}
}  // namespace

int q4k_gemv_ex(const void *w, int64_t n, int64_t k, const void *x, int64_t batch, int64_t ldx,
                float *y, int64_t ldy, uint32_t flags, void *stream) {
  bool empty = false;
  int st = check_gemv(w, n, k, x, batch, ldx, y, ldy, flags, &empty);
  if (st != Q4K_OK || empty) return st;
  st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w, x, y});
  if (st != Q4K_OK) return st;
  return run_gemv(w, nullptr, n, k, x, batch, ldx, y, ldy, flags, stream);
}

int q4k_gemv(const void *w, int64_t n, int64_t k, const void *x, int64_t batch, int64_t ldx,
             float *y, int64_t ldy, void *stream) {
  return q4k_gemv_ex(w, n, k, x, batch, ldx, y, ldy, 0u, stream);
}

int q4k_gemv_glu(const void *w_gate, const void *w_up, int64_t n, int64_t k, const void *x,
                 int64_t batch, int64_t ldx, float *h, int64_t ldh, uint32_t flags, void *stream) {
  bool empty = false;
  int st = check_gemv(w_gate, n, k, x, batch, ldx, h, ldh, flags, &empty);
  if (st != Q4K_OK || empty) return st;
  if (!w_up) return Q4K_ERR_NULL;
  if (!aligned(w_up, 16)) return Q4K_ERR_ALIGN;
  st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w_gate, w_up, x, h});
  if (st != Q4K_OK) return st;
  return run_gemv(w_gate, w_up, n, k, x, batch, ldx, h, ldh, flags, stream);
}

int q4k_gemv_seq(const q4k_gemv_op *ops, int64_t count, int64_t batch, uint32_t flags,
                 void *stream) {
  if (count < 0) return Q4K_ERR_SHAPE;
  if (count == 0) return Q4K_OK;
  if (!ops) return Q4K_ERR_NULL;
  bool any = false;
  for (int64_t i = 0; i < count; ++i) {
    const q4k_gemv_op &o = ops[i];
    bool empty = false;
    const int st = check_gemv(o.w, o.n, o.k, o.x, batch, o.ldx, o.y, o.ldy, flags, &empty);
    if (st != Q4K_OK) return st;
    if (!empty && o.w_up && !aligned(o.w_up, 16)) return Q4K_ERR_ALIGN;
    any = any || !empty;
  }
  if (!any) return Q4K_OK;
  int st = check_device();
  if (st != Q4K_OK) return st;
  for (int64_t i = 0; i < count; ++i) {
    const q4k_gemv_op &o = ops[i];
    if (o.n == 0) continue;
    st = check_device_memory({o.w, o.w_up, o.x, o.y});
    if (st != Q4K_OK) return st;
  }
  const bool overlap = (flags & Q4K_FLAG_OVERLAP_WEIGHTS) != 0;
  bool strides32 = true;
  for (int64_t i = 0; i < count; ++i)
    strides32 = strides32 && (ops[i].n == 0 || (ops[i].ldx <= INT32_MAX && ops[i].ldy <= INT32_MAX));
  if (strides32 || batch == 1) {
    std::vector<StreamOpDesc> d;
    d.reserve((size_t)count);
    for (int64_t i = 0; i < count; ++i) {
      const q4k_gemv_op &o = ops[i];
      d.push_back(StreamOpDesc{o.w, o.w_up, o.x, o.y, o.n, o.k, stream_stride(batch, o.ldx),
                               stream_stride(batch, o.ldy)});
    }
    // one persistent launch streams every op's weights back to back
    if (batch <= stream_max_batch())
      return map_launch(
          launch_stream(d.data(), count, (int)batch, overlap, static_cast<cudaStream_t>(stream)));
    if (wide_worth_it(d.data(), count, (int)batch))
      return map_launch(
          launch_wide(d.data(), count, (int)batch, overlap, static_cast<cudaStream_t>(stream)));
  }
  for (int64_t i = 0; i < count; ++i) {
    const q4k_gemv_op &o = ops[i];
    if (o.n == 0) continue;
    st = map_launch(launch_gemv(o.w, o.w_up, o.n, o.k, o.x, batch, o.ldx, o.y, o.ldy, overlap,
                                static_cast<cudaStream_t>(stream)));
    if (st != Q4K_OK) return st;
  }
  return Q4K_OK;
}

int q4k_gemm(const void *w, int64_t n, int64_t k, const void *x, int64_t m, int64_t ldx, void *y,
             int64_t ldy, void *stream) {
  if (n < 0 || k <= 0 || (k % kQK) != 0 || m < 0) return Q4K_ERR_SHAPE;
  if (n > INT32_MAX / 2 || m > INT32_MAX / 2 || k > INT32_MAX / 2) return Q4K_ERR_SHAPE;
  if (n == 0 || m == 0) return Q4K_OK;
  if (ldx < k || ldy < n) return Q4K_ERR_SHAPE;
  if (!w || !x || !y) return Q4K_ERR_NULL;
  if (!aligned(w, 16) || !aligned(x, 16) || !aligned(y, 16) || (ldx % 8) != 0 || (ldy % 8) != 0)
    return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w, x, y});
  if (st != Q4K_OK) return st;
  return map_launch(launch_gemm(w, n, k, x, m, ldx, y, ldy, static_cast<cudaStream_t>(stream)));
}

int q4k_gemm_rmsnorm(const void *w, int64_t n, int64_t k, const void *x, int64_t m, int64_t ldx,
                     const float *gamma, float eps, float *rinv, void *y, int64_t ldy,
                     void *stream) {
  if (n < 0 || k <= 0 || (k % kQK) != 0 || m < 0) return Q4K_ERR_SHAPE;
  if (n > INT32_MAX / 2 || m > INT32_MAX / 2 || k > INT32_MAX / 2) return Q4K_ERR_SHAPE;
  if (!(eps >= 0.f) || eps > 3.0e38f) return Q4K_ERR_SHAPE;  // negative, NaN or infinite
  if (n == 0 || m == 0) return Q4K_OK;
  if (ldx < k || ldy < n) return Q4K_ERR_SHAPE;
  if (!w || !x || !y || !gamma || !rinv) return Q4K_ERR_NULL;
  if (!aligned(w, 16) || !aligned(x, 16) || !aligned(y, 16) || (ldx % 8) != 0 || (ldy % 8) != 0 ||
      !aligned(gamma, 16) || !aligned(rinv, 4))
    return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w, x, y, gamma, rinv});
  if (st != Q4K_OK) return st;
  return map_launch(launch_gemm_rmsnorm(w, n, k, x, m, ldx, gamma, eps, rinv, y, ldy,
                                        static_cast<cudaStream_t>(stream)));
}

int q4k_kq_block_bytes(int32_t format) {
  return format == 4 ? kBlockBytes : kq_block_bytes(format);
}

int q4k_kq_dequant(int32_t format, const void *w, int64_t n, int64_t k, void *out, int out_dtype,
                   void *stream) {
  if (format == 4) return q4k_dequant(w, n, k, out, out_dtype, stream);
  if (kq_block_bytes(format) == 0) return Q4K_ERR_SHAPE;
  if (n < 0 || k <= 0 || (k % kQK) != 0 || (out_dtype != 0 && out_dtype != 1)) return Q4K_ERR_SHAPE;
  if (n == 0) return Q4K_OK;
  if (!w || !out) return Q4K_ERR_NULL;
  if (!aligned(w, 16) || !aligned(out, 16)) return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w, out});
  if (st != Q4K_OK) return st;
  return map_launch(
      launch_kq_dequant(format, w, n, k, out, out_dtype, static_cast<cudaStream_t>(stream)));
}

namespace {
// The k-quant projections the tensor-core stream kernel takes: batch 1..4
// (with 32-bit batch-row strides beyond batch 1), as for Q4_K.
bool kq_stream(int32_t format, int64_t batch, int64_t ldx, int64_t ldy) {
  (void)format;
  return stream_batch(batch, ldx, ldy);
}
// Argument checks of one k-quant projection (format != 4), before any launch.
int check_kq(int32_t format, const void *w, int64_t n, int64_t k, const void *x, int64_t batch,
             int64_t ldx, const float *y, int64_t ldy, bool *empty) {
  *empty = false;
  if (kq_block_bytes(format) == 0) return Q4K_ERR_SHAPE;
  if (n < 0 || k <= 0 || (k % kQK) != 0 || batch < 0 || batch > 16) return Q4K_ERR_SHAPE;
  if (n > INT32_MAX / 2 || kq_gemv_smem(format, k) > 227 * 1024) return Q4K_ERR_SHAPE;
  if (n == 0 || batch == 0) {
    *empty = true;
    return Q4K_OK;
  }
  if (ldx < k || ldy < n) return Q4K_ERR_SHAPE;
  if (!w || !x || !y) return Q4K_ERR_NULL;
  if (!aligned(w, 16) || !aligned(x, 16) || (ldx % 8) != 0 || !aligned(y, 4)) return Q4K_ERR_ALIGN;
  return Q4K_OK;
}
}  // namespace

int q4k_kq_gemv(int32_t format, const void *w, int64_t n, int64_t k, const void *x, int64_t batch,
                int64_t ldx, float *y, int64_t ldy, void *stream) {
  if (format == 4) return q4k_gemv(w, n, k, x, batch, ldx, y, ldy, stream);
  bool empty = false;
  int st = check_kq(format, w, n, k, x, batch, ldx, y, ldy, &empty);
  if (st != Q4K_OK || empty) return st;
  st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w, x, y});
  if (st != Q4K_OK) return st;
  if (kq_stream(format, batch, ldx, ldy)) {  // tensor cores, as Q4_K
    const StreamOpDesc d = {w, nullptr, x, y, n, k, stream_stride(batch, ldx), stream_stride(batch, ldy)};
    return map_launch(
        launch_stream(&d, 1, (int)batch, false, static_cast<cudaStream_t>(stream), format));
  }
  return map_launch(launch_kq_gemv(format, w, n, k, x, batch, ldx, y, ldy,
                                   static_cast<cudaStream_t>(stream)));
}

int q4k_kq_gemv_seq(int32_t format, const q4k_gemv_op *ops, int64_t count, int64_t batch,
                    uint32_t flags, void *stream) {
  if (format == 4) return q4k_gemv_seq(ops, count, batch, flags, stream);
  if (kq_block_bytes(format) == 0 || count < 0) return Q4K_ERR_SHAPE;
  if (flags & ~(uint32_t)Q4K_FLAG_OVERLAP_WEIGHTS) return Q4K_ERR_SHAPE;
  if (count == 0) return Q4K_OK;
  if (!ops) return Q4K_ERR_NULL;
  bool any = false;
  for (int64_t i = 0; i < count; ++i) {
    const q4k_gemv_op &o = ops[i];
    bool empty = false;
    const int st = check_kq(format, o.w, o.n, o.k, o.x, batch, o.ldx, o.y, o.ldy, &empty);
    if (st != Q4K_OK) return st;
    if (o.w_up) return Q4K_ERR_SHAPE;  // no fused gate/up for these formats
    any = any || !empty;
  }
  if (!any) return Q4K_OK;
  int st = check_device();
  if (st != Q4K_OK) return st;
  for (int64_t i = 0; i < count; ++i) {
    const q4k_gemv_op &o = ops[i];
    if (o.n == 0) continue;
    st = check_device_memory({o.w, o.x, o.y});
    if (st != Q4K_OK) return st;
  }
  const bool overlap = (flags & Q4K_FLAG_OVERLAP_WEIGHTS) != 0;
  bool on_stream = true;
  for (int64_t i = 0; i < count; ++i)
    on_stream = on_stream && (ops[i].n == 0 || kq_stream(format, batch, ops[i].ldx, ops[i].ldy));
  if (on_stream) {  // persistent launches of the tensor-core stream kernel
    std::vector<StreamOpDesc> d;
    d.reserve((size_t)count);
    for (int64_t i = 0; i < count; ++i) {
      const q4k_gemv_op &o = ops[i];
      d.push_back(StreamOpDesc{o.w, nullptr, o.x, o.y, o.n, o.k, stream_stride(batch, o.ldx),
                               stream_stride(batch, o.ldy)});
    }
    return map_launch(launch_stream(d.data(), count, (int)batch, overlap,
                                    static_cast<cudaStream_t>(stream), format));
  }
  for (int64_t i = 0; i < count; ++i) {
    const q4k_gemv_op &o = ops[i];
    if (o.n == 0) continue;
    st = map_launch(launch_kq_gemv(format, o.w, o.n, o.k, o.x, batch, o.ldx, o.y, o.ldy,
                                   static_cast<cudaStream_t>(stream)));
    if (st != Q4K_OK) return st;
  }
  return Q4K_OK;
}

size_t q4k_moe_workspace_size(int32_t n_experts, int32_t n_tokens, int32_t top_k, int64_t hidden,
                              int64_t ffn) {
  if (n_experts <= 0 || n_tokens < 0 || top_k <= 0 || hidden <= 0 || ffn <= 0) return 0;
  return moe_workspace_size(n_experts, n_tokens, top_k, hidden, ffn);
}

int q4k_moe_workspace_views(int32_t n_experts, int32_t n_tokens, int32_t top_k, int64_t hidden,
                            int64_t ffn, uint64_t offsets[5]) {
  if (!offsets) return Q4K_ERR_NULL;
  if (n_experts <= 0 || n_tokens <= 0 || top_k <= 0 || hidden <= 0 || ffn <= 0) return Q4K_ERR_SHAPE;
  moe_workspace_views(n_experts, n_tokens, top_k, hidden, ffn, offsets);
  return Q4K_OK;
}

int q4k_moe_gemv(const void *w_gate, const void *w_up, const void *w_down, int64_t expert_stride,
                 int32_t n_experts, int64_t hidden, int64_t ffn, const void *x, int32_t n_tokens,
                 int64_t ldx, const int32_t *ids, const float *wts, int32_t top_k, float *y,
                 int64_t ldy, void *workspace, size_t workspace_bytes, void *stream) {
  return q4k_moe_gemv_ex(w_gate, w_up, w_down, expert_stride, n_experts, hidden, ffn, x, n_tokens,
                         ldx, ids, wts, top_k, y, ldy, 0u, workspace, workspace_bytes, stream);
}

int q4k_moe_gemv_ex(const void *w_gate, const void *w_up, const void *w_down,
                    int64_t expert_stride, int32_t n_experts, int64_t hidden, int64_t ffn,
                    const void *x, int32_t n_tokens, int64_t ldx, const int32_t *ids,
                    const float *wts, int32_t top_k, float *y, int64_t ldy, uint32_t flags,
                    void *workspace, size_t workspace_bytes, void *stream) {
  if (flags & ~(uint32_t)Q4K_MOE_WEIGHTED_DOWN) return Q4K_ERR_SHAPE;
  if (n_experts <= 0 || n_experts > 2048 || hidden <= 0 || ffn <= 0 || (hidden % kQK) ||
      (ffn % kQK) || n_tokens < 0 || n_tokens > 64 || top_k < 1 || top_k > 16)
    return Q4K_ERR_SHAPE;
  if (hidden > (1 << 20) || ffn > (1 << 20)) return Q4K_ERR_SHAPE;
  if (expert_stride < (ffn * hidden / kQK) * kBlockBytes) return Q4K_ERR_SHAPE;
  if (n_tokens == 0) return Q4K_OK;
  if (ldx < hidden || ldy < hidden) return Q4K_ERR_SHAPE;
  if (!w_gate || !w_up || !w_down || !x || !ids || !wts || !y) return Q4K_ERR_NULL;
  if (!workspace ||
      workspace_bytes < moe_workspace_size(n_experts, n_tokens, top_k, hidden, ffn))
    return Q4K_ERR_WORKSPACE;
  if (!aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) || (expert_stride % 16) ||
      !aligned(x, 16) || (ldx % 8) || !aligned(y, 4) || !aligned(ids, 4) || !aligned(wts, 4) ||
      !aligned(workspace, 16))
    return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w_gate, w_up, w_down, x, ids, wts, y, workspace});
  if (st != Q4K_OK) return st;
  return map_launch(launch_moe(w_gate, w_up, w_down, expert_stride, n_experts, hidden, ffn, x,
                               n_tokens, ldx, ids, wts, top_k, y, ldy, workspace,
                               (flags & Q4K_MOE_WEIGHTED_DOWN) != 0,
                               static_cast<cudaStream_t>(stream)));
}

size_t q4k_moe_prefill_workspace_size(int32_t n_experts, int32_t n_tokens, int32_t top_k,
                                      int64_t hidden, int64_t ffn) {
  if (n_experts <= 0 || n_tokens < 0 || top_k <= 0 || hidden <= 0 || ffn <= 0) return 0;
  return moe_prefill_workspace_size(n_experts, n_tokens, top_k, hidden, ffn);
}

int q4k_moe_prefill(const void *w_gate, const void *w_up, const void *w_down,
                    int64_t expert_stride, int32_t n_experts, int64_t hidden, int64_t ffn,
                    const void *x, int32_t n_tokens, int64_t ldx, const int32_t *ids,
                    const float *wts, int32_t top_k, float *y, int64_t ldy, void *workspace,
                    size_t workspace_bytes, void *stream) {
  if (n_experts <= 0 || n_experts > 2048 || hidden <= 0 || ffn <= 0 || (hidden % kQK) ||
      (ffn % kQK) || n_tokens < 0 || n_tokens > 65535 || top_k < 1 || top_k > 16)
    return Q4K_ERR_SHAPE;
  if (hidden > (1 << 20) || ffn > (1 << 20)) return Q4K_ERR_SHAPE;
  if ((int64_t)n_tokens * top_k * (hidden > ffn ? hidden : ffn) > ((int64_t)1 << 31))
    return Q4K_ERR_SHAPE;
  if (expert_stride < (ffn * hidden / kQK) * kBlockBytes) return Q4K_ERR_SHAPE;
  if (n_tokens == 0) return Q4K_OK;
  if (ldx < hidden || ldy < hidden) return Q4K_ERR_SHAPE;
  if (!w_gate || !w_up || !w_down || !x || !ids || !wts || !y) return Q4K_ERR_NULL;
  if (!workspace ||
      workspace_bytes < moe_prefill_workspace_size(n_experts, n_tokens, top_k, hidden, ffn))
    return Q4K_ERR_WORKSPACE;
  if (!aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) || (expert_stride % 16) ||
      !aligned(x, 16) || (ldx % 8) || !aligned(y, 4) || !aligned(ids, 4) || !aligned(wts, 4) ||
      !aligned(workspace, 16))
    return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w_gate, w_up, w_down, x, ids, wts, y, workspace});
  if (st != Q4K_OK) return st;
  return map_launch(launch_moe_prefill(w_gate, w_up, w_down, expert_stride, n_experts, hidden, ffn,
                                       x, n_tokens, ldx, ids, wts, top_k, y, ldy, workspace,
                                       static_cast<cudaStream_t>(stream)));
}

int q4k_moe_gemv_noalloc(const void *w_gate, const void *w_up, const void *w_down,
                         int64_t expert_stride, int32_t n_experts, int64_t hidden, int64_t ffn,
                         const void *x, int32_t n_tokens, int64_t ldx, const int32_t *ids,
                         const float *wts, int32_t top_k, float *y, int64_t ldy, void *stream) {
  if (n_experts <= 0 || n_experts > 2048 || hidden <= 0 || ffn <= 0 || (hidden % kQK) ||
      (ffn % kQK) || n_tokens < 0 || n_tokens > 64 || top_k < 1 || top_k > 16)
    return Q4K_ERR_SHAPE;
  if (hidden > (1 << 20) || ffn > (1 << 20)) return Q4K_ERR_SHAPE;
  if (expert_stride < (ffn * hidden / kQK) * kBlockBytes) return Q4K_ERR_SHAPE;
  if (n_tokens == 0) return Q4K_OK;
  if (ldx < hidden || ldy < hidden) return Q4K_ERR_SHAPE;
  if (!w_gate || !w_up || !w_down || !x || !ids || !wts || !y) return Q4K_ERR_NULL;
  if (moe_workspace_size(n_experts, n_tokens, top_k, hidden, ffn) > kMoeScratchBytes)
    return Q4K_ERR_WORKSPACE;
  if (!aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) || (expert_stride % 16) ||
      !aligned(x, 16) || (ldx % 8) || !aligned(y, 4) || !aligned(ids, 4) || !aligned(wts, 4))
    return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({w_gate, w_up, w_down, x, ids, wts, y});
  if (st != Q4K_OK) return st;
  return map_launch(launch_moe_scratch(w_gate, w_up, w_down, expert_stride, n_experts, hidden, ffn,
                                       x, n_tokens, ldx, ids, wts, top_k, y, ldy,
                                       static_cast<cudaStream_t>(stream)));
}

int q4k_kv_plan(const int32_t *lens, const int32_t *add, int32_t n, int32_t *table, int64_t ldt,
                int32_t max_pages, int32_t page_size, int32_t *pool, int32_t pool_size,
                const int32_t *pool_state, int32_t *lens_out, int64_t *cu, int32_t *slots,
                int32_t *pos, int64_t n_slots, int32_t *status, int32_t *pool_state_out,
                void *stream) {
  if (n < 0 || n > 65536 || max_pages <= 0 || page_size <= 0 || pool_size <= 0 || n_slots < 0 ||
      n_slots > INT32_MAX || ldt < max_pages || (int64_t)pool_size * page_size > INT32_MAX ||
      (int64_t)max_pages * page_size > (1 << 30))
    return Q4K_ERR_SHAPE;
  // Without requests nothing of theirs is touched, but the state, cu[0] and the
  // slot map are outputs all the same.
  if ((n > 0 && (!lens || !add || !table || !pool || !lens_out || !status)) || !pool_state || !cu ||
      !pool_state_out || (n_slots > 0 && (!slots || !pos)))
    return Q4K_ERR_NULL;
  if (!aligned(lens, 4) || !aligned(add, 4) || !aligned(table, 4) || !aligned(pool, 4) ||
      !aligned(pool_state, 4) || !aligned(lens_out, 4) || !aligned(cu, 8) || !aligned(slots, 4) ||
      !aligned(pos, 4) || !aligned(status, 4) || !aligned(pool_state_out, 4))
    return Q4K_ERR_ALIGN;
  int st = check_device();
  // (an empty call succeeds on a machine without a GPU, as all others do)
  if (st != Q4K_OK) return n == 0 && no_device() ? Q4K_OK : st;
  if (n == 0)
    st = check_device_memory({pool_state, cu, n_slots ? slots : nullptr, n_slots ? pos : nullptr, pool_state_out});
  else
    st = check_device_memory({lens, add, table, pool, pool_state, lens_out, cu, slots, pos, status,
                              pool_state_out});
  if (st != Q4K_OK) return st;
  return map_launch(launch_kv_plan(lens, add, n, table, ldt, max_pages, page_size, pool, pool_size,
                                   pool_state, lens_out, cu, slots, pos, n_slots, status,
                                   pool_state_out, static_cast<cudaStream_t>(stream)));
}

namespace {
// The cache arguments that q4k_kv_write and q4k_paged_attn share.  Strides are
// in elements, multiples of 16 bytes; no stride may make rows overlap.
int check_cache(int32_t kv_heads, int32_t dim, int cache_dtype, int64_t n_pages, int32_t page_size,
                int64_t page_stride, int64_t head_stride, int64_t token_stride) {
  if (dim != 64 && dim != 128 && dim != 256) return Q4K_ERR_SHAPE;
  if (cache_dtype != Q4K_DTYPE_BF16 && cache_dtype != Q4K_DTYPE_E4M3) return Q4K_ERR_SHAPE;
  if (kv_heads <= 0 || kv_heads > 1024 || n_pages <= 0 || page_size <= 0 ||
      n_pages > INT32_MAX / page_size)
    return Q4K_ERR_SHAPE;
  const int64_t kMax = (int64_t)1 << 40;
  if (page_stride < dim || head_stride < dim || token_stride < dim || page_stride > kMax ||
      head_stride > kMax || token_stride > kMax)
    return Q4K_ERR_SHAPE;
  // By size, whatever their order, each stride has to step over all of the next
  // smaller one (dimensions of 1 have no stride to speak of).
  struct Dim {
    int64_t stride, extent;
  } d[3] = {{token_stride, page_size}, {head_stride, kv_heads}, {page_stride, n_pages}};
  std::sort(d, d + 3, [](const Dim &x, const Dim &y) { return x.stride < y.stride; });
  const Dim *inner = nullptr;
  for (const Dim &x : d) {
    if (x.extent == 1) continue;
    if (inner && x.stride / inner->stride < inner->extent) return Q4K_ERR_SHAPE;
    inner = &x;
  }
  const int64_t unit = cache_dtype == Q4K_DTYPE_BF16 ? 8 : 16;
  if (page_stride % unit || head_stride % unit || token_stride % unit) return Q4K_ERR_ALIGN;
  return Q4K_OK;
}
}  // namespace

int q4k_kv_write(const void *k, const void *v, int in_dtype, int64_t ld_token, int64_t ld_head,
                 const int32_t *slots, int64_t tokens, int32_t kv_heads, int32_t dim, void *k_cache,
                 void *v_cache, int cache_dtype, int64_t n_pages, int32_t page_size,
                 int64_t page_stride, int64_t head_stride, int64_t token_stride, float *k_scale,
                 float *v_scale, void *stream) {
  if (in_dtype != Q4K_DTYPE_FP32 && in_dtype != Q4K_DTYPE_BF16) return Q4K_ERR_SHAPE;
  int st = check_cache(kv_heads, dim, cache_dtype, n_pages, page_size, page_stride, head_stride,
                       token_stride);
  if (st != Q4K_OK) return st;
  if (tokens < 0 || tokens > INT32_MAX / kv_heads || ld_head < dim || ld_token < 0)
    return Q4K_ERR_SHAPE;
  if (tokens == 0) return Q4K_OK;
  const bool e4m3 = cache_dtype == Q4K_DTYPE_E4M3;
  if (!k || !v || !slots || !k_cache || !v_cache || (e4m3 && (!k_scale || !v_scale)))
    return Q4K_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || ld_token % 8 || ld_head % 8)
    return Q4K_ERR_ALIGN;
  st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({k, v, slots, k_cache, v_cache, e4m3 ? k_scale : nullptr,
                            e4m3 ? v_scale : nullptr});
  if (st != Q4K_OK) return st;
  return map_launch(launch_kv_write(k, v, in_dtype, ld_token, ld_head, slots, tokens, kv_heads, dim,
                                    k_cache, v_cache, cache_dtype, n_pages, page_size, page_stride,
                                    head_stride, token_stride, k_scale, v_scale,
                                    static_cast<cudaStream_t>(stream)));
}

size_t q4k_paged_attn_workspace_size(int32_t n, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  if (n < 0 || q_heads <= 0 || kv_heads <= 0 || dim <= 0) return 0;
  return paged_attn_workspace_size(n, q_heads, kv_heads, dim);
}

int q4k_paged_attn(const void *q, int64_t ldq, int64_t ldq_head, int32_t n, int32_t q_heads,
                   int32_t kv_heads, int32_t dim, const void *k_cache, const void *v_cache,
                   int cache_dtype, int64_t n_pages, int32_t page_size, int64_t page_stride,
                   int64_t head_stride, int64_t token_stride, const float *k_scale,
                   const float *v_scale, const int32_t *table, int64_t ldt, int32_t max_pages,
                   const int32_t *lens, float softmax_scale, int32_t window, void *out, int64_t ldo,
                   float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_cache(kv_heads, dim, cache_dtype, n_pages, page_size, page_stride, head_stride,
                       token_stride);
  if (st != Q4K_OK) return st;
  if (n < 0 || n > 65536 || q_heads <= 0 || q_heads > 1024 || q_heads % kv_heads) return Q4K_ERR_SHAPE;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return Q4K_ERR_SHAPE;
  if (max_pages <= 0 || max_pages > (1 << 30) / page_size || ldt < max_pages || window < 0)
    return Q4K_ERR_SHAPE;
  if (!(softmax_scale - softmax_scale == 0.f)) return Q4K_ERR_SHAPE;  // NaN or infinite
  if (ldq_head < dim || ldq < 0 || ldo < (int64_t)q_heads * dim) return Q4K_ERR_SHAPE;
  if (n == 0) return Q4K_OK;
  const bool e4m3 = cache_dtype == Q4K_DTYPE_E4M3;
  if (!q || !k_cache || !v_cache || !table || !lens || !out || (e4m3 && (!k_scale || !v_scale)))
    return Q4K_ERR_NULL;
  if (!workspace || workspace_bytes < paged_attn_workspace_size(n, q_heads, kv_heads, dim))
    return Q4K_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) ||
      !aligned(v_scale, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 16) || ldq % 8 || ldq_head % 8 || ldo % 8)
    return Q4K_ERR_ALIGN;
  st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({q, k_cache, v_cache, table, lens, out, lse, workspace,
                            e4m3 ? k_scale : nullptr, e4m3 ? v_scale : nullptr});
  if (st != Q4K_OK) return st;
  AttnArgs a = {};
  a.q = q, a.cache[0] = k_cache, a.cache[1] = v_cache, a.scale[0] = k_scale, a.scale[1] = v_scale;
  a.table = table, a.lens = lens, a.out = out, a.lse = lse, a.workspace = workspace;
  a.ldq = ldq, a.ldq_head = ldq_head, a.ldo = ldo, a.ldt = ldt, a.n_pages = n_pages;
  a.page_stride = page_stride, a.head_stride = head_stride, a.token_stride = token_stride;
  a.n = n, a.q_heads = q_heads, a.kv_heads = kv_heads, a.dim = dim, a.page = page_size;
  a.max_pages = max_pages, a.window = window, a.softmax_scale = softmax_scale;
  a.cache_dtype = cache_dtype, a.err = device_error_word();
  return map_launch(launch_paged_attn(a, static_cast<cudaStream_t>(stream)));
}

int q4k_add_rmsnorm(const void *x, int x_dtype, int64_t ldx, const void *residual, int res_dtype,
                    int64_t ldr, const float *gamma, float eps, int64_t m, int64_t hidden, void *y,
                    int y_dtype, int64_t ldy, void *residual_out, int64_t ldro, float *scales,
                    int64_t lds, void *stream) {
  const bool e4m3 = y_dtype == Q4K_DTYPE_E4M3;
  if ((x_dtype != Q4K_DTYPE_FP32 && x_dtype != Q4K_DTYPE_BF16) ||
      (y_dtype != Q4K_DTYPE_BF16 && !e4m3) ||
      (residual && res_dtype != Q4K_DTYPE_FP32 && res_dtype != Q4K_DTYPE_BF16))
    return Q4K_ERR_SHAPE;
  if (m < 0 || m > INT32_MAX || hidden <= 0 || hidden > 32768 || hidden % 8) return Q4K_ERR_SHAPE;
  if (!(eps >= 0.f) || !(eps - eps == 0.f)) return Q4K_ERR_SHAPE;
  if (m == 0) return Q4K_OK;
  if (ldx < hidden || ldy < hidden || (residual && (ldr < hidden || ldro < hidden)) ||
      (e4m3 && lds < (hidden + 127) / 128))
    return Q4K_ERR_SHAPE;
  if (!x || !gamma || !y || (residual && !residual_out) || (e4m3 && !scales)) return Q4K_ERR_NULL;
  if (!aligned(x, 16) || !aligned(gamma, 16) || !aligned(y, 16) || ldx % 8 || ldy % 8 ||
      (residual && (!aligned(residual, 16) || !aligned(residual_out, 16) || ldr % 8 || ldro % 8)) ||
      (e4m3 && !aligned(scales, 4)))
    return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({x, residual, gamma, y, residual ? residual_out : nullptr,
                            e4m3 ? scales : nullptr});
  if (st != Q4K_OK) return st;
  return map_launch(launch_add_rmsnorm(x, x_dtype, ldx, residual, res_dtype, ldr, gamma, eps, m, hidden,
                                       y, y_dtype, ldy, residual_out, ldro, scales, lds,
                                       static_cast<cudaStream_t>(stream)));
}

int q4k_sample(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
               const float *u, const float *temperature, const int32_t *top_k, const float *top_p,
               const float *min_p, int32_t *token, float *logp, void *stream) {
  if (dtype != Q4K_DTYPE_FP32 && dtype != Q4K_DTYPE_BF16) return Q4K_ERR_SHAPE;
  if (rows < 0 || rows > (1 << 24) || vocab <= 0 || vocab > 262144 || ld < vocab) return Q4K_ERR_SHAPE;
  if (rows == 0) return Q4K_OK;
  if (!logits || !u || !token) return Q4K_ERR_NULL;
  if (!aligned(logits, dtype == Q4K_DTYPE_FP32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(token, 4) ||
      !aligned(logp, 4))
    return Q4K_ERR_ALIGN;
  int st = check_device();
  if (st != Q4K_OK) return st;
  st = check_device_memory({logits, u, temperature, top_k, top_p, min_p, token, logp});
  if (st != Q4K_OK) return st;
  return map_launch(launch_sample(logits, dtype, rows, vocab, ld, u, temperature, top_k, top_p, min_p,
                                  token, logp, static_cast<cudaStream_t>(stream)));
}

int q4k_selftest_wait_timeout(void *stream) {
  int st = check_device();
  if (st != Q4K_OK) return st;
  selftest_wait_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(device_error_word());
  return map_launch(cudaGetLastError());
}

int q4k_get_device_error(void *stream, uint32_t *bits) {
  if (!bits) return Q4K_ERR_NULL;
  *bits = 0;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return Q4K_ERR_CUDA;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof v) != cudaSuccess) return Q4K_ERR_CUDA;
  if (v && cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero) != cudaSuccess) return Q4K_ERR_CUDA;
  *bits = v;
  return v ? Q4K_ERR_DATA : Q4K_OK;
}

}  // extern "C"
