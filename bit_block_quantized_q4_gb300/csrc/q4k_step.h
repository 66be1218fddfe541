// q4k_step.h -- host-side declarations of the launchers around the projections
// (cache plan and write, paged attention, norm, sampling).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "q4k_internal.h"

namespace q4k {

// A kernel's limit of dynamic shared memory, raised once per device, whichever
// thread comes first; the others wait for it and see its outcome.
struct SmemLimit {
  std::once_flag once[kMaxDevices];
  cudaError_t status[kMaxDevices];
};
template <typename Kernel>
cudaError_t raise_smem_limit(SmemLimit &l, Kernel kernel, int bytes) {
  const int dev = device_facts()->device;
  std::call_once(l.once[dev], [&] {
    l.status[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
  return l.status[dev];
}

// Around the projections (q4k_kv.cu, q4k_norm.cu, q4k_attn.cu, q4k_sample.cu);
// arguments as the entry points of the same names.
cudaError_t launch_kv_plan(const int32_t *lens, const int32_t *add, int32_t n, int32_t *table,
                           int64_t ldt, int32_t width, int32_t page, int32_t *pool,
                           int32_t pool_size, const int32_t *state, int32_t *lens_out, int64_t *cu,
                           int32_t *slots, int32_t *pos, int64_t n_slots, int32_t *status,
                           int32_t *state_out, cudaStream_t stream);
cudaError_t launch_kv_write(const void *k, const void *v, int in_dtype, int64_t ld_token,
                            int64_t ld_head, const int32_t *slots, int64_t tokens, int32_t heads,
                            int32_t dim, void *k_cache, void *v_cache, int cache_dtype,
                            int64_t n_pages, int32_t page, int64_t page_stride, int64_t head_stride,
                            int64_t token_stride, float *k_scale, float *v_scale,
                            cudaStream_t stream);
cudaError_t launch_add_rmsnorm(const void *x, int x_dtype, int64_t ldx, const void *res,
                               int res_dtype, int64_t ldr, const float *gamma, float eps,
                               int64_t m, int64_t h, void *y, int y_dtype, int64_t ldy,
                               void *res_out, int64_t ldro, float *scales, int64_t lds,
                               cudaStream_t stream);
struct AttnArgs {
  const void *q;
  const void *cache[2];     // K, V: bf16 or e4m3 [page][head][token][dim], strides below
  const float *scale[2];    // e4m3: fp32 [page][head][token], contiguous
  const int32_t *table;
  const int32_t *lens;
  void *out;                // bf16 [request][q_head][dim], row stride ldo
  float *lse;               // fp32 [request][q_head], or nullptr
  void *workspace;
  int64_t ldq, ldq_head, ldo, ldt;
  int64_t n_pages, page_stride, head_stride, token_stride;
  int n, q_heads, kv_heads, dim, page, max_pages, window;
  float softmax_scale;
  int cache_dtype;
  unsigned *err;
};
size_t paged_attn_workspace_size(int32_t n, int32_t q_heads, int32_t kv_heads, int32_t dim);
cudaError_t launch_paged_attn(const AttnArgs &a, cudaStream_t stream);
// Chunks: q, out and lse of `tokens` tokens, request r's are cu[r] .. cu[r + 1] - 1.
size_t paged_attn_chunk_workspace_size(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t dim);
cudaError_t launch_paged_attn_chunk(const AttnArgs &a, int64_t tokens, const int64_t *cu,
                                    cudaStream_t stream);
// Norm of heads, rotation, and with caches the write of keys and values
// (q4k_rope.cu): [0] queries, [1] keys, [2] values.
struct RopeArgs {
  const void *in[3];
  int64_t ld_token[3], ld_head[3];
  int64_t tokens;
  int heads[2];             // queries; keys and values
  int dim, rot;
  const float *gamma[2];    // queries, keys; or nullptr
  float eps, amplitude;
  const int32_t *pos, *slots;
  const uint64_t *steps;    // [rot / 2] turns per position, in units of 2^-64
  void *out;                // queries, bf16 or fp32
  int64_t ldo_token, ldo_head;
  int out_dtype;
  void *cache[2];           // nullptr: queries alone
  float *scale[2];
  int cache_dtype;
  uint32_t n_slots;
  int page;
  int64_t page_stride, head_stride, token_stride;
  unsigned *err;
};
// The table of frequencies, on the host; false: one is not finite.
bool rope_steps(int rot, double base, double factor, int64_t original, double beta_fast,
                double beta_slow, const float *factors, uint64_t *steps, float *amplitude);
cudaError_t launch_rope(const RopeArgs &r, int dtype, bool interleaved, cudaStream_t stream);
cudaError_t launch_logprobs(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                            const int32_t *tokens, int top, float *logp, int32_t *rank,
                            float *entropy, int32_t *top_tokens, float *top_logp,
                            cudaStream_t stream);
cudaError_t launch_sample(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                          const float *u, const float *temperature, const int32_t *top_k,
                          const float *top_p, const float *min_p, int32_t *token, float *logp,
                          cudaStream_t stream);

}  // namespace q4k
