// q4k_attn.cu -- attention of one new token per request over the paged cache
// (q4k_paged_attn).
//
// "spec: specialized model runtimes", section "Architecture": attention is an
// op of kernel tier T0.
//
// One pass over the keys with the running maximum m and sum l of a softmax:
//   z_j = scale q.k_j,  m' = max(m, z_j),  l' = l e^(m-m') + e^(z_j-m'),
//   o' = o e^(m-m') + e^(z_j-m') v_j.
// One block per (request, query head); its four warps take tokens in turn and
// are joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/q4k.h"
#include "q4k_device.cuh"
#include "q4k_internal.h"
#include "q4k_step.cuh"

namespace q4k {
namespace {

template <int D, bool E4M3>
__global__ void __launch_bounds__(128) paged_attn_kernel(const AttnArgs a) {
  constexpr int V = D / 32;  // values per lane
  const int r = blockIdx.x, i = blockIdx.y, h = i / (a.q_heads / a.kv_heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float sm[4], sl[4], so[4][D];
  float q[V], o[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    q[c] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[r * a.ldq + i * a.ldq_head + lane + 32 * c]);
    o[c] = 0.f;
  }
  int64_t len = max(a.lens[r], 0);
  if (len > (int64_t)a.max_pages * a.page) {
    len = (int64_t)a.max_pages * a.page;
    set_device_error(a.err, kDevErrBadPage);
  }
  const int64_t start = a.window ? max(len - a.window, (int64_t)0) : 0;
  for (int64_t j = start + warp; j < len; j += 4) {
    const int64_t page = a.table[r * a.ldt + j / a.page], off = j % a.page;
    if (page < 0 || page >= a.n_pages) {
      set_device_error(a.err, kDevErrBadPage);
      continue;
    }
    const int64_t at = page * a.page_stride + h * a.head_stride + off * a.token_stride + lane;
    const int64_t sat = (page * a.kv_heads + h) * a.page + off;
    float z = 0.f, v[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if (E4M3) {
        z += q[c] * (float)static_cast<const __nv_fp8_e4m3 *>(a.cache[0])[at + 32 * c];
        v[c] = (float)static_cast<const __nv_fp8_e4m3 *>(a.cache[1])[at + 32 * c];
      } else {
        z += q[c] * __bfloat162float(static_cast<const __nv_bfloat16 *>(a.cache[0])[at + 32 * c]);
        v[c] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.cache[1])[at + 32 * c]);
      }
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    z *= a.softmax_scale;
    float vs = 1.f;
    if (E4M3) z *= a.scale[0][sat], vs = a.scale[1][sat];
    const float mn = fmaxf(m, z), f = m == mn ? 1.f : expf(m - mn), p = expf(z - mn);
    l = l * f + p;
    m = mn;
#pragma unroll
    for (int c = 0; c < V; ++c) o[c] = o[c] * f + p * vs * v[c];
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int c = 0; c < V; ++c) so[warp][lane + 32 * c] = o[c];
  __syncthreads();
  float mx = sm[0], lt = 0.f, f[4];
  for (int w = 1; w < 4; ++w) mx = fmaxf(mx, sm[w]);
  for (int w = 0; w < 4; ++w) f[w] = sm[w] == -INFINITY ? 0.f : expf(sm[w] - mx), lt += f[w] * sl[w];
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + r * a.ldo + (int64_t)i * D;
  for (int d = threadIdx.x; d < D; d += 128) {
    float t = 0.f;
    for (int w = 0; w < 4; ++w) t += f[w] * so[w][d];
    out[d] = __float2bfloat16(lt > 0.f ? t / lt : mx == -INFINITY ? 0.f : t / lt);
  }
  if (a.lse && threadIdx.x == 0) a.lse[(int64_t)r * a.q_heads + i] = mx == -INFINITY ? -INFINITY : mx + logf(lt);
}

}  // namespace

size_t paged_attn_workspace_size(int32_t, int32_t, int32_t, int32_t) { return 16; }

cudaError_t launch_paged_attn(const AttnArgs &a, cudaStream_t s) {
  const dim3 grid(a.n, a.q_heads);
  const bool e = a.cache_dtype == Q4K_DTYPE_E4M3;
  if (a.dim == 64) e ? paged_attn_kernel<64, true><<<grid, 128, 0, s>>>(a) : paged_attn_kernel<64, false><<<grid, 128, 0, s>>>(a);
  else if (a.dim == 128) e ? paged_attn_kernel<128, true><<<grid, 128, 0, s>>>(a) : paged_attn_kernel<128, false><<<grid, 128, 0, s>>>(a);
  else e ? paged_attn_kernel<256, true><<<grid, 128, 0, s>>>(a) : paged_attn_kernel<256, false><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace q4k
