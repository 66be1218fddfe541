// q4k_norm.cu -- residual addition and root-mean-square norm (q4k_add_rmsnorm).
//
// "spec: specialized model runtimes", section "Architecture": norms are an op
// of kernel tier T0.
//
//   h = x + residual (fp32);  residual_out = h rounded once;
//   y = h * rsqrt(mean(h^2) + eps) * gamma, rounded once to bf16, or to e4m3
//   with one fp32 scale per 128 values: s = max(max|y|, 2^-100) / 448,
//   q = e4m3(y * (448 / max)).
// Every sum is fp32, in a fixed order.  The statistics and y use the unrounded
// h, so a bf16 residual stream costs its own rounding only.
//
// What bounds it: bytes.  Each row is read once and held in registers (NV
// vectors of 8 values per thread) between the sum of squares and the output.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/q4k.h"
#include "q4k_device.cuh"
#include "q4k_internal.h"
#include "q4k_step.cuh"

namespace q4k {
namespace {

constexpr int kMinBlocks = 1;
constexpr int kThreadsPerRow = 640;

struct NormArgs {
  const void *x;
  const void *res;
  const float *gamma;
  void *y;
  void *res_out;
  float *scales;
  int64_t m, ldx, ldr, ldy, ldro, lds;
  int h;
  float eps;
};

// Block (tpr, rows): tpr threads (whole warps) per row.  Vector i of thread t
// is vector t + i * tpr of the row, so the 16 vectors of a 128-value block lie
// in one half-warp (tpr is a multiple of 32).
template <int NV, typename TX, typename TR, bool E4M3>
__global__ void __launch_bounds__(1024, NV <= 2 ? kMinBlocks : 1) add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float part[32];
  const int tpr = blockDim.x;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.m;
  const int nvec = a.h >> 3;
  float v[NV][8];
  float ss = 0.f;
  if (live) {
    const TX *x = static_cast<const TX *>(a.x) + row * a.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = threadIdx.x + i * tpr;
      if (vec < nvec) load8(x + vec * 8, v[i]);
    }
    if (a.res) {
      const TR *r = static_cast<const TR *>(a.res) + row * a.ldr;
      TR *ro = static_cast<TR *>(a.res_out) + row * a.ldro;
      float w[NV][8];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int vec = threadIdx.x + i * tpr;
        if (vec < nvec) load8(r + vec * 8, w[i]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int vec = threadIdx.x + i * tpr;
        if (vec < nvec) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += w[i][j];
          store8(ro + vec * 8, v[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (threadIdx.x + i * tpr < nvec) {
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
      }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (tpr > 32) {
    const int warps = tpr >> 5, w0 = threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) part[w0 + (threadIdx.x >> 5)] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < warps; ++i) ss += part[w0 + i];
  }
  if (!live) return;
  const float rinv = rsqrtf(ss / (float)a.h + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = threadIdx.x + i * tpr;
    const bool in = vec < nvec;
    float amax = 0.f;
    if (in) {
      float g[8];
      load8(a.gamma + vec * 8, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = v[i][j] * rinv * g[j];
        if (E4M3) amax = fmaxf(amax, fabsf(v[i][j]));
      }
    }
    if (!E4M3) {
      if (in) store8(static_cast<__nv_bfloat16 *>(a.y) + row * a.ldy + vec * 8, v[i]);
    } else {
      // the half-warp that holds a block takes part as a whole: lanes past the
      // end of the row bring 0
#pragma unroll
      for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      amax = fmaxf(amax, kAmaxFloor);
      if (in) {
        const float inv = 448.f / amax;
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.y) + row * a.ldy + vec * 8) =
            to_e4m3x8(v[i], inv);
        if ((vec & 15) == 0) a.scales[row * a.lds + (vec >> 4)] = amax / 448.f;
      }
    }
  }
}

template <int NV, typename TX, typename TR>
void launch_nv(const NormArgs &a, bool e4m3, dim3 grid, dim3 block, cudaStream_t s) {
  if (e4m3)
    add_rmsnorm_kernel<NV, TX, TR, true><<<grid, block, 0, s>>>(a);
  else
    add_rmsnorm_kernel<NV, TX, TR, false><<<grid, block, 0, s>>>(a);
}

template <typename TX, typename TR>
void launch_types(const NormArgs &a, bool e4m3, cudaStream_t s) {
  const int nvec = a.h / 8;
  int nv = (nvec + kThreadsPerRow - 1) / kThreadsPerRow;
  if (nv > 4) nv = 4;
  const int tpr = ((nvec + nv - 1) / nv + 31) / 32 * 32;
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  const dim3 block(tpr, rows), grid((unsigned)((a.m + rows - 1) / rows));
  switch (nv) {
    case 1: launch_nv<1, TX, TR>(a, e4m3, grid, block, s); break;
    case 2: launch_nv<2, TX, TR>(a, e4m3, grid, block, s); break;
    case 3: launch_nv<3, TX, TR>(a, e4m3, grid, block, s); break;
    default: launch_nv<4, TX, TR>(a, e4m3, grid, block, s); break;
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void *x, int x_dtype, int64_t ldx, const void *res,
                               int res_dtype, int64_t ldr, const float *gamma, float eps,
                               int64_t m, int64_t h, void *y, int y_dtype, int64_t ldy,
                               void *res_out, int64_t ldro, float *scales, int64_t lds,
                               cudaStream_t stream) {
  const NormArgs a = {x, res, gamma, y, res_out, scales, m, ldx, ldr, ldy, ldro, lds, (int)h, eps};
  const bool e4m3 = y_dtype == Q4K_DTYPE_E4M3;
  const bool xb = x_dtype == Q4K_DTYPE_BF16, rb = !res || res_dtype == Q4K_DTYPE_BF16;
  if (xb && rb) launch_types<__nv_bfloat16, __nv_bfloat16>(a, e4m3, stream);
  else if (xb) launch_types<__nv_bfloat16, float>(a, e4m3, stream);
  else if (rb) launch_types<float, __nv_bfloat16>(a, e4m3, stream);
  else launch_types<float, float>(a, e4m3, stream);
  return cudaGetLastError();
}

}  // namespace q4k
