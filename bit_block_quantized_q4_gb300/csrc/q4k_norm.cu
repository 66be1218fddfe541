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
#include "q4k_step.h"

namespace q4k {
namespace {

constexpr int kMaxStages = 4;
constexpr int kRowsSmThreads = 1536;  // threads per SM of the many-rows kernel
constexpr int kRingBytes = 200 << 10;  // shared memory of an SM given to rings

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
  unsigned *err;
};

// y of one 8-value vector, to row pointers y and scales: `in` is false for lanes
// past the end of the row, which take part in the half-warp's block maximum with
// 0.
template <bool E4M3>
__device__ __forceinline__ void write_y(const float *gamma, uint8_t *y, float *scales, int vec, bool in, float rinv, float (&v)[8]) {
  float amax = 0.f;
  if (in) {
    float g[8];
    load8(gamma + vec * 8, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = v[j] * rinv * g[j];
      if (E4M3) amax = fmaxf(amax, fabsf(v[j]));
    }
  }
  if constexpr (E4M3) {
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float scale;
    const float inv = block_factor(fmaxf(amax, kAmaxFloor), threadIdx.x & 15, 0xffffffffu, scale);
    if (in) {
      *reinterpret_cast<uint2 *>(y + vec * 8) = to_e4m3x8(v, inv);
      if ((vec & 15) == 0) scales[vec >> 4] = scale;
    }
  } else if (in) {
    store8(reinterpret_cast<__nv_bfloat16 *>(y) + vec * 8, v);
  }
}
template <bool E4M3>
__device__ __forceinline__ uint8_t *row_of_y(const NormArgs &a, int64_t row) {
  return static_cast<uint8_t *>(a.y) + row * a.ldy * (E4M3 ? 1 : 2);
}

// Few rows: a block (tpr, rows) loads its rows straight into registers, tpr
// threads (whole warps) per row.  Vector i of thread t is vector t + i * tpr of
// the row, so the 16 vectors of a 128-value block lie in one half-warp.
template <int NV, typename TX, typename TR, bool E4M3>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float part[32];
  const int tpr = blockDim.x;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.m;
  const int nvec = a.h >> 3;
  float v[NV][8];
  float ss = 0.f;
  if (live) {
    const TX *x = static_cast<const TX *>(a.x) + row * a.ldx;
    const TR *r = static_cast<const TR *>(a.res) + row * a.ldr;
    Raw8<TX> xv[NV];
    Raw8<TR> rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = threadIdx.x + i * tpr;
      if (vec < nvec) {
        xv[i].load(x + vec * 8);
        if (a.res) rv[i].load(r + vec * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = threadIdx.x + i * tpr;
      if (vec >= nvec) continue;
      xv[i].to(v[i]);
      if (a.res) {
        float w[8];
        rv[i].to(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += w[j];
        store8(static_cast<TR *>(a.res_out) + row * a.ldro + vec * 8, v[i]);
      }
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
  uint8_t *y = row_of_y<E4M3>(a, row);
  float *scales = E4M3 ? a.scales + row * a.lds : nullptr;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = threadIdx.x + i * tpr;
    write_y<E4M3>(a.gamma, y, scales, vec, vec < nvec, rinv, v[i]);
  }
}

// Many rows: persistent blocks, each with a ring of rows in shared memory that
// bulk copies fill `stages` rows ahead (x, then the residual), so that the loads
// of the next rows never stop.  A thread takes up to KEEP vectors of a row, which
// it keeps in registers between the sum of squares and y; with KEEP = 0 it takes
// any number and reads them again.  One barrier per row: behind it every thread
// has its part of the sum, and every thread has left the row before, whose stage
// is then refilled.  (8191 x 5120 to e4m3: 47.3 us kept, 49.3 read again in the
// same run, 47.9 in others; 2000 x 17408: 31.6 us read again, 35.6 with 8 kept,
// whose registers leave room for one block per SM only.)
template <typename TX, typename TR, bool E4M3, int KEEP>
__global__ void __launch_bounds__(512) add_rmsnorm_rows_kernel(const NormArgs a, int stages) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float part[2][16];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
  const int nvec = a.h >> 3, loops = (nvec + threads - 1) / threads;
  const uint32_t xb = a.h * sizeof(TX), rb = a.res ? a.h * sizeof(TR) : 0;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  int64_t next = blockIdx.x;  // thread 0: the next row to fetch
  const auto fetch = [&](int slot) {
    if (next >= a.m) return;
    uint8_t *to = ring + slot * (xb + rb);
    mbar_arrive_expect_tx(&full[slot], xb + rb);
    bulk_load(to, static_cast<const TX *>(a.x) + next * a.ldx, xb, &full[slot]);
    if (rb) bulk_load(to + xb, static_cast<const TR *>(a.res) + next * a.ldr, rb, &full[slot]);
    next += gridDim.x;
  };
  if (tid == 0)
    for (int s = 0; s < stages; ++s) fetch(s);
  int slot = 0, prev = -1, flip = 0;
  uint32_t phase = 0;
  const float inv_h = 1.f / (float)a.h;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
    const bool ok = mbar_wait(&full[slot], phase, a.err);
    const TX *x = reinterpret_cast<const TX *>(ring + slot * (xb + rb));
    const TR *r = reinterpret_cast<const TR *>(ring + slot * (xb + rb) + xb);
    TR *res_out = rb ? static_cast<TR *>(a.res_out) + row * a.ldro : nullptr;
    float ss = 0.f;
    // h of a vector: x + residual, added to the sum and stored where `first`
    const auto load_h = [&](int vec, float (&v)[8], bool first) {
      load8(x + vec * 8, v);
      if (rb) {
        float w[8];
        load8(r + vec * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += w[j];
        if (first) store8(res_out + vec * 8, v);
      }
      if (first) {
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
      }
    };
    float v[KEEP ? KEEP : 1][8];
    if (ok) {
      if constexpr (KEEP > 0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
          if (tid + i * threads < nvec) load_h(tid + i * threads, v[i], true);
      } else {
        for (int vec = tid; vec < nvec; vec += threads) load_h(vec, v[0], true);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((tid & 31) == 0) part[flip][tid >> 5] = ss;
    if (__syncthreads_or(!ok)) {
      // a copy did not arrive in time: give the others the same time, then end
      if (tid == 0) drain_ring(full, stages, slot, phase, stages);
      return;
    }
    if (tid == 0 && prev >= 0) fetch(prev);
    ss = 0.f;
    for (int i = 0; i < warps; ++i) ss += part[flip][i];
    const float rinv = rsqrtf(ss * inv_h + a.eps);
    uint8_t *y = row_of_y<E4M3>(a, row);
    float *scales = E4M3 ? a.scales + row * a.lds : nullptr;
    if constexpr (KEEP > 0) {
#pragma unroll
      for (int i = 0; i < KEEP; ++i)
        write_y<E4M3>(a.gamma, y, scales, tid + i * threads, tid + i * threads < nvec, rinv, v[i]);
    } else {
      for (int i = 0; i < loops; ++i) {
        const int vec = tid + i * threads;
        if (vec < nvec) load_h(vec, v[0], false);
        write_y<E4M3>(a.gamma, y, scales, vec, vec < nvec, rinv, v[0]);
      }
    }
    prev = slot;
    flip ^= 1;
    if (++slot == stages) slot = 0, phase ^= 1u;
  }
}

template <int NV, typename TX, typename TR>
void launch_nv(const NormArgs &a, bool e4m3, dim3 grid, dim3 block, cudaStream_t s) {
  if (e4m3)
    add_rmsnorm_kernel<NV, TX, TR, true><<<grid, block, 0, s>>>(a);
  else
    add_rmsnorm_kernel<NV, TX, TR, false><<<grid, block, 0, s>>>(a);
}

template <typename TX, typename TR, bool E4M3, int KEEP>
cudaError_t launch_rows_kept(const NormArgs &a, int stage, int threads, cudaStream_t s) {
  const DeviceFacts *f = device_facts();
  static SmemLimit limit;
  const cudaError_t e = raise_smem_limit(limit, add_rmsnorm_rows_kernel<TX, TR, E4M3, KEEP>, kRingBytes);
  if (e != cudaSuccess) return e;
  // blocks per SM: as many as keep two rows each in flight, up to 1536 threads
  int blocks = kRowsSmThreads / threads;
  if (blocks > kRingBytes / (2 * stage)) blocks = kRingBytes / (2 * stage);
  if (blocks > 16) blocks = 16;
  if (blocks < 1) blocks = 1;
  int stages = kRingBytes / blocks / stage;
  if (stages > kMaxStages) stages = kMaxStages;
  int64_t grid = (int64_t)f->sm_count * blocks;
  if (grid > a.m) grid = a.m;
  add_rmsnorm_rows_kernel<TX, TR, E4M3, KEEP><<<(unsigned)grid, threads, stages * stage, s>>>(a, stages);
  return cudaGetLastError();
}
template <typename TX, typename TR, bool E4M3>
cudaError_t launch_rows(const NormArgs &a, int stage, cudaStream_t s) {
  // Threads per row, before vectors were kept: 8192 rows of 5120 bf16 to e4m3 took
  // 50.8 us with 320, 53.7 with 256, 56.6 with 160; 2000 rows of 17408 32.0 us with
  // 512, 34.4 with 320, 44.7 with 160.
  const int nvec = a.h / 8, most = nvec > 2048 ? 512 : 320, loops = (nvec + most - 1) / most;
  const int threads = ((nvec + loops - 1) / loops + 31) / 32 * 32;
  if (loops <= 2) return launch_rows_kept<TX, TR, E4M3, 2>(a, stage, threads, s);
  if (loops <= 4) return launch_rows_kept<TX, TR, E4M3, 4>(a, stage, threads, s);
  return launch_rows_kept<TX, TR, E4M3, 0>(a, stage, threads, s);
}

template <typename TX, typename TR>
cudaError_t launch_types(const NormArgs &a, bool e4m3, cudaStream_t s) {
  const int nvec = a.h / 8, sms = device_facts()->sm_count;
  const int stage = a.h * (int)(sizeof(TX) + (a.res ? sizeof(TR) : 0));
  // Rows of up to 4096 values fit the registers of a block often enough to keep
  // the memory busy (30000 x 1024: 37.4 us against 45.1 through the ring; 8192 x
  // 4096 from fp32: 47.0 against 51.6); longer ones do not (8191 x 5120 to e4m3:
  // 56.8 against 47.3; 2000 x 17408: 42.7 against 31.6).  With fewer than 4 rows
  // per SM there is nothing to fetch ahead.
  if (nvec > 512 && a.m > 4 * sms && 2 * stage <= kRingBytes)
    return e4m3 ? launch_rows<TX, TR, true>(a, stage, s) : launch_rows<TX, TR, false>(a, stage, s);
  const int nv = nvec > 256 && nvec <= 512 ? 2 : (nvec + 1023) / 1024;
  const int tpr = ((nvec + nv - 1) / nv + 31) / 32 * 32;
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  const dim3 block(tpr, rows), grid((unsigned)((a.m + rows - 1) / rows));
  switch (nv) {
    case 1: launch_nv<1, TX, TR>(a, e4m3, grid, block, s); break;
    case 2: launch_nv<2, TX, TR>(a, e4m3, grid, block, s); break;
    case 3: launch_nv<3, TX, TR>(a, e4m3, grid, block, s); break;
    default: launch_nv<4, TX, TR>(a, e4m3, grid, block, s); break;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void *x, int x_dtype, int64_t ldx, const void *res,
                               int res_dtype, int64_t ldr, const float *gamma, float eps,
                               int64_t m, int64_t h, void *y, int y_dtype, int64_t ldy,
                               void *res_out, int64_t ldro, float *scales, int64_t lds,
                               cudaStream_t stream) {
  const NormArgs a = {x, res, gamma, y, res_out, scales, m, ldx, ldr, ldy, ldro, lds, (int)h, eps,
                      device_error_word()};
  const bool e4m3 = y_dtype == Q4K_DTYPE_E4M3;
  const bool xb = x_dtype == Q4K_DTYPE_BF16, rb = !res || res_dtype == Q4K_DTYPE_BF16;
  if (xb && rb) return launch_types<__nv_bfloat16, __nv_bfloat16>(a, e4m3, stream);
  if (xb) return launch_types<__nv_bfloat16, float>(a, e4m3, stream);
  if (rb) return launch_types<float, __nv_bfloat16>(a, e4m3, stream);
  return launch_types<float, float>(a, e4m3, stream);
}

}  // namespace q4k
