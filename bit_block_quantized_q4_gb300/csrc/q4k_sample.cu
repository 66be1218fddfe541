// q4k_sample.cu -- the choice of the next token from given random numbers
// (q4k_sample): temperature, top-k, top-p, min-p and the draw.
//
// "spec: specialized model runtimes", section "Architecture": the sampler is
// part of tier T1.
//
// Each token's weight e_i = exp((x_i - max) / temperature) is an integer,
// rint(2^44 e_i), so that sums are exact and the same in any order; a row of
// 2^18 tokens sums below 2^62.
//
// Every filter keeps a prefix of the tokens in the order (logit descending,
// index ascending).  With the composite key c_i = (monotone integer image of
// x_i) << 32 | ~i that order is the descending one of distinct integers, and a
// filter is a smallest key kept; the kept set is c_i >= the largest of them.
//
// One block per row; each threshold is found by bisecting the 64-bit keys with
// one pass over the row per bit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/q4k.h"
#include "q4k_device.cuh"
#include "q4k_internal.h"

namespace q4k {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = 1024;
constexpr double kOne = 17592186044416.0;  // 2^44

struct SampleArgs {
  const void *logits;
  int64_t ld;
  int vocab;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *token;
  float *logp;
};

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and +0 are one value
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <typename T>
__device__ __forceinline__ float load_logit(const T *p, int i) {
  float x = (float)p[i];
  return x == x ? x : -INFINITY;
}

template <typename F>
__device__ u64 block_sum(u64 *part, F f, int n) {
  u64 s = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += f(i);
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0;
  for (int w = 0; w < kThreads / 32; ++w) s += part[w];
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  __shared__ u64 part[32];
  __shared__ u64 best;
  __shared__ int chosen;
  const int row = blockIdx.x, n = a.vocab;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  if (threadIdx.x == 0) best = 0, chosen = -1;
  __syncthreads();
  u64 mx = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const u64 c = (u64)key_of(load_logit(x, i)) << 32 | (uint32_t)~i;
    mx = max(mx, c);
  }
  atomicMax(&best, mx);
  __syncthreads();
  const int first = ~(uint32_t)best;
  const float high = load_logit(x, first);
  const float t = a.temperature ? a.temperature[row] : 1.f;
  if (high == -INFINITY || !(t > 0.f)) {
    if (threadIdx.x == 0) {
      a.token[row] = high == -INFINITY ? -1 : first;
      if (a.logp) a.logp[row] = high == -INFINITY ? -INFINITY : 0.f;
    }
    return;
  }
  const auto comp = [&](int i) { return (u64)key_of(load_logit(x, i)) << 32 | (uint32_t)~i; };
  const auto weight = [&](int i) -> u64 {
    const float v = load_logit(x, i);
    if (v == high) return (u64)kOne;
    if (v == -INFINITY) return 0;
    return (u64)rint(kOne * exp(((double)v - (double)high) / (double)t));
  };
  u64 cut = 0;
  const int k = a.top_k ? a.top_k[row] : 0;
  if (k > 0 && k < n) {  // the largest cut with at least k keys at or above it
    for (int bit = 63; bit >= 0; --bit) {
      const u64 c = cut | 1ull << bit;
      if (block_sum(part, [&](int i) -> u64 { return comp(i) >= c; }, n) >= (u64)k) cut = c;
    }
  }
  const float p = a.top_p ? a.top_p[row] : 1.f;
  if (p < 1.f) {
    const u64 total = block_sum(part, [&](int i) -> u64 { return comp(i) >= cut ? weight(i) : 0; }, n);
    const double want = (double)fmaxf(p, 0.f) * (double)total;
    // the largest cut whose keys at or above it hold at least `want`: the key
    // equal to it is the last one whose predecessors hold less
    u64 c2 = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const u64 c = c2 | 1ull << bit;
      if (c > best) continue;
      if ((double)block_sum(part, [&](int i) -> u64 { return comp(i) >= c ? weight(i) : 0; }, n) >= want) c2 = c;
    }
    cut = max(cut, c2);
  }
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  if (mp > 0.f) {
    const double thr = (double)high + (double)t * log((double)fminf(mp, 1.f));
    cut = max(cut, (u64)key_of(high == INFINITY ? high : __double2float_ru(thr)) << 32);
  }
  const u64 total = block_sum(part, [&](int i) -> u64 { return comp(i) >= cut ? weight(i) : 0; }, n);
  const float u = fminf(fmaxf(a.u[row], 0.f), 1.f);
  u64 target = (u64)((double)u * (double)total);  // first index with cumulative > u * total
  if (target >= total) target = total - 1;
  // contiguous runs of indexes, one per thread
  const int run = (n + kThreads - 1) / kThreads, i0 = min(n, (int)threadIdx.x * run), i1 = min(n, i0 + run);
  u64 own = 0;
  for (int i = i0; i < i1; ++i) own += comp(i) >= cut ? weight(i) : 0;
  u64 incl = own;
  for (int o = 1; o < 32; o <<= 1) {
    const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
    if ((threadIdx.x & 31) >= o) incl += up;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 31) part[threadIdx.x >> 5] = incl;
  __syncthreads();
  for (int w = 0; w < (threadIdx.x >> 5); ++w) incl += part[w];
  if (incl > target && incl - own <= target) {
    u64 c = incl - own;
    for (int i = i0; i < i1; ++i) {
      const u64 w = comp(i) >= cut ? weight(i) : 0;
      c += w;
      if (c > target) {
        a.token[row] = i;
        if (a.logp) a.logp[row] = (float)log((double)w / (double)total);
        break;
      }
    }
  }
}

}  // namespace

cudaError_t launch_sample(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                          const float *u, const float *temperature, const int32_t *top_k,
                          const float *top_p, const float *min_p, int32_t *token, float *logp,
                          cudaStream_t stream) {
  const SampleArgs a = {logits, ld, (int)vocab, u, temperature, top_p, min_p, top_k, token, logp};
  if (dtype == Q4K_DTYPE_BF16) sample_kernel<__nv_bfloat16><<<(unsigned)rows, kThreads, 0, stream>>>(a);
  else sample_kernel<float><<<(unsigned)rows, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace q4k
