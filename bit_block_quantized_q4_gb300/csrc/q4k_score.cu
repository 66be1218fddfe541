// q4k_score.cu -- log-probability and rank of given tokens, the distribution's
// entropy and its most likely tokens (q4k_logprobs).
//
// "spec: specialized model runtimes", section "Architecture": what is read off
// the logits belongs to tier T1, with the sampler.
//
// Mathematics.  With M a reference near the row's maximum, in one pass
//   l = sum e^(x_i - M),   w = sum e^(x_i - M) (x_i - M),
//   logp(t) = x_t - M - ln l,   entropy = ln l - w / l,
// two parts with references M, M' are joined by l' e^(M' - M) and
// (w' + (M' - M) l') e^(M' - M).  Differences below -128 count as -128, whose
// e is 0 in fp32: so a logit of -infinity, or the lowest number of its type,
// adds 0 and not 0 times infinity.
//
// Order.  Tokens are ordered by logit, highest first, equal ones by index: the
// descending order of the distinct integers key_i = (monotone image of x_i) <<
// 32 | ~i.
//
// Alternatives.  Every thread keeps the first of its highest logits.  The n-th
// highest of the 32 maxima of half warps is a bound that at least n tokens
// reach; a few dozen do in all, found again among the tokens of the threads whose
// own maximum reaches it.  Should more reach it than the list holds, they are
// taken one after the other instead.
//
// What bounds it: the logits are read once.  A row is one CTA's, or while rows
// are few a cluster's, whose CTAs take equal slices and send sums and lists to
// the first one.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/q4k.h"
#include "q4k_device.cuh"
#include "q4k_internal.h"
#include "q4k_step.cuh"
#include "q4k_step.h"

namespace q4k {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = 512, kWarps = kThreads / 32, kGroups = 2 * kWarps;
constexpr int kTop = 32, kList = 1024, kMaxCluster = 8;
constexpr float kLow = -128.f;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
  const void *logits;
  int64_t ld;
  int vocab, slice, top;  // slice: tokens per CTA, a multiple of 64
  const int32_t *tokens;
  float *logp, *entropy, *top_logp;
  int32_t *rank, *top_tokens;
};

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and +0 are one value
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// NaN counts as -infinity; so does what is not listed: 0.
__device__ __forceinline__ u64 key_at(float x, uint32_t i) {
  return x > -INFINITY ? (u64)key_of(x) << 32 | (uint32_t)~i : 0ull;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ float one(const T *p) {
  return (float)*p;
}

// What a thread, a warp, a CTA knows of the tokens that it has seen.
struct Sums {
  float m, l, w;
};
__device__ __forceinline__ void join(Sums &a, const Sums &b) {
  const float m = fmaxf(a.m, b.m);
  // without a token l is 0, and its reference says nothing
  const float da = a.l == 0.f ? 0.f : fmaxf(a.m - m, kLow), db = b.l == 0.f ? 0.f : fmaxf(b.m - m, kLow);
  const float fa = ex2(da * kLog2e), fb = ex2(db * kLog2e);
  a.w = fa * fmaf(da, a.l, a.w) + fb * fmaf(db, b.l, b.w);
  a.l = fa * a.l + fb * b.l;
  a.m = m;
}

struct Shared {
  Sums sums[kWarps];
  int count[kWarps], infinite[kWarps];
  u64 group[kGroups];       // highest key of each half warp
  u64 list[kList];
  u64 chosen[kTop];
  u64 bound;
  int listed;
  // of all CTAs of the cluster, in the first one
  Sums all_sums[kMaxCluster];
  int all_count[kMaxCluster], all_infinite[kMaxCluster];
  u64 all_keys[kMaxCluster * kTop];
};

__device__ __forceinline__ u64 shfl64(u64 v, int from) {
  return (u64)__shfl_sync(0xffffffffu, (unsigned)(v >> 32), from) << 32 | __shfl_sync(0xffffffffu, (unsigned)v, from);
}
__device__ __forceinline__ u64 max64(u64 a, u64 b) { return a > b ? a : b; }

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const Args a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = (int)gridDim.x, rank = (int)blockIdx.x;
  const int64_t row = blockIdx.y;
  const T *x = static_cast<const T *>(a.logits) + row * a.ld;
  const int lo = min(rank * a.slice, a.vocab), hi = min(lo + a.slice, a.vocab);
  const int token = a.tokens[row];
  const bool real = token >= 0 && token < a.vocab;
  float xt = real ? one(x + token) : INFINITY;
  xt = xt > -INFINITY ? xt : -INFINITY;  // NaN
  if (tid == 0) sh.listed = 0;
  // every CTA of the cluster has started before one writes into the first one's memory
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");

  // Vectors of 8 from the first 16-byte boundary on; the tokens before and after
  // it one by one.  Thread i takes vector i, i + kThreads, ...: its tokens come in
  // rising order.
  constexpr int kV = 8;
  const int head = min(hi - lo, (int)((16 - ((uintptr_t)(x + lo) & 15)) & 15) / (int)sizeof(T));
  const int v0 = lo + head, vectors = (hi - v0) / kV, tail = v0 + vectors * kV;
  Sums s = {-3.4028235e38f, 0.f, 0.f};
  float best = -INFINITY;  // highest logit, and where it was first seen (its vector's first token)
  int best_at = -1, count = 0, infinite = 0;

  const auto ahead = [&](float v, int i) {  // NaN counts as -infinity
    const float c = v > -INFINITY ? v : -INFINITY;
    return c > xt || (c == xt && i < token);
  };
  const auto single = [&](int i) {
    const float v = one(x + i);
    if (v > best) best = v, best_at = i;
    count += ahead(v, i);
    if (v == INFINITY) ++infinite;
    const Sums t = {v > -INFINITY ? v : s.m, v > -INFINITY ? 1.f : 0.f, 0.f};
    join(s, t);
  };
  if (tid < head) single(lo + tid);
  const auto eight = [&](const float (&v)[8], int i) {
    float top = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
    if (top > best) best = top, best_at = i;
    if (!(top < xt)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) count += ahead(v[j], i + j);
    }
    if (top > s.m + 8.f) {
      if (s.l != 0.f) {
        const float d = fmaxf(s.m - top, kLow), f = ex2(d * kLog2e);
        s.w = f * fmaf(d, s.l, s.w);
        s.l *= f;
      }
      s.m = top;
    }
    if (s.m == INFINITY) {
#pragma unroll
      for (int j = 0; j < 8; ++j) infinite += v[j] == INFINITY;
      return;
    }
    const float2 m2 = make_float2(-s.m, -s.m);
    float2 l2 = make_float2(0.f, 0.f), w2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float2 d = __fadd2_rn(make_float2(v[j], v[j + 1]), m2);
      d = make_float2(fmaxf(d.x, kLow), fmaxf(d.y, kLow));  // (NaN too)
      const float2 z = __fmul2_rn(d, make_float2(kLog2e, kLog2e)), e = make_float2(ex2(z.x), ex2(z.y));
      l2 = __fadd2_rn(l2, e);
      w2 = __ffma2_rn(e, d, w2);
    }
    s.l += l2.x + l2.y;
    s.w += w2.x + w2.y;
  };
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // vectors on their way
  for (int k0 = tid; k0 < vectors; k0 += U * kThreads) {
    Raw8<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u * kThreads < vectors) raw[u].load(x + v0 + (k0 + u * kThreads) * kV);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u * kThreads < vectors) {
        float v[8];
        raw[u].to(v);
        eight(v, v0 + (k0 + u * kThreads) * kV);
      }
  }
  if (tid < hi - tail) single(tail + tid);

  // the key of this thread's best
  u64 key = 0;
  if (a.top && best > -INFINITY) {
    int at = best_at;
    while (one(x + at) != best) ++at;  // within its vector
    key = key_at(best, at);
  }

  // ---- sums of the CTA
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Sums t;
    t.m = __shfl_xor_sync(0xffffffffu, s.m, o), t.l = __shfl_xor_sync(0xffffffffu, s.l, o), t.w = __shfl_xor_sync(0xffffffffu, s.w, o);
    // the lower lane's part first, on both sides: the same sums in every lane
    if (lane & o) {
      join(t, s);
      s = t;
    } else {
      join(s, t);
    }
  }
  count = __reduce_add_sync(0xffffffffu, count);
  infinite = __reduce_add_sync(0xffffffffu, infinite);
  if (lane == 0) sh.sums[warp] = s, sh.count[warp] = count, sh.infinite[warp] = infinite;
  if (a.top) {
    u64 g = key;
#pragma unroll
    for (int o = 8; o; o >>= 1) g = max64(g, shfl64(g, lane ^ o));
    if ((lane & 15) == 0) sh.group[2 * warp + lane / 16] = g;
  }
  __syncthreads();

  // ---- this CTA's `top` highest keys, in order, in chosen[]
  const int n = a.top;
  if (n) {
    if (warp == 0) {
      const u64 g = sh.group[lane];
      int above = 0;
      for (int i = 0; i < kGroups; ++i) above += shfl64(g, i) > g;
      // equal keys are 0 only: with fewer than n groups that have a token, all count
      const unsigned at = __ballot_sync(0xffffffffu, above == n - 1 && g);
      const u64 b = at ? shfl64(g, __ffs(at) - 1) : 1ull;
      if (lane == 0) sh.bound = b;
    }
    __syncthreads();
    const u64 bound = sh.bound;
    const auto offer = [&](u64 k) {
      if (k >= bound) {
        const int i = atomicAdd(&sh.listed, 1);
        if (i < kList) sh.list[i] = k;
      }
    };
    // the threads whose best reaches the bound: a warp goes through the tokens of one at a time
    unsigned todo = __ballot_sync(0xffffffffu, key >= bound);
    while (todo) {
      const int src = __ffs(todo) - 1, th = warp * 32 + src;
      todo &= todo - 1;
      for (int k = th + lane * kThreads; k < vectors; k += 32 * kThreads) {
        float v[8];
        const int i = v0 + k * kV;
        load8(x + i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) offer(key_at(v[j], i + j));
      }
      if (lane == 0 && th < head) offer(key_at(one(x + lo + th), lo + th));
      if (lane == 1 && th < hi - tail) offer(key_at(one(x + tail + th), tail + th));
    }
    __syncthreads();
    const int listed = sh.listed;
    if (listed <= kList) {
      for (int i = tid; i < listed; i += kThreads) {
        const u64 k = sh.list[i];
        int above = 0;
        for (int j = 0; j < listed; ++j) above += sh.list[j] > k;
        if (above < n) sh.chosen[above] = k;
      }
      if (tid >= listed && tid < n) sh.chosen[tid] = 0;
    } else {
      // more tokens reach the bound than the list holds: one after the other
      u64 last = ~0ull;
      for (int c = 0; c < n; ++c) {
        u64 g = 0;
        for (int k = tid; k < vectors; k += kThreads) {
          float v[8];
          load8(x + v0 + k * kV, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const u64 q = key_at(v[j], v0 + k * kV + j);
            if (q < last) g = max64(g, q);
          }
        }
        for (int i = tid; i < head + hi - tail; i += kThreads) {
          const int at = i < head ? lo + i : tail + i - head;
          const u64 q = key_at(one(x + at), at);
          if (q < last) g = max64(g, q);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) g = max64(g, shfl64(g, lane ^ o));
        if (lane == 0) sh.group[warp] = g;
        __syncthreads();
        g = 0;
        for (int i = 0; i < kWarps; ++i) g = max64(g, sh.group[i]);
        if (tid == 0) sh.chosen[c] = g;
        last = g;
        __syncthreads();
      }
    }
    __syncthreads();
  }

  // ---- to the cluster's first CTA
  if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
  if (warp == 0) {
    s = sh.sums[0];
    for (int i = 1; i < kWarps; ++i) join(s, sh.sums[i]);
    count = lane < kWarps ? sh.count[lane] : 0, infinite = lane < kWarps ? sh.infinite[lane] : 0;
    count = __reduce_add_sync(0xffffffffu, count);
    infinite = __reduce_add_sync(0xffffffffu, infinite);
    Shared *first = &sh;
    if (ranks > 1) {
      uint64_t p;
      asm("mapa.u64 %0, %1, 0;\n" : "=l"(p) : "l"((uint64_t)&sh));
      first = reinterpret_cast<Shared *>(p);
    }
    if (lane == 0) first->all_sums[rank] = s, first->all_count[rank] = count, first->all_infinite[rank] = infinite;
    if (lane < n) first->all_keys[rank * kTop + lane] = sh.chosen[lane];
  }
  if (ranks > 1) cluster_sync();
  else __syncthreads();
  if (rank) return;
  s = sh.all_sums[0], count = sh.all_count[0], infinite = sh.all_infinite[0];
  for (int i = 1; i < ranks; ++i) join(s, sh.all_sums[i]), count += sh.all_count[i], infinite += sh.all_infinite[i];
  // logits of +infinity share all the mass
  const float ln = infinite ? logf((float)infinite) : logf(s.l);
  const auto logp_of = [&](float v) {
    if (!(v > -INFINITY)) return -INFINITY;
    return infinite ? (v == INFINITY ? -ln : -INFINITY) : (v - s.m) - ln;
  };
  if (tid == 0) {
    a.logp[row] = real ? logp_of(xt) : -INFINITY;
    if (a.rank) a.rank[row] = real ? count : -1;
    if (a.entropy) a.entropy[row] = infinite ? ln : s.l == 0.f ? 0.f : ln - s.w / s.l;
  }
  // the n highest of all: of ranks x n keys, those with fewer than n above
  if (tid < ranks * n) {
    const u64 k = sh.all_keys[tid / n * kTop + tid % n];
    int above = 0;
    for (int i = 0; i < ranks; ++i)
      for (int j = 0; j < n; ++j) {
        const u64 o = sh.all_keys[i * kTop + j];
        above += o > k || (o == k && i * n + j < tid);  // (only those of no token, 0, are equal)
      }
    if (above < n) {
      a.top_tokens[row * n + above] = k ? (int32_t)~(uint32_t)k : -1;
      a.top_logp[row * n + above] = k ? logp_of(of_key((uint32_t)(k >> 32))) : -INFINITY;
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                            const int32_t *tokens, int top, float *logp, int32_t *rank,
                            float *entropy, int32_t *top_tokens, float *top_logp,
                            cudaStream_t stream) {
  const int64_t sms = device_facts()->sm_count;
  // A cluster per row while rows do not fill the GPU, of slices of 4096 tokens or more.
  int ranks = 1;
  while (ranks < kMaxCluster && rows * ranks * 2 <= 2 * sms && vocab >= (int64_t)ranks * 2 * 4096) ranks *= 2;
  const int slice = (int)(((vocab + ranks - 1) / ranks + 63) / 64 * 64);
  for (int64_t r0 = 0; r0 < rows; r0 += 65535) {  // rows are the grid's y
    const int64_t n = rows - r0 < 65535 ? rows - r0 : 65535;
    const Args a = {static_cast<const uint8_t *>(logits) + r0 * ld * (dtype == Q4K_DTYPE_BF16 ? 2 : 4), ld, (int)vocab, slice, top,
                    tokens + r0, logp + r0, entropy ? entropy + r0 : nullptr, top_logp ? top_logp + r0 * top : nullptr,
                    rank ? rank + r0 : nullptr, top_tokens ? top_tokens + r0 * top : nullptr};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)n);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = dtype == Q4K_DTYPE_BF16 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<__nv_bfloat16>, a)
                                            : cudaLaunchKernelEx(&cfg, logprobs_kernel<float>, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace q4k
