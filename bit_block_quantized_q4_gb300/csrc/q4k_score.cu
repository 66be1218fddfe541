// q4k_score.cu -- log-probability and rank of given tokens, the distribution's
// entropy and its most likely tokens (q4k_logprobs).
//
// "spec: specialized model runtimes", section "Architecture": what is read off
// the logits belongs to tier T1, with the sampler.
//
// Mathematics.  In base 2: z_i = x_i log2 e - c with c a reference near the row's
// maximum, one multiply-add with one rounding, and in one pass
//   l = sum 2^z_i,   w = sum 2^z_i z_i,
//   logp(t) = (z_t - log2 l) ln 2,   entropy = (log2 l - w / l) ln 2;
// two parts with references c, c' are joined by l' 2^(c' - c) and
// (w' + (c' - c) l') 2^(c' - c).  Logits below -10^30 count as -10^30 beside any
// that are not: their weight is 0, and 0 times their z is 0 and not 0 times infinity.
// That one rounding of c leaves a residue of |c| 2^-24 in every z, which is the same
// for all and for z_t: of no account while |c| is small.  Rows whose maximum is beyond
// 2^22 either way (all masked with the lowest number, say) are done again by
// differences, x_i - max.
//
// Order.  Tokens are ordered by logit, highest first, equal ones by index: the
// descending order of the distinct integers key_i = (monotone image of x_i) <<
// 32 | ~i.
//
// Alternatives.  Every thread keeps the first of its highest logits.  The n-th
// highest of the maxima of 32 groups of threads is a bound that at least n tokens
// reach; a few dozen do in all, found again among the tokens of the threads whose
// own maximum reaches it.  Should more reach it than the list holds, they are
// taken one after the other instead.
//
// What bounds it: the logits are read once.  A row is one CTA's, or while rows
// are few a cluster's, whose CTAs take equal slices and send sums and lists to
// the first one.  Measured: 2047 x 131072 bf16 111 us (72% of the copy rate; issue
// slots 79% busy, the ALU pipe 59%), 1024 x 131072 fp32 87 us (92%; with 5
// alternatives 99), 64 x 131072 17 us,
// one row of 32000 11 us, of which the chain launch, load, cluster barrier, list is most.
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
constexpr int kThreads = 256, kWarps = kThreads / 32, kGroups = 4 * kWarps, kGroup = kThreads / kGroups;
static_assert(kGroups == 32 && kGroup == 8, "one warp looks at the maxima of all groups, eight lanes each");
constexpr int kTop = 32, kList = 1024, kMaxCluster = 8;
constexpr float kLow = -1e30f, kPlain = 4194304.f;  // what counts as masked; maxima up to here need no second pass
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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
  float c, l, w;
};
// (A reference stays finite, so that a vector with an infinite logit lies above any.)
constexpr float kNoRef = -3.0e38f, kMaxRef = 1e38f;
__device__ __forceinline__ void join(Sums &a, const Sums &b) {
  const float c = fmaxf(a.c, b.c);
  // without a token l is 0, and its reference says nothing; beyond 2^-200 a part counts for nothing
  const float da = a.l == 0.f ? 0.f : fmaxf(a.c - c, -200.f), db = b.l == 0.f ? 0.f : fmaxf(b.c - c, -200.f);
  const float fa = ex2(da), fb = ex2(db);
  a.w = fa * fmaf(da, a.l, a.w) + fb * fmaf(db, b.l, b.w);
  a.l = fa * a.l + fb * b.l;
  a.c = c;
}
// Eight logits as fp32, none below kLow and none NaN, and their maximum; with `raw`
// their maximum as they are (NaN only if all are).
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  static __device__ __forceinline__ float raw_top(const Raw8<float> &r) {
    return fmaxf(fmaxf(fmaxf(r.a.x, r.a.y), fmaxf(r.a.z, r.a.w)), fmaxf(fmaxf(r.b.x, r.b.y), fmaxf(r.b.z, r.b.w)));
  }
  static __device__ __forceinline__ float below(float x) {  // the next number below a finite one
    const int b = __float_as_int(x + 0.f);
    return b == 0 ? -1.4e-45f : __int_as_float(b > 0 ? b - 1 : b + 1);
  }
  static __device__ __forceinline__ float above(const Raw8<float> &r, float bar) {  // how many lie above
    float v[8];
    r.to(v);
    int n = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) n += v[j] > bar;
    return (float)n;
  }
  static __device__ __forceinline__ void clamped(const Raw8<float> &r, float (&v)[8]) {
    r.to(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fmaxf(v[j], kLow);
  }
};
template <>
struct Eight<__nv_bfloat16> {
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }
  static __device__ __forceinline__ float raw_top(const Raw8<__nv_bfloat16> &r) {
    const __nv_bfloat162 t = __hmax2(__hmax2(pair(r.a.x), pair(r.a.y)), __hmax2(pair(r.a.z), pair(r.a.w)));
    return fmaxf(__low2float(t), __high2float(t));
  }
  static __device__ __forceinline__ float below(float x) {
    const int b = __float_as_int(x + 0.f) >> 16;
    return b == 0 ? __int_as_float(0x80010000) : __int_as_float((b > 0 ? b - 1 : b + 1) << 16);
  }
  static __device__ __forceinline__ float above(const Raw8<__nv_bfloat16> &r, float bar) {
    const __nv_bfloat162 t = __float2bfloat162_rn(bar);  // (a bf16 value)
    const __nv_bfloat162 n = __hadd2(__hadd2(__hgt2(pair(r.a.x), t), __hgt2(pair(r.a.y), t)), __hadd2(__hgt2(pair(r.a.z), t), __hgt2(pair(r.a.w), t)));
    return __low2float(n) + __high2float(n);
  }
  static __device__ __forceinline__ void clamped(const Raw8<__nv_bfloat16> &r, float (&v)[8]) {
    const __nv_bfloat162 low = __float2bfloat162_rn(kLow);
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 p = __hmax2(pair(w[j]), low);
      const uint32_t u = *reinterpret_cast<const uint32_t *>(&p);
      v[2 * j] = __uint_as_float(u << 16), v[2 * j + 1] = __uint_as_float(u & 0xffff0000u);
    }
  }
};

struct Shared {
  Sums sums[kWarps];
  int count[kWarps], infinite[kWarps];
  float top[kWarps];        // highest logit
  u64 group[kGroups];       // highest key of each group
  u64 list[kList];
  u64 chosen[kTop];
  u64 bound;
  int listed;
  // of all CTAs of the cluster, in the first one
  Sums all_sums[kMaxCluster];
  int all_count[kMaxCluster], all_infinite[kMaxCluster];
  float all_top[kMaxCluster];
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
  Sums s = {kNoRef, 0.f, 0.f};
  float best = -INFINITY;  // highest logit, and where it was first seen (its vector's first token)
  int best_at = -1, count = 0, infinite = 0;
  float above = 0.f;                           // tokens above the given one (whole numbers below 2^24)
  const bool plain_xt = fabsf(xt) < INFINITY;  // has a next number below
  const float under = plain_xt ? Eight<T>::below(xt) : xt;
  float2 l2 = make_float2(0.f, 0.f), w2 = l2;  // s.l and s.w of the vectors

  const auto ahead = [&](float v, int i) {  // NaN counts as -infinity
    const float c = v > -INFINITY ? v : -INFINITY;
    return c > xt || (c == xt && i < token);
  };
  const auto single = [&](int i) {
    const float v = one(x + i);
    if (v > best || (v == best && i < best_at)) best = v, best_at = i;
    count += ahead(v, i);
    infinite += v == INFINITY;
    if (!(v > 0.1f * kLow) || v == INFINITY) return;
    const float c = v * kLog2e;
    if (c > s.c + 12.f) {  // as below
      const float d = fmaxf(s.c - c, -200.f), f = ex2(d);
      s.w = f * fmaf(d, s.l, s.w), s.l *= f, s.c = fminf(c, kMaxRef);
    }
    // (not as 2^0 with a reference of its own: c's rounding is the same for all only where c is)
    const float z = fmaf(v, kLog2e, -s.c), e = ex2(z);
    s.l += e, s.w = fmaf(e, z, s.w);
  };
  const auto eight = [&](const Raw8<T> &raw, int i) {
    const float top = Eight<T>::raw_top(raw);
    if (top > best) best = top, best_at = i;
    if (!(top < xt)) {
      // before the token equal logits count, after it they do not
      if (i + 8 <= token ? plain_xt : i >= token) {
        above += Eight<T>::above(raw, i >= token ? xt : under);
      } else {
        float v[8];
        raw.to(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) count += ahead(v[j], i + j);
      }
    }
    if (!(top > 0.1f * kLow)) return;  // nothing but what is masked
    const float ct = top * kLog2e;
    if (ct > s.c + 12.f) {  // the reference follows when it lies 2^12 and more below
      if (top == INFINITY) {
        float v[8];
        raw.to(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) infinite += v[j] == INFINITY;
      } else {
        // (l is 0 while there is no reference)
        const float d = fmaxf(s.c - ct, -200.f), f = ex2(d);
        const float2 f2 = make_float2(f, f);
        w2 = __fmul2_rn(f2, __ffma2_rn(make_float2(d, d), l2, w2));
        l2 = __fmul2_rn(f2, l2);
        s.c = fminf(ct, kMaxRef);
      }
    }
    float v[8];
    Eight<T>::clamped(raw, v);
    const float2 c2 = make_float2(-s.c, -s.c), log2e2 = make_float2(kLog2e, kLog2e);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 z = __ffma2_rn(make_float2(v[j], v[j + 1]), log2e2, c2), e = make_float2(ex2(z.x), ex2(z.y));
      l2 = __fadd2_rn(l2, e);
      w2 = __ffma2_rn(e, z, w2);
    }
  };
  // the next vectors are on their way while these are worked on
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  Raw8<T> next[U], raw[U];
  const T *from = x + v0;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (tid + u * kThreads < vectors) next[u].load(from + (tid + u * kThreads) * kV);
  for (int k0 = tid; k0 < vectors; k0 += U * kThreads) {
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = next[u];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + (U + u) * kThreads;
      if (k < vectors) next[u].load(from + k * kV);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kThreads;
      if (k < vectors) eight(raw[u], v0 + k * kV);
    }
  }
  s.l = l2.x + l2.y, s.w = w2.x + w2.y;
  if (tid < head) single(lo + tid);
  if (tid < hi - tail) single(tail + tid);
  count += (int)above;

  // the key of this thread's best
  u64 key = 0;
  if (a.top && best > -INFINITY) {
    int at = best_at;
    if (at >= v0 && at < tail) {  // the first of its vector that is as high
      float v[8];
      load8(x + at, v);
      int j = 7;
#pragma unroll
      for (int e = 6; e >= 0; --e) j = v[e] == best ? e : j;
      at += j;
    }
    key = key_at(best, at);
  }

  // ---- sums of the CTA: to the highest reference of the warp, then of the CTA
  const auto onto = [&](float c) {
    const float d = s.l == 0.f ? 0.f : fmaxf(s.c - c, -200.f), f = ex2(d);
    s.w = f * fmaf(d, s.l, s.w);
    s.l *= f;
    s.c = c;
  };
  onto(of_key(__reduce_max_sync(0xffffffffu, key_of(s.c))));
#pragma unroll
  for (int o = 16; o; o >>= 1) s.l += __shfl_xor_sync(0xffffffffu, s.l, o), s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
  count = __reduce_add_sync(0xffffffffu, count);
  infinite = __reduce_add_sync(0xffffffffu, infinite);
  float top = of_key(__reduce_max_sync(0xffffffffu, key_of(best)));
  if (lane == 0) sh.sums[warp] = s, sh.count[warp] = count, sh.infinite[warp] = infinite, sh.top[warp] = top;
  if (a.top) {
    u64 g = key;
#pragma unroll
    for (int o = kGroup / 2; o; o >>= 1) g = max64(g, shfl64(g, lane ^ o));
    if (lane % kGroup == 0) sh.group[(32 / kGroup) * warp + lane / kGroup] = g;
  }
  __syncthreads();

  // ---- this CTA's `top` highest keys, in order, in chosen[]
  const int n = a.top;
  if (n == 1) {
    if (warp == 0) {
      u64 g = sh.group[lane];
#pragma unroll
      for (int o = 16; o; o >>= 1) g = max64(g, shfl64(g, lane ^ o));
      if (lane == 0) sh.chosen[0] = g;
    }
  } else if (n) {
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
    const float bar = bound > 1 ? of_key((uint32_t)(bound >> 32)) : -INFINITY;
    const auto offer = [&](u64 k) {
      if (k >= bound) {
        const int i = atomicAdd(&sh.listed, 1);
        if (i < kList) sh.list[i] = k;
      }
    };
    // the threads whose best reaches the bound: they still hold all of their vectors, or
    // a warp goes through the tokens of one at a time
    const bool held = vectors <= U * kThreads;
    if (held && key >= bound) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (tid + u * kThreads < vectors && Eight<T>::raw_top(raw[u]) >= bar) {
          const int i = v0 + (tid + u * kThreads) * kV;
          float v[8];
          raw[u].to(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) offer(key_at(v[j], i + j));
        }
      if (tid < head) offer(key_at(one(x + lo + tid), lo + tid));
      if (tid < hi - tail) offer(key_at(one(x + tail + tid), tail + tid));
    }
    unsigned todo = __ballot_sync(0xffffffffu, !held && key >= bound);
    while (todo) {
      const int src = __ffs(todo) - 1, th = warp * 32 + src;
      todo &= todo - 1;
      for (int k = th + lane * kThreads; k < vectors; k += 32 * kThreads) {
        Raw8<T> r;
        const int i = v0 + k * kV;
        r.load(x + i);
        if (Eight<T>::raw_top(r) >= bar) {
          float v[8];
          r.to(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) offer(key_at(v[j], i + j));
        }
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
    const bool in = lane < kWarps;
    s = {in ? sh.sums[lane].c : kNoRef, in ? sh.sums[lane].l : 0.f, in ? sh.sums[lane].w : 0.f};
    count = __reduce_add_sync(0xffffffffu, in ? sh.count[lane] : 0);
    infinite = __reduce_add_sync(0xffffffffu, in ? sh.infinite[lane] : 0);
    top = of_key(__reduce_max_sync(0xffffffffu, key_of(in ? sh.top[lane] : -INFINITY)));
    onto(of_key(__reduce_max_sync(0xffffffffu, key_of(s.c))));
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) s.l += __shfl_xor_sync(0xffffffffu, s.l, o), s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
    __syncwarp();  // chosen[0]
    Shared *first = &sh;
    if (ranks > 1) {
      uint64_t p;
      asm("mapa.u64 %0, %1, 0;\n" : "=l"(p) : "l"((uint64_t)&sh));
      first = reinterpret_cast<Shared *>(p);
    }
    if (lane == 0) first->all_sums[rank] = s, first->all_count[rank] = count, first->all_infinite[rank] = infinite, first->all_top[rank] = top;
    if (lane < n) first->all_keys[rank * kTop + lane] = sh.chosen[lane];
  }
  if (ranks > 1) cluster_sync();
  else __syncthreads();
  if (rank) return;
  s = sh.all_sums[0], count = sh.all_count[0], infinite = sh.all_infinite[0], top = sh.all_top[0];
  for (int i = 1; i < ranks; ++i) {
    join(s, sh.all_sums[i]);
    count += sh.all_count[i], infinite += sh.all_infinite[i], top = fmaxf(top, sh.all_top[i]);
  }
  // a finite maximum beyond what one rounding of the reference allows: again by differences
  const bool again = fabsf(top) > kPlain && fabsf(top) < INFINITY;
  if (again) {
    s = {0.f, 0.f, 0.f};
    for (int i = tid; i < a.vocab; i += kThreads) {
      const float z = fmaxf((one(x + i) - top) * kLog2e, -200.f), e = ex2(z);  // (NaN too)
      s.l += e;
      s.w = fmaf(e, z, s.w);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s.l += __shfl_xor_sync(0xffffffffu, s.l, o), s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
    if (lane == 0) sh.sums[warp] = s;
    __syncthreads();
    s = sh.sums[0];
    for (int i = 1; i < kWarps; ++i) s.l += sh.sums[i].l, s.w += sh.sums[i].w;
  }
  // logits of +infinity share all the mass
  const float lg = log2f(infinite ? (float)infinite : s.l);
  const auto logp_of = [&](float v) {
    if (!(v > -INFINITY)) return -INFINITY;
    if (infinite) return v == INFINITY ? -lg * kLn2 : -INFINITY;
    if (again) return (v - top) - lg * kLn2;
    return v < kLow ? v - (s.c + lg) * kLn2 : (fmaf(v, kLog2e, -s.c) - lg) * kLn2;  // (v log2 e may be beyond all numbers)
  };
  if (tid == 0) {
    a.logp[row] = real ? logp_of(xt) : -INFINITY;
    if (a.rank) a.rank[row] = real ? count : -1;
    if (a.entropy) a.entropy[row] = (infinite ? lg : s.l == 0.f ? 0.f : lg - s.w / s.l) * kLn2;
  }
  // the n highest of all: of ranks x n keys, those with fewer than n above
  if (tid < ranks * n) {
    // each CTA's are in order: its own place, and by halving those above in the others
    // (only keys of no token, 0, are equal: there the earlier CTA's come first)
    const int mine = tid / n;
    const u64 k = sh.all_keys[mine * kTop + tid % n];
    int above = tid % n;
    for (int i = 0; i < ranks; ++i)
      if (i != mine) {
        int lo_n = 0, hi_n = n;
        while (lo_n < hi_n) {
          const int mid = (lo_n + hi_n) >> 1;
          const u64 o = sh.all_keys[i * kTop + mid];
          if (o > k || (o == k && i < mine)) lo_n = mid + 1;
          else hi_n = mid;
        }
        above += lo_n;
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
  // A cluster per row while rows do not fill the GPU, of slices of 2048 tokens or more.
  // Measured, us with clusters / without: 1 x 32000 fp32 11.0 / 12.4, 8 x 131072 bf16 12.3
  // / 22.6, 64 x 131072 fp32 17.2 / 30.0.  Clusters while CTAs are at most 1 / 2 / 4 / 8 times
  // the SMs: 64 x 131072 20.6 / 17.2 / 18.4 / 18.5, 256 x 131072 37.8 / 37.8 / 33.1 / 37.7, 120
  // x 32000 12.4 / 12.4 / 13.1 / 16.7.  Slices of 4096: 1 x 32000 12.4; of 1024: the same.
  int ranks = 1;
  while (ranks < kMaxCluster && rows * ranks * 2 <= 2 * sms && vocab >= (int64_t)ranks * 2 * 2048) ranks *= 2;
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
