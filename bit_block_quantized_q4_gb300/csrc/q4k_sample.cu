// q4k_sample.cu -- the choice of the next token from given random numbers
// (q4k_sample): temperature, top-k, top-p, min-p and the draw.
//
// "spec: specialized model runtimes", section "Architecture": the sampler is
// part of tier T1.
//
// Weights.  The draw and top-p compare sums of e_i = exp((x_i - max) /
// temperature) with borders, and in a flat row of 10^5 tokens a border lies
// within 10^-5 of any point: with weights good to 2^-23 about one row in a
// hundred would give another token than exact arithmetic.  So a weight is the
// integer rint(2^43 e_i), computed in pairs of fp32 numbers to about 2^-42 (fp64
// has 1/64 of the fp32 rate here and would take over a millisecond for 256 rows
// of 131072).  Integer sums are exact, the same in any order; 2^18 tokens sum
// below 2^61.
//
// Order.  Every filter keeps a prefix of the tokens in the order (logit
// descending, index ascending).  With c_i = (monotone integer image of x_i) <<
// 32 | ~i that order is the descending one of distinct integers, a filter is the
// smallest c_i kept, and the kept set is c_i >= the largest of these.
//
// Selection.  A cluster of up to 8 CTAs holds a row in its shared memory.  A
// histogram counts the tokens over (max - x) in kBins equal steps of the 46
// binary orders in which weights are not 0.  It gives the bin of the k-th token;
// and since the weights in a bin differ by a factor of 2^(46/kBins) at most, it
// bounds all sums of weights from both sides, and with them the bins in which
// the cumulative weight can reach top_p of the total.
//   - Up to kShort tokens down to the last of these bins (nearly always): they
//     are sent to the cluster's first CTA, which compares all pairs of them (up to
//     kThreads) or sorts them, and does the rest on the list.  Top-p without top-k needs the exact total of all weights too.
//   - Else each filter's smallest key is found by histograms over ever smaller
//     ranges of c_i, of counts or of exact weights, until at most kList tokens are
//     left, which are compared in pairs (whatever the ties); the draw then goes
//     over all tokens.  After top-p it takes the weights before the border's bins
//     from the pass that summed them: 256 rows of 131072 with top-p 0.9 alone
//     324 -> 301 us, flat ones 457 -> 415.
// Exact weights in the first histogram as well, by three more shared-memory
// additions per token, made 256 rows of 131072 with top-p alone take 370 us.
//
// What bounds it: the logits are read once from memory (bulk copies); after that
// a row with a top-k is bound by latency (barriers of the cluster, about 0.5 us
// each), and a row whose weights are all needed by their instructions, about 70
// each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/q4k.h"
#include "q4k_device.cuh"
#include "q4k_internal.h"
#include "q4k_step.h"

namespace q4k {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024, kList = kThreads, kShort = 2048;
constexpr float kOrders = 46.f;
constexpr float kOne = 8796093022208.f;  // weight of the highest logit, 2^43
constexpr float kLeastTemperature = 3.7615819e-37f;  // 2^-121
constexpr int kMaxCluster = 8, kMaxVocab = 262144;
// Tokens per CTA: few rows are spread as thin as kSliceLeast, many rows take as
// few CTAs as hold them with two CTAs per SM.
constexpr int kSliceMost = 16384, kSliceLeast = 2048;

struct SampleArgs {
  const void *logits;
  int64_t ld;
  int vocab, slice;  // slice: tokens per CTA, a multiple of 64
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *token;
  float *logp;
  unsigned *err;
};

// 2^(-j/256) as the sum of two fp32 numbers.
struct PowTable {
  float hi[256], lo[256];
};
constexpr PowTable make_pow() {
  PowTable t = {};
  for (int j = 0; j < 256; ++j) {
    const double z = -0.69314718055994530942 * j / 256;
    double term = 1, sum = 1;
    for (int i = 1; i < 24; ++i) {
      term *= z / i;
      sum += term;
    }
    t.hi[j] = (float)sum;
    t.lo[j] = (float)(sum - (double)t.hi[j]);
  }
  return t;
}
__device__ const PowTable kPow = make_pow();

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and +0 are one value
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// What a row's weights depend on.  Differences are taken of halves so that
// they cannot overflow; c = 2 log2(e) / temperature as two fp32 numbers.
struct Scale {
  float high, half, ch, cl, cb;
  const float2 *pow;  // 2^(-j/256) in shared memory
};

// 2^-y for 0 <= y = yh + yl < 64 as (wh + wl) 2^-e, to about 2^-42; wh in (0.49,
// 1.01).  (Every operation is written out, so that all passes over a row round
// alike.)
struct Pow {
  float wh, wl;
  int e;
};
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it leaves an integer in the low bits
__device__ __forceinline__ int magic_int(float x) { return __float_as_int(x) - 0x4B400000; }
__device__ __forceinline__ Pow pow_of(const float2 *table, float yh, float yl) {
  // y = n / 256 + r, |r| <= 1/512 and a little
  const float nm = __fmaf_rn(yh, 256.f, kMagic), nf = __fadd_rn(nm, -kMagic);
  const int n = magic_int(nm);
  const float r0 = __fmaf_rn(nf, -1.f / 256.f, yh), r = __fadd_rn(r0, yl);
  const float rl = __fsub_rn(yl, __fsub_rn(r, r0));
  // 2^-r - 1 = z + z^2/2 + ... as eh + el, z = -r ln 2
  constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.904654300e-9f;
  const float zh = __fmul_rn(r, -kLn2h);
  const float zl = __fmaf_rn(rl, -kLn2h, __fmaf_rn(r, -kLn2l, __fmaf_rn(r, -kLn2h, -zh)));
  const float q = __fmul_rn(__fmul_rn(zh, zh), __fmaf_rn(zh, __fmaf_rn(zh, 1.f / 24.f, 1.f / 6.f), 0.5f));
  const float eh = __fadd_rn(zh, q), el = __fadd_rn(__fsub_rn(q, __fsub_rn(eh, zh)), zl);
  // 2^-(n mod 256)/256 (1 + eh + el)
  const float2 p = table[n & 255];
  const float ph = __fmul_rn(p.x, eh), wh = __fadd_rn(p.x, ph);
  const float t = __fmaf_rn(p.x, el, __fmaf_rn(p.y, eh, p.y));
  const float wl = __fadd_rn(__fsub_rn(ph, __fsub_rn(wh, p.x)), __fadd_rn(__fmaf_rn(p.x, eh, -ph), t));
  return {wh, wl, n >> 8};
}

// rint(2^43 exp((x - max) / temperature)), to about 2^-42 relative.
__device__ __forceinline__ u64 weight(const Scale &s, float x) {
  // d = (max - x) / 2 as dh + dl, exactly
  const float b = -0.5f * x, dh = __fadd_rn(s.half, b), yh = __fmul_rn(dh, s.ch);
  if (!(yh < kOrders)) return 0;  // below 2^-46; -infinity, NaN
  const float bb = __fsub_rn(dh, s.half);
  const float dl = __fadd_rn(__fsub_rn(s.half, __fsub_rn(dh, bb)), __fsub_rn(b, bb));
  // y = d c in binary orders, as yh + yl
  const Pow p = pow_of(s.pow, yh, __fmaf_rn(dl, s.ch, __fmaf_rn(dh, s.cl, __fmaf_rn(dh, s.ch, -yh))));
  // 2^43 2^-e (wh + wl) = 2^22 (i + f), i an integer below 2^22, |f| <= 9/16
  const float scale = __int_as_float((148 - p.e) << 23);  // 2^(21-e)
  const float im = __fmaf_rn(p.wh, scale, kMagic), i = __fadd_rn(im, -kMagic);
  const float f = __fmaf_rn(p.wl, scale, __fmaf_rn(p.wh, scale, -i));
  return (u64)((int64_t)magic_int(im) * 4194304 + magic_int(__fmaf_rn(f, 4194304.f, kMagic)));
}

// ln(w / total) for 0 < w <= total, rounded once but for about 2^-40: y0 from
// fp32, then y0 + (w - total e^y0) / w, e^y0 in fp32 pairs and the difference in
// fp64 (a 64-bit division and logarithm cost 2 us here).
__device__ __forceinline__ float log_share(const float2 *table, u64 w, u64 total) {
  if (w == total) return 0.f;
  const float y0 = fminf(logf((float)w / (float)total), 0.f);
  constexpr float kLog2eh = 1.44269502162933349609375f, kLog2el = 1.925962991e-8f;
  const float yh = -y0 * kLog2eh, yl = fmaf(-y0, kLog2eh, -yh) - y0 * kLog2el;
  const Pow p = pow_of(table, yh, yl);
  const float f = __int_as_float((127 - p.e) << 23);  // 2^-e
  const double t = (double)total;
  const double d = fma(-t, (double)(p.wl * f), fma(-t, (double)(p.wh * f), (double)w));
  return y0 + (float)d / (float)w;
}

// Bin of a token, b for (max - x) in [b - 1/2, b + 1/2] steps: 0 for the largest,
// kBins and above for those of weight 0 (and for -infinity and NaN).  Not
// increasing in x.
__device__ __forceinline__ int bin_of(const Scale &s, float x) {
  const float t = __fmul_rn(__fmaf_rn(-0.5f, x, s.half), s.cb);
  return t < (float)kBins ? magic_int(__fadd_rn(t, kMagic)) : kBins;
}

__device__ __forceinline__ uint32_t ld_peer32(const void *p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(peer_smem(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ u64 ld_peer64(const void *p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];\n" : "=l"(v) : "r"(peer_smem(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_peer128(const void *p, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(peer_smem(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ void st_peer64(void *p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(peer_smem(smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_peer32(uint32_t *p, uint32_t rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;\n" : "=r"(old) : "r"(peer_smem(smem_u32(p), rank)), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void min_peer32(uint32_t *p, uint32_t rank, uint32_t v) {
  asm volatile("red.shared::cluster.min.u32 [%0], %1;\n" ::"r"(peer_smem(smem_u32(p), rank)), "r"(v) : "memory");
}
// p[i] += v in this CTA's shared memory, without a result.
__device__ __forceinline__ void add_own32(uint32_t base, int i, uint32_t v) {
  asm volatile("red.shared.add.u32 [%0], %1;\n" ::"r"(base + i * 4), "r"(v) : "memory");
}

// All threads of the cluster.  The barrier's instruction wants whole warps.
__device__ __forceinline__ void sync_cluster() {
  __syncwarp();
  cluster_sync();
}

// Sum over the block of the values before this thread's, and of all.
template <typename T>
__device__ __forceinline__ T scan_block(T *part, T v, T &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();  // earlier uses of part
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  T w = lane < kWarps ? part[lane] : T(0);
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, kWarps - 1);
  const T prev = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  return (warp ? prev : T(0)) + incl - v;
}

struct __align__(16) Shared {
  uint32_t top[kBins];  // the first histogram, over the cluster
  union {
    struct {
      uint32_t count[kBins];
      u64 weight[kBins];
    } split;
    u64 short_list[kShort];  // in the cluster's first CTA
  };
  // One use after the other, a cluster barrier between: the CTA's own sums (the
  // weights in three parts of 16 bits or less, so that 32768 tokens add up in 32
  // bits with the native additions), then the lists, or the short list's weights.
  union {
    struct {
      uint32_t count[kBins], w[3][kBins];
    } own;
    struct {
      u64 mine[kList], all[kList], weights[kList];
    } list;
    u64 short_weight[kShort];
  };
  float2 pow[256];
  u64 part[kWarps];
  float partf[kWarps];
  u64 found[4];  // bin, count before, weight before, count in it
  u64 cut;
  u64 total[kMaxCluster], before[kMaxCluster], inside[kMaxCluster], drawn[kMaxCluster];
  uint64_t full;
  float high;
  uint32_t listed, counts[kMaxCluster];
  int lo_bin;
  uint32_t best;  // the first token of the highest logit; in the draw, the warp of the target
};

__device__ __forceinline__ float2 load2(const float *x, int i) { return *reinterpret_cast<const float2 *>(x + i); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *x, int i) {
  const uint32_t w = *reinterpret_cast<const uint32_t *>(x + i);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T>
struct Ctx {
  Shared &s;
  const T *x;    // this CTA's tokens
  int n, base;   // how many, and the index of the first
  uint32_t rank, ranks;
  Scale sc;

  __device__ __forceinline__ u64 comp(int i, float v) const { return (u64)key_of(v) << 32 | (uint32_t)~(base + i); }

  __device__ __forceinline__ void zero_own() {
    uint32_t *zero = reinterpret_cast<uint32_t *>(&s.own);
    for (int i = threadIdx.x; i < (int)(sizeof(s.own) / 4); i += kThreads) zero[i] = 0;
  }

  // s.top: tokens per bin, over the cluster.  s.own and s.top are zero before.
  __device__ __forceinline__ void count_bins() {
    const int tid = threadIdx.x;
    const uint32_t at = smem_u32(s.own.count);
#pragma unroll 4
    for (int i = 2 * tid; i < n; i += 2 * kThreads) {
      const float2 v = load2(x, i);
      const int b0 = bin_of(sc, v.x), b1 = bin_of(sc, v.y);
      if (b0 < kBins) add_own32(at, b0, 1);
      if (b1 < kBins) add_own32(at, b1, 1);
    }
    sync_cluster();
    // Every CTA sums all CTAs' bins itself, which is cheaper than a second
    // barrier: 4 bins per thread, of half of the CTAs.
    static_assert(kThreads == kBins / 2, "two threads for 4 bins");
    const int v4 = tid & (kBins / 4 - 1), half = tid / (kBins / 4);
    uint4 c = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kMaxCluster / 2; ++j) {
      if (2 * j + half >= ranks) break;
      const uint32_t p = (rank + 2 * j + half) & (ranks - 1);  // not all from the same CTA at once
      const uint4 v = ld_peer128(&s.own.count[v4 * 4], p);
      c.x += v.x, c.y += v.y, c.z += v.z, c.w += v.w;
    }
    const uint32_t to = smem_u32(s.top);
    if (c.x) add_own32(to, v4 * 4, c.x);
    if (c.y) add_own32(to, v4 * 4 + 1, c.y);
    if (c.z) add_own32(to, v4 * 4 + 2, c.z);
    if (c.w) add_own32(to, v4 * 4 + 3, c.w);
    __syncthreads();
  }

  // s.split: counts and weights of kBins steps of 2^shift keys down from hi, of
  // the keys in [lo, hi].  (The members are copied first: the additions to shared
  // memory would have them loaded again for every token.)
  __device__ void split_range(u64 lo, u64 hi, int shift, bool with_weights) {
    const int tid = threadIdx.x, n = this->n, base = this->base;
    const uint32_t rank = this->rank, ranks = this->ranks, lo32 = (uint32_t)(lo >> 32), hi32 = (uint32_t)(hi >> 32);
    const Scale sc = this->sc;
    const T *const x = this->x;
    Shared &s = this->s;
    zero_own();
    __syncthreads();
    const uint32_t at = smem_u32(&s.own);
    const auto add = [&](int i, float e) {
      const uint32_t k32 = key_of(e);
      if (k32 < lo32 || k32 > hi32) return;
      const u64 k = (u64)k32 << 32 | (uint32_t)~(base + i);
      if (k < lo || k > hi) return;
      const int b = (int)((hi - k) >> shift);
      add_own32(at, b, 1);
      if (with_weights) {
        const u64 w = weight(sc, e);
        add_own32(at, kBins + b, (uint32_t)w & 0xffffu);
        add_own32(at, 2 * kBins + b, (uint32_t)(w >> 16) & 0xffffu);
        add_own32(at, 3 * kBins + b, (uint32_t)(w >> 32));
      }
    };
    for (int i = 2 * tid; i < n; i += 2 * kThreads) {
      const float2 v = load2(x, i);
      add(i, v.x);
      add(i + 1, v.y);
    }
    sync_cluster();
    if (tid < kBins / 4) {
      uint32_t c[4] = {};
      u64 w[4] = {};
#pragma unroll 2
      for (uint32_t j = 0; j < ranks; ++j) {
        const uint32_t p = (rank + j) & (ranks - 1);  // not all from the same CTA at once
        const uint4 v = ld_peer128(&s.own.count[tid * 4], p);
        c[0] += v.x, c[1] += v.y, c[2] += v.z, c[3] += v.w;
        if (with_weights) {
          const uint4 a0 = ld_peer128(&s.own.w[0][tid * 4], p), a1 = ld_peer128(&s.own.w[1][tid * 4], p),
                      a2 = ld_peer128(&s.own.w[2][tid * 4], p);
          w[0] += a0.x + ((u64)a1.x << 16) + ((u64)a2.x << 32);
          w[1] += a0.y + ((u64)a1.y << 16) + ((u64)a2.y << 32);
          w[2] += a0.z + ((u64)a1.z << 16) + ((u64)a2.z << 32);
          w[3] += a0.w + ((u64)a1.w << 16) + ((u64)a2.w << 32);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s.split.count[tid * 4 + j] = c[j], s.split.weight[tid * 4 + j] = w[j];
    }
    __syncthreads();
  }

  // The step of s.split in which the sum of counts (or weights), from c0 and w0
  // on, first reaches `want`: found[] = step, count and weight before it, its
  // count.
  __device__ void find(bool by_weight, u64 want, u64 c0, u64 w0) {
    constexpr int PER = kBins / kThreads;
    const int tid = threadIdx.x;
    u64 c = 0, w = 0, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) c += s.split.count[tid * PER + j], w += s.split.weight[tid * PER + j];
    u64 ci = c0 + scan_block(s.part, c, all), wi = w0 + scan_block(s.part, w, all);
    if (tid == 0) s.found[0] = kBins;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const u64 hc = s.split.count[tid * PER + j], hw = s.split.weight[tid * PER + j];
      const u64 from = by_weight ? wi : ci, to = from + (by_weight ? hw : hc);
      if (from < want && to >= want) s.found[0] = tid * PER + j, s.found[1] = ci, s.found[2] = wi, s.found[3] = hc;
      ci += hc, wi += hw;
    }
    __syncthreads();
  }

  // The smallest key of a bin <= b: bins do not increase with the key, so 32
  // keys at a time tell between which two it lies.
  __device__ uint32_t least_key(int b) const {
    const uint32_t lane = threadIdx.x & 31;
    const Scale sc = this->sc;
    uint32_t l = 0, r = key_of(sc.high);  // the answer is in [l, r]
    while (l < r) {
      const uint32_t step = (r - l) / 33 + 1, m = l + min((r - l), step * lane);
      const unsigned in = __ballot_sync(0xffffffffu, bin_of(sc, of_key(m)) <= b);
      const int f = in ? __ffs(in) - 1 : 32;  // the first key that is
      if (f < 32) r = l + min(r - l, step * f);
      if (f > 0) l = min(l + min(r - l, step * (f - 1)) + 1, r);
      else r = l;
    }
    return l;
  }

  // The smallest key kept when a token is kept if the sum of counts (or
  // weights) of those before it is less than `want`; it lies in bins b0 .. b1,
  // which hold `count` tokens, with c0 tokens and weight w0 before them.
  __device__ u64 select(bool by_weight, u64 want, int b0, int b1, u64 c0, u64 w0, u64 count) {
    const int tid = threadIdx.x, n = this->n, base = this->base;
    const uint32_t ranks = this->ranks;
    const Scale sc = this->sc;
    const T *const x = this->x;
    Shared &s = this->s;
    u64 lo = (u64)least_key(b1) << 32;
    u64 hi = b0 ? ((u64)least_key(b0 - 1) << 32) - 1 : (u64)key_of(sc.high) << 32 | 0xffffffffu;
    while (count > kList) {
      const int bits = 64 - __clzll((long long)(hi - lo));
      const int shift = bits > 10 ? bits - 10 : 0;
      sync_cluster();  // the lists or sums that shared this memory are read
      split_range(lo, hi, shift, by_weight);
      find(by_weight, want, c0, w0);
      const u64 b = s.found[0];
      if (b >= kBins) return 0;  // cannot be: the sum reaches `want` in this range
      c0 = s.found[1], w0 = s.found[2], count = s.found[3];
      hi -= b << shift;
      const u64 width = (1ull << shift) - 1;
      lo = hi - lo > width ? hi - width : lo;
    }
    // list the tokens: each CTA its own, then all of them everywhere
    sync_cluster();
    if (tid == 0) s.listed = 0, s.cut = ~0ull;
    __syncthreads();
    const uint32_t lo32 = (uint32_t)(lo >> 32), hi32 = (uint32_t)(hi >> 32);
    const auto list = [&](int i, float e) {
      const uint32_t k32 = key_of(e);
      if (k32 < lo32 || k32 > hi32) return;
      const u64 k = (u64)k32 << 32 | (uint32_t)~(base + i);
      if (k >= lo && k <= hi) s.list.mine[atomicAdd(&s.listed, 1u)] = k;
    };
#pragma unroll 4
    for (int i = 2 * tid; i < n; i += 2 * kThreads) {
      const float2 v = load2(x, i);
      list(i, v.x);
      list(i + 1, v.y);
    }
    sync_cluster();
    if (tid < (int)ranks) s.counts[tid] = ld_peer32(&s.listed, tid);
    __syncthreads();
    const int at = (int)count;
    if (tid < at) {
      uint32_t p = 0, i = tid;
      while (p + 1 < ranks && i >= s.counts[p]) i -= s.counts[p++];
      const u64 k = ld_peer64(&s.list.mine[min(i, (uint32_t)kList - 1)], p);
      s.list.all[tid] = k;
      s.list.weights[tid] = by_weight ? weight(sc, of_key((uint32_t)(k >> 32))) : 0;
    }
    __syncthreads();
    if (tid < at) {
      const u64 k = s.list.all[tid];
      u64 before = by_weight ? w0 : c0;
      for (int j = 0; j < at; ++j)
        if (s.list.all[j] > k) before += by_weight ? s.list.weights[j] : 1;
      if (before < want) atomicMin(&s.cut, k);
    }
    __syncthreads();
    return s.cut;
  }
};

// Sort key[0 .. E * kThreads) descending by a bitonic network, E keys per
// thread: steps within a thread in registers, within a warp by shuffles, and
// the few across warps through shared memory.  Unrolled, so that the steps'
// directions are constants or one predicate (as loops a step of 1024 keys took
// 270 cycles).
template <int E>
__device__ __noinline__ void sort_keys(u64 *key) {
  const int tid = threadIdx.x;
  u64 e[E];
#pragma unroll
  for (int a = 0; a < E; ++a) e[a] = key[tid * E + a];
#pragma unroll
  for (int k = 2; k <= E * kThreads; k *= 2) {
#pragma unroll
    for (int j = k / 2; j; j /= 2) {
      if (j < E) {
#pragma unroll
        for (int a = 0; a < E; ++a) {
          if (a & j) continue;
          const bool down = k < E ? (a & k) == 0 : ((tid * E) & k) == 0;
          const u64 p = e[a], q = e[(a | j) % E];
          if ((p < q) == down) e[a] = q, e[(a | j) % E] = p;
        }
      } else {
        const int m = j / E;  // distance of the partner thread
        const bool larger = (((tid * E) & k) == 0) == ((tid & m) == 0);  // this one keeps the larger
        if (m >= 32) {
          __syncthreads();
#pragma unroll
          for (int a = 0; a < E; ++a) key[tid * E + a] = e[a];
          __syncthreads();
        }
#pragma unroll
        for (int a = 0; a < E; ++a) {
          const u64 q = m >= 32 ? key[(tid ^ m) * E + a] : __shfl_xor_sync(0xffffffffu, e[a], m & 31);
          if ((q > e[a]) == larger) e[a] = q;
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < E; ++a) key[tid * E + a] = e[a];
  __syncthreads();
}
// Sort the first m of kShort keys; the keys behind them are made 0.
__device__ __forceinline__ void sort_down(u64 *key, int m) {
  const int size = m <= 2 * kThreads ? 2 * kThreads : 4 * kThreads;
  static_assert(kShort == 4 * kThreads, "the list is what 4 keys per thread sort");
  for (int i = m + threadIdx.x; i < size; i += kThreads) key[i] = 0;
  __syncthreads();
  if (size == 2 * kThreads) sort_keys<2>(key);
  else sort_keys<4>(key);
}

__device__ __forceinline__ u64 share_of(float part, u64 total) {  // floor(part * total), part in [0, 1]
  return (u64)((double)part * (double)total);
}
// before < top_p * total, and at least the first token: before < want
__device__ __forceinline__ u64 want_of(float p, u64 total) {
  return max(1ull, (u64)ceil((double)fmaxf(p, 0.f) * (double)total));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared &s = *reinterpret_cast<Shared *>(raw);
  T *x = reinterpret_cast<T *>(raw + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.y;
  const int row = blockIdx.x;
  const int base = (int)rank * a.slice, n = a.slice, live = max(0, min(a.vocab - base, n));
  const T *in = static_cast<const T *>(a.logits) + row * a.ld + base;
  Ctx<T> c = {s, x, n, base, rank, ranks, {}};

  // ---- the row's slice into shared memory, and its maximum
  const T kNone = (T)-INFINITY;
  const bool aligned = (reinterpret_cast<uintptr_t>(in) & 15) == 0;
  constexpr int V = 16 / sizeof(T);
  const int bulk = aligned ? live / V * V : 0;  // tokens that come by bulk copies
  if (tid == 0) {
    mbar_init(&s.full, 1);
    fence_mbar_init();
    if (bulk) {
      constexpr int kPiece = 8192;
      mbar_arrive_expect_tx(&s.full, bulk * sizeof(T));
      for (int at = 0; at < bulk * (int)sizeof(T); at += kPiece)
        bulk_load(reinterpret_cast<uint8_t *>(x) + at, reinterpret_cast<const uint8_t *>(in) + at,
                  min(kPiece, bulk * (int)sizeof(T) - at), &s.full);
    }
    s.listed = 0, s.best = 0xffffffffu;
  }
  const float t = a.temperature ? a.temperature[row] : 1.f;
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.f;
  const float u = fminf(fmaxf(a.u[row], 0.f), 1.f);
  for (int i = bulk + tid; i < n; i += kThreads) x[i] = i < live ? in[i] : kNone;
  for (int i = tid; i < 256; i += kThreads) s.pow[i] = make_float2(kPow.hi[i], kPow.lo[i]);
  for (int i = tid; i < kBins; i += kThreads) s.top[i] = 0;
  c.zero_own();
  __syncthreads();
  // a copy that does not arrive in time ends the whole cluster, at the barrier
  // below; the row's outputs are then not written
  const bool late = bulk && !mbar_wait(&s.full, 0, a.err);
  float high = -INFINITY;
  if (!late)
    for (int i = 2 * tid; i < n; i += 2 * kThreads) {
      const float2 v = load2(x, i);
      high = fmaxf(high, fmaxf(v.x, v.y));  // NaN is passed over
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
  if (lane == 0) s.partf[warp] = high;
  const int any_late = __syncthreads_or(late);
  if (tid < 32) {
    high = lane < kWarps ? s.partf[lane] : -INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
    if (lane == 0) s.high = any_late ? NAN : high;
  }
  sync_cluster();
  const float h = __uint_as_float(ld_peer32(&s.high, lane & (ranks - 1)));  // ranks is a power of two
  if (__any_sync(0xffffffffu, h != h)) {
    if (any_late && tid == 0) drain_ring(&s.full, 1, 0, 0, 1);
    sync_cluster();
    return;
  }
  high = h;
#pragma unroll
  for (int o = kMaxCluster / 2; o; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));

  const bool none = high == -INFINITY;
  if (none || !(t > 0.f)) {
    // the first token of the highest logit, sent to the first CTA
    uint32_t best = 0xffffffffu;
    for (int i = 2 * tid; i < n; i += 2 * kThreads) {
      const float2 v = load2(x, i);
      if (v.y == high) best = min(best, (uint32_t)(base + i + 1));
      if (v.x == high) best = min(best, (uint32_t)(base + i));
    }
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0 && best != 0xffffffffu) min_peer32(&s.best, 0, best);
    sync_cluster();
    if (rank == 0 && tid == 0) {
      a.token[row] = none ? -1 : (int32_t)s.best;
      if (a.logp) a.logp[row] = none ? -INFINITY : 0.f;
    }
    return;
  }
  if (high == INFINITY) {  // its tokens share everything: they are the row's only ones
    for (int i = tid; i < n; i += kThreads) x[i] = (float)x[i] == high ? (T)0.f : kNone;
    high = 0.f;
    __syncthreads();
  }
  // c = 2 log2(e) / t as two fp32 numbers.  The least temperature keeps c, and
  // the bins per difference, finite.
  constexpr float kLh = 2.8853900432586669922f, kLl = 3.851925982e-8f;
  const float least_t = fmaxf(t, kLeastTemperature), ch = kLh / least_t;
  const float cl = ch > 0.f ? (fmaf(-ch, least_t, kLh) + kLl) / least_t : 0.f;
  c.sc = {high, 0.5f * high, ch, cl, ch * (kBins / kOrders), s.pow};
  // min-p: e_i >= min_p, as weights
  const u64 least = mp > 0.f ? max(1ull, (u64)ceilf(fminf(mp, 1.f) * kOne)) : 0;

  // The tokens of a warp are contiguous, so that the order of the warps' sums is
  // that of the indexes.
  const int run = (n + 2 * kThreads - 1) / (2 * kThreads) * 64, i0 = min(n, warp * run), i1 = min(n, i0 + run);

  // ---- the filters, each as the smallest key it keeps
  u64 cut = 0;
  // Top-p leaves the weight of this warp's tokens in bins before b0, all of them
  // kept, to the draw, which then looks at bins b0 .. b1 only.
  bool have_less = false;
  u64 warp_less = 0;
  int b0 = 0, b1 = 0;
  const bool use_k = k > 0 && k < a.vocab, use_p = p < 1.f;
  if (use_k || use_p) {
    c.count_bins();
    // Tokens before and in this thread's bins; the bin of the k-th; and bounds
    // of the weights of the first k in each bin, with a little to spare for the
    // bins' rounded borders.
    constexpr int PER = kBins / kThreads;
    const float step = kOrders / kBins;
    uint32_t have[PER], tokens = 0, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) have[j] = s.top[tid * PER + j], tokens += have[j];
    const uint32_t first = scan_block(reinterpret_cast<uint32_t *>(s.partf), tokens, all);
    const bool whole = !use_k || all <= (uint32_t)k;  // the top-k set is everything of any weight
    const uint32_t most = whole ? all : (uint32_t)k;
    if (tid == 0) s.found[0] = kBins - 1, s.found[1] = 0, s.found[2] = all;
    __syncthreads();
    uint32_t at = first;
    float kept_in[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      kept_in[j] = (float)(at < most ? min(have[j], most - at) : 0);
      if (at < most && at + have[j] >= most) s.found[0] = tid * PER + j, s.found[1] = at, s.found[2] = at + have[j];
      at += have[j];
    }
    __syncthreads();
    const int bk = (int)s.found[0];  // the bin of the last of them, and the tokens before and up to it
    const uint32_t before_k = (uint32_t)s.found[1], upto_k = (uint32_t)s.found[2];
    // The first bin up to which the sum over bins of tokens times
    // 2^-((b + shift) step) reaches `part` of the sum over all bins with all_shift
    // (the highest logit itself counts 1); at most bk.
    const auto reach = [&](float shift, float all_shift, float part) {
      float v[PER], sum = 0.f, other = 0.f, total, other_total;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int b = tid * PER + j;
        const float most_one = b == 0 ? fminf(kept_in[j], 1.f) : 0.f;
        v[j] = (kept_in[j] - most_one) * exp2f(-fmaxf(b + shift, 0.f) * step) + most_one;
        sum += v[j];
        other += (kept_in[j] - most_one) * exp2f(-fmaxf(b + all_shift, 0.f) * step) + most_one;
      }
      float c0 = scan_block(s.partf, sum, total);
      scan_block(s.partf, other, other_total);
      if (tid == 0) s.lo_bin = bk;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        c0 += v[j];
        if (have[j] && c0 >= part * other_total) atomicMin(&s.lo_bin, tid * PER + j);
      }
      __syncthreads();
      const int b = s.lo_bin;
      __syncthreads();
      return b;
    };
    // tokens before bin b0 and up to bin b1
    const auto span = [&](int b0, int b1, uint32_t &before, uint32_t &upto) {
      uint32_t sum = first;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (tid * PER + j == b0) s.found[0] = sum;
        sum += have[j];
        if (tid * PER + j == b1) s.found[3] = sum;
      }
      __syncthreads();
      before = (uint32_t)s.found[0], upto = (uint32_t)s.found[3];
    };
    const float pp = fmaxf(p, 0.f);
    b1 = bk;  // the last bin in which the last kept token can lie
    uint32_t count = upto_k, unused;
    if (use_p && whole) {  // the weights of a bin are at least those of its end, all at most those of their bins' beginnings
      b1 = reach(0.51f, -0.51f, pp * 1.001f);
      span(0, b1, unused, count);
    }
    bool have_total = false;
    u64 total_p = 0, less_p = 0;
    if (count > kShort && use_k && !whole) cut = c.select(false, (u64)k, bk, bk, before_k, 0, upto_k - before_k);
    if (count > kShort && use_p) {
      // Exact sums: the total of the top-k set, and the weight before bin b0 and
      // up to bin b1, at first for the bins next to where the middles of all
      // bins put the border, then for the bins that are sure to hold it.
      for (int round = 0; round < 2; ++round) {
        b0 = round ? reach(-0.51f, 0.51f, pp * 0.999f) : reach(0.f, 0.f, pp * 0.996f);
        b1 = round ? reach(0.51f, -0.51f, pp * 1.001f) : reach(0.f, 0.f, pp * 1.004f);
        b0 = min(b0, b1);
        u64 sum = 0, less = 0, in = 0, mine;
        for (int i = i0 + 2 * lane; i < i1; i += 64) {
          const float2 v = load2(x, i);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float e = j ? v.y : v.x;
            const u64 w = !cut || c.comp(i + j, e) >= cut ? weight(c.sc, e) : 0;
            const int b = bin_of(c.sc, e);
            sum += w;
            if (b < b0) less += w;
            if (b <= b1) in += w;
          }
        }
        warp_less = less;
        sync_cluster();  // earlier sums are read
        scan_block(s.part, sum, mine);
        if (tid < (int)ranks) st_peer64(&s.total[rank], tid, mine);
        scan_block(s.part, less, mine);
        if (tid < (int)ranks) st_peer64(&s.before[rank], tid, mine);
        scan_block(s.part, in, mine);
        if (tid < (int)ranks) st_peer64(&s.inside[rank], tid, mine);
        sync_cluster();
        total_p = less_p = in = 0;
        for (uint32_t q = 0; q < ranks; ++q) total_p += s.total[q], less_p += s.before[q], in += s.inside[q];
        const u64 want = want_of(p, total_p);
        if (less_p < want && want <= in) break;
      }
      have_total = true;
      uint32_t before_p, upto_p;
      span(b0, b1, before_p, upto_p);
      if (whole && upto_p <= kShort) {
        count = upto_p;
      } else {
        cut = max(cut, c.select(true, want_of(p, total_p), b0, b1, before_p, less_p, upto_p - before_p));
        have_less = least == 0;
      }
    }
    const int last = b1;
    if (count <= kShort) {
      // Top-p without top-k: its total is that of all tokens.
      const bool sum_all = use_p && whole && !have_total;
      u64 sum = 0, total;
#pragma unroll 4
      for (int i = 2 * tid; i < n; i += 2 * kThreads) {
        const float2 v = load2(x, i);
        if (bin_of(c.sc, v.x) <= last) st_peer64(&s.short_list[add_peer32(&s.listed, 0, 1)], 0, c.comp(i, v.x));
        if (bin_of(c.sc, v.y) <= last) st_peer64(&s.short_list[add_peer32(&s.listed, 0, 1)], 0, c.comp(i + 1, v.y));
        if (sum_all) sum += weight(c.sc, v.x) + weight(c.sc, v.y);
      }
      if (sum_all) {
        scan_block(s.part, sum, total);
        if (tid == 0) st_peer64(&s.total[rank], 0, total);
      }
      sync_cluster();
      if (rank != 0) return;
      const int m = (int)count;
      if (m <= kThreads) {
        // One token per thread, compared with all others: of those before it
        // (larger keys) the number and the weight; then of the kept ones the
        // weight up to it in the order of the indexes.
        const u64 key = tid < m ? s.short_list[tid] : 0;
        u64 w = tid < m ? weight(c.sc, of_key((uint32_t)(key >> 32))) : 0;
        if (tid < m) s.short_weight[tid] = w;
        if (tid == 0) s.cut = have_total ? total_p : 0;
        __syncthreads();
        u64 before = 0;
        uint32_t place = 0;
        const bool mine = warp * 32 < m;  // the warp has tokens
        if (mine) {
#pragma unroll 4
          for (int j = 0; j < m; ++j)
            if (s.short_list[j] > key) ++place, before += s.short_weight[j];
        }
        if (use_p) {
          // the total of the top-k set: up to its last token
          if (!whole && tid < m && place == (uint32_t)k - 1) s.cut = before + w;
          if (sum_all && tid == 0)
            for (uint32_t q = 0; q < ranks; ++q) s.cut += s.total[q];
          __syncthreads();
          if (before >= want_of(p, s.cut)) w = 0;
        }
        if (use_k && place >= (uint32_t)k) w = 0;
        if (w < least) w = 0;
        __syncthreads();
        if (tid < m) s.short_weight[tid] = w;
        __syncthreads();
        if (!mine) return;
        u64 upto = 0;
        total = 0;
#pragma unroll 4
        for (int j = 0; j < m; ++j) {
          const u64 e = s.short_weight[j];
          total += e;
          if ((uint32_t)s.short_list[j] >= (uint32_t)key) upto += e;  // the low half is ~index
        }
        u64 target = share_of(u, total);
        if (target >= total) target = total - 1;
        if (w && upto > target && upto - w <= target) {
          a.token[row] = (int32_t)~(uint32_t)key;
          if (a.logp) a.logp[row] = log_share(s.pow, w, total);
        }
        return;
      }
      constexpr int PS = kShort / kThreads;  // tokens per thread, in order
      sort_down(s.short_list, m);
      const int kept_k = use_k ? min(m, k) : m;
      u64 w[PS], key[PS];
      sum = 0;
#pragma unroll
      for (int j = 0; j < PS; ++j) {
        const int i = PS * tid + j;
        key[j] = i < kept_k ? s.short_list[i] : 0;
        w[j] = i < kept_k ? weight(c.sc, of_key((uint32_t)(key[j] >> 32))) : 0;
        sum += w[j];
      }
      u64 before = scan_block(s.part, sum, total);
      if (have_total) total = total_p;
      if (sum_all) {
        total = 0;
        for (uint32_t q = 0; q < ranks; ++q) total += s.total[q];
      }
      const u64 want = use_p ? want_of(p, total) : ~0ull;
      int mine = 0;
#pragma unroll
      for (int j = 0; j < PS; ++j) {
        const u64 e = w[j];
        if (before >= want || e < least) w[j] = 0;
        before += e;
        mine += w[j] != 0;
      }
      int kept;  // the first `kept` of the order
      scan_block(reinterpret_cast<int *>(s.partf), mine, kept);
      // by index: ~i high, the place in the order low
#pragma unroll
      for (int j = 0; j < PS; ++j) {
        const int i = PS * tid + j;
        if (i < kept) {
          s.short_weight[i] = w[j];
          s.short_list[i] = key[j] << 32 | (uint32_t)i;
        }
      }
      sort_down(s.short_list, kept);
      sum = 0;
#pragma unroll
      for (int j = 0; j < PS; ++j) {
        const int i = PS * tid + j;
        key[j] = i < kept ? s.short_list[i] : 0;
        w[j] = i < kept ? s.short_weight[(uint32_t)key[j]] : 0;
        sum += w[j];
      }
      before = scan_block(s.part, sum, total);
      u64 target = share_of(u, total);
      if (target >= total) target = total - 1;
#pragma unroll
      for (int j = 0; j < PS; ++j) {
        if (before <= target && target < before + w[j]) {
          a.token[row] = (int32_t)~(uint32_t)(key[j] >> 32);
          if (a.logp) a.logp[row] = log_share(s.pow, w[j], total);
        }
        before += w[j];
      }
      return;
    }
  }

  // ---- the draw
  const auto kept1 = [&](int i, float v) -> u64 {
    if (c.comp(i, v) < cut) return 0;
    const u64 w = weight(c.sc, v);
    return w < least ? 0 : w;
  };
  u64 sum = 0;
  if (have_less) {
    sum = warp_less;
    for (int i = i0 + 2 * lane; i < i1; i += 64) {
      const float2 v = load2(x, i);
      const int bx = bin_of(c.sc, v.x), by = bin_of(c.sc, v.y);
      if (bx >= b0 && bx <= b1) sum += kept1(i, v.x);
      if (by >= b0 && by <= b1) sum += kept1(i + 1, v.y);
    }
  } else if (cut == 0 && least == 0) {
    for (int i = i0 + 2 * lane; i < i1; i += 64) {
      const float2 v = load2(x, i);
      sum += weight(c.sc, v.x) + weight(c.sc, v.y);
    }
  } else {
    for (int i = i0 + 2 * lane; i < i1; i += 64) {
      const float2 v = load2(x, i);
      sum += kept1(i, v.x) + kept1(i + 1, v.y);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  u64 mine, before = scan_block(s.part, lane == 0 ? sum : 0, mine);
  before = __shfl_sync(0xffffffffu, before, 0);  // before this warp's tokens
  if (tid < (int)ranks) st_peer64(&s.drawn[rank], tid, mine);
  sync_cluster();  // from here on the CTAs are on their own
  u64 total = 0;
  for (uint32_t q = 0; q < ranks; ++q) {
    if (q < rank) before += s.drawn[q];
    total += s.drawn[q];
  }
  // cumulative > u * total, for an integer: cumulative > floor(u * total)
  u64 target = share_of(u, total);
  if (target >= total) target = total - 1;
  // The warp whose tokens reach the target tells the block, which goes through
  // them again together (one warp alone took 6 us for its 1024).
  if (lane == 0 && before <= target && target < before + sum) s.best = warp, s.cut = before;
  __syncthreads();
  if (s.best == 0xffffffffu) return;
  const int from = min(n, (int)s.best * run), to = min(n, from + run);
  const int per = (run + 2 * kThreads - 1) / (2 * kThreads) * 2, j0 = min(to, from + tid * per), j1 = min(to, j0 + per);
  u64 own = 0;
  for (int i = j0; i < j1; i += 2) {
    const float2 v = load2(x, i);
    own += kept1(i, v.x) + kept1(i + 1, v.y);
  }
  u64 upto = s.cut + scan_block(s.part, own, mine);
  if (upto <= target && target < upto + own) {
    for (int i = j0; i < j1; ++i) {
      const u64 w = kept1(i, (float)x[i]);
      upto += w;
      if (upto > target) {
        a.token[row] = base + i;
        if (a.logp) a.logp[row] = log_share(s.pow, w, total);
        break;
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const SampleArgs &a, int64_t rows, int ranks, cudaStream_t stream) {
  static SmemLimit limit;
  cudaError_t e = raise_smem_limit(limit, sample_kernel<T>, (int)sizeof(Shared) + kMaxVocab / kMaxCluster * (int)sizeof(T));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows, ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared) + (size_t)a.slice * sizeof(T);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = ranks;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                          const float *u, const float *temperature, const int32_t *top_k,
                          const float *top_p, const float *min_p, int32_t *token, float *logp,
                          cudaStream_t stream) {
  int ranks = 1;
  while (ranks < kMaxCluster && (vocab > ranks * kSliceMost || (vocab > ranks * kSliceLeast && rows * ranks < 2 * device_facts()->sm_count))) ranks *= 2;
  const int slice = (int)((vocab + ranks - 1) / ranks + 63) / 64 * 64;
  const SampleArgs a = {logits, ld, (int)vocab, slice, u, temperature, top_p, min_p, top_k, token, logp, device_error_word()};
  return dtype == Q4K_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, rows, ranks, stream) : launch_t<float>(a, rows, ranks, stream);
}

}  // namespace q4k
