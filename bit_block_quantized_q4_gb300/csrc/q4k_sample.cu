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
// histogram over (max - x) in kBins equal steps of the 46 binary orders in which
// weights are not 0 (counts, and the exact weight of each bin where top-p needs
// it) gives the bin in which the k-th token lies, or in which the cumulative
// weight reaches top_p of the total.
//   - Up to kShort tokens in that bin and above (nearly always with a top-k):
//     they are sent to the cluster's first CTA, which sorts them and does the
//     rest on the list.
//   - Else each filter's smallest key is found (the bin's tokens compared in
//     pairs; a bin of more than kList tokens is split further by histograms over
//     ranges of c_i, whatever the ties), and the draw goes over all tokens.
//
// What bounds it: the logits are read once from memory; after that a row with a
// top-k is bound by latency (barriers of the cluster, about 0.5 us each), and a
// row whose weights are all needed by their instructions.
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
constexpr int kUnroll = 1;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024, kList = kThreads, kShort = 2048;
constexpr float kOrders = 46.f;
constexpr int kMaxCluster = 8, kMaxVocab = 262144;
// Tokens per CTA: few rows are spread as thin as kSliceLeast, many rows take as
// few CTAs as hold them with two CTAs per SM.
constexpr int kSliceMost = 16384, kSliceLeast = 2048;
constexpr float kOne = 8796093022208.f;  // weight of the highest logit, 2^43

struct SampleArgs {
  const void *logits;
  int64_t ld;
  int vocab, slice;  // slice: tokens per CTA, a multiple of 64
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *token;
  float *logp;
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

// Two fp32 numbers in one instruction.
struct F2 {
  u64 v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 operator-(F2 a, F2 b) { return fma2(b, f2(-1.f), a); }

// 2^-y for 0 <= y = yh + yl < 64 as (wh + wl) 2^-e, to about 2^-42; wh in (0.49,
// 1.01).  Two at a time.
struct Pow2 {
  F2 wh, wl;
  int e0, e1;
};
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it leaves an integer in the low bits
constexpr int kMagicBits = 0x4B400000;
__device__ __forceinline__ int magic_int(float x) { return __float_as_int(x) - kMagicBits; }
__device__ __forceinline__ Pow2 pow_of(const float2 *table, F2 yh, F2 yl) {
  // y = n / 256 + r, |r| <= 1/512 and a little
  const F2 nm = fma2(yh, f2(256.f), f2(kMagic)), nf = nm + f2(-kMagic);
  const float2 nn = parts(nm);
  const int n0 = magic_int(nn.x), n1 = magic_int(nn.y);
  const F2 r0 = fma2(nf, f2(-1.f / 256.f), yh), r = r0 + yl, rl = yl - (r - r0);
  // 2^-r - 1 = z + z^2/2 + ... as eh + el, z = -r ln 2
  constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.904654300e-9f;
  const F2 zh = r * f2(-kLn2h);
  const F2 zl = fma2(r, f2(-kLn2h), zh * f2(-1.f)) + fma2(r, f2(-kLn2l), rl * f2(-kLn2h));
  const F2 q = zh * zh * fma2(zh, fma2(zh, f2(1.f / 24.f), f2(1.f / 6.f)), f2(0.5f));
  const F2 eh = zh + q, el = (q - (eh - zh)) + zl;
  // 2^-(n mod 256)/256 (1 + eh + el)
  const float2 p0 = table[n0 & 255], p1 = table[n1 & 255];
  const F2 px = f2(p0.x, p1.x), py = f2(p0.y, p1.y);
  const F2 ph = px * eh, wh = px + ph;
  const F2 wl = (ph - (wh - px)) + (fma2(px, eh, ph * f2(-1.f)) + fma2(px, el, fma2(py, eh, py)));
  return {wh, wl, n0 >> 8, n1 >> 8};
}

// rint(2^43 exp((x - max) / temperature)) of two logits, to about 2^-42 relative.
__device__ __forceinline__ void weights(const Scale &s, float x0, float x1, u64 &w0, u64 &w1) {
  // d = (max - x) / 2 as dh + dl, exactly
  const F2 half = f2(s.half), b = f2(x0, x1) * f2(-0.5f);
  const F2 d = half + b;
  const float2 dd = parts(d);
  // 0 below 2^-46 (and for -infinity, for which the rest would be NaN)
  const bool in0 = dd.x * s.ch < kOrders, in1 = dd.y * s.ch < kOrders;
  if (!in0 && !in1) {
    w0 = w1 = 0;
    return;
  }
  const F2 dh = f2(in0 ? dd.x : 0.f, in1 ? dd.y : 0.f), c = f2(s.ch);
  const F2 bs = f2(in0 ? -0.5f * x0 : -s.half, in1 ? -0.5f * x1 : -s.half), bb = dh - half;
  const F2 dl = (half - (dh - bb)) + (bs - bb);
  // y = d c in binary orders, as yh + yl
  const F2 yh = dh * c;
  const F2 yl = fma2(dl, c, fma2(dh, f2(s.cl), fma2(dh, c, yh * f2(-1.f))));
  const Pow2 p = pow_of(s.pow, yh, yl);
  // 2^43 2^-e (wh + wl) = 2^22 (i1 + f), i1 an integer below 2^22, |f| <= 9/16
  const F2 scale = f2(__int_as_float((148 - p.e0) << 23), __int_as_float((148 - p.e1) << 23));  // 2^(21-e)
  const F2 am = fma2(p.wh, scale, f2(kMagic)), ai = am + f2(-kMagic);
  const F2 f = fma2(p.wl, scale, fma2(p.wh, scale, ai * f2(-1.f)));
  const F2 fm = fma2(f, f2(4194304.f), f2(kMagic));
  const float2 i1 = parts(am), i2 = parts(fm);
  w0 = in0 ? (u64)((int64_t)magic_int(i1.x) * 4194304 + magic_int(i2.x)) : 0;
  w1 = in1 ? (u64)((int64_t)magic_int(i1.y) * 4194304 + magic_int(i2.y)) : 0;
}
__device__ __forceinline__ u64 weight(const Scale &s, float x) {
  u64 w0, w1;
  weights(s, x, x, w0, w1);
  return w0;
}

// ln(w / total) for 0 < w <= total, rounded once but for about 2^-40: y0 from
// fp32, then y0 + (w - total e^y0) / w, e^y0 in fp32 pairs and the difference in
// fp64 (a 64-bit division and logarithm cost 2 us here).
__device__ __forceinline__ float log_share(const float2 *table, u64 w, u64 total) {
  if (w == total) return 0.f;
  const float y0 = fminf(logf((float)w / (float)total), 0.f);
  constexpr float kLog2eh = 1.44269502162933349609375f, kLog2el = 1.925962991e-8f;
  const float yh = -y0 * kLog2eh, yl = fmaf(-y0, kLog2eh, -yh) - y0 * kLog2el;
  const Pow2 p = pow_of(table, f2(yh), f2(yl));
  const float f = __int_as_float((127 - p.e0) << 23);  // 2^-e
  const double t = (double)total;
  const double d = fma(-t, (double)(parts(p.wl).x * f), fma(-t, (double)(parts(p.wh).x * f), (double)w));
  return y0 + (float)d / (float)w;
}

// Bin of a token: 0 for the largest, kBins and above for those of weight 0 (and
// for -infinity).  Not increasing in x.
__device__ __forceinline__ int bin_of(const Scale &s, float x) {
  const float t = fmaf(-0.5f, x, s.half) * s.cb;
  return t < (float)kBins ? (int)t : kBins;
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

// All threads of the cluster.  The barrier's instruction wants whole warps.
__device__ __forceinline__ void sync_cluster() {
  __syncwarp();
  cluster_sync();
}

struct Hist {  // counts and weights of all bins, over the cluster
  uint32_t count[kBins];
  u64 weight[kBins];
};
struct __align__(16) Shared {
  Hist top;
  union {
    Hist split;
    u64 short_list[kShort];  // in the cluster's first CTA
  };
  // One use after the other, a cluster barrier between: the CTA's own sums (the
  // weights in three parts of 16 bits or less, so that 32768 tokens add up in 32
  // bits with the native atomics), then the lists, or the short list's weights.
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
  u64 part[2][kWarps];
  u64 found[4];   // bin, count before, weight before, count in it
  u64 cut, kept_weight, total;
  float high;
  uint32_t listed, counts[kMaxCluster];
  uint32_t best;  // the first token of the highest logit; in the draw, the warp of the target
};

struct Ctx {
  Shared &s;
  const SampleArgs &a;
  const float *x;       // this CTA's tokens
  int n, base;          // how many, and the index of the first
  uint32_t rank, ranks;
  Scale sc;

  __device__ u64 comp(int i, float v) const { return (u64)key_of(v) << 32 | (uint32_t)~(base + i); }

  // Fill h with the cluster's histogram of bin(i, x_i) (bins >= kBins: none).
  template <typename F>
  __device__ void histogram(Hist &h, bool with_weights, F bin) {
    const int tid = threadIdx.x;
    uint32_t *zero = reinterpret_cast<uint32_t *>(&s.own);
    for (int i = tid; i < (int)(sizeof(s.own) / 4); i += kThreads) zero[i] = 0;
    __syncthreads();
    for (int i = 2 * tid; i < n; i += 2 * kThreads) {
      const float2 v = *reinterpret_cast<const float2 *>(x + i);
      const int b0 = bin(i, v.x), b1 = bin(i + 1, v.y);
      if (b0 >= kBins && b1 >= kBins) continue;
      u64 w0 = 0, w1 = 0;
      if (with_weights) weights(sc, v.x, v.y, w0, w1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = j ? b1 : b0;
        const u64 w = j ? w1 : w0;
        if (b >= kBins) continue;
        atomicAdd(&s.own.count[b], 1u);
        if (with_weights) {
          atomicAdd(&s.own.w[0][b], (uint32_t)w & 0xffffu);
          atomicAdd(&s.own.w[1][b], (uint32_t)(w >> 16) & 0xffffu);
          atomicAdd(&s.own.w[2][b], (uint32_t)(w >> 32));
        }
      }
    }
    sync_cluster();
    // every CTA sums all CTAs' bins itself, 4 bins per thread: cheaper than a
    // second barrier
    if (tid < kBins / 4) {
      uint32_t c[4] = {};
      u64 w[4] = {};
#pragma unroll 4
      for (uint32_t p = 0; p < ranks; ++p) {
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
      for (int j = 0; j < 4; ++j) h.count[tid * 4 + j] = c[j], h.weight[tid * 4 + j] = w[j];
    }
    __syncthreads();
  }

  // The bin in which the sum of counts (or weights), from c0 and w0 on, first
  // reaches `want`: found[] = bin, count and weight before it, its count.
  // False if the sum stays below.
  __device__ bool find(const Hist &h, bool by_weight, u64 want, u64 c0, u64 w0) {
    constexpr int PER = kBins / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    u64 c = 0, w = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) c += h.count[tid * PER + j], w += h.weight[tid * PER + j];
    u64 ci = c, wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 cu = __shfl_up_sync(0xffffffffu, ci, o), wu = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) ci += cu, wi += wu;
    }
    if (lane == 31) s.part[0][warp] = ci, s.part[1][warp] = wi;
    if (tid == 0) s.found[0] = kBins;
    __syncthreads();
    ci += c0 - c, wi += w0 - w;  // before this thread's bins
    for (int v = 0; v < warp; ++v) ci += s.part[0][v], wi += s.part[1][v];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const u64 hc = h.count[tid * PER + j], hw = h.weight[tid * PER + j];
      const u64 from = by_weight ? wi : ci, to = from + (by_weight ? hw : hc);
      if (from < want && to >= want) s.found[0] = tid * PER + j, s.found[1] = ci, s.found[2] = wi, s.found[3] = hc;
      ci += hc, wi += hw;
    }
    __syncthreads();
    return s.found[0] < kBins;
  }

  // The smallest key kept when a token is kept if the sum of counts (or
  // weights) of those before it is less than `want` > 0; 0 if all are.
  // s.kept_weight: the weight of the kept ones (0 unless h has weights).
  __device__ u64 select(bool by_weight, u64 want, bool with_weights) {
    const int tid = threadIdx.x;
    if (!find(s.top, by_weight, want, 0, 0)) return 0;
    int b = (int)s.found[0];
    u64 c0 = s.found[1], w0 = s.found[2];
    u64 count = s.found[3];
    u64 lo = 0, hi = ~0ull;  // the range of keys in question; all of bin b at first
    bool by_bin = true;
    while (count > kList) {
      if (by_bin) {
        // keys of bin b: bins do not increase with the key
        const auto least = [&](int most) {  // smallest key of a bin <= most
          uint32_t l = 0, r = key_of(sc.high);
          while (l < r) {
            const uint32_t m = l + (r - l) / 2;
            if (bin_of(sc, of_key(m)) <= most) r = m;
            else l = m + 1;
          }
          return l;
        };
        lo = (u64)least(b) << 32;
        hi = b ? ((u64)least(b - 1) << 32) - 1 : (u64)key_of(sc.high) << 32 | 0xffffffffu;
        by_bin = false;
      }
      const u64 range = hi - lo;
      const int bits = 64 - __clzll((long long)range);
      const int shift = bits > 10 ? bits - 10 : 0;
      sync_cluster();  // the lists or sums that shared this memory are read
      histogram(s.split, with_weights, [&](int i, float v) {
        const u64 k = comp(i, v);
        return k >= lo && k <= hi ? (int)((hi - k) >> shift) : kBins;
      });
      if (!find(s.split, by_weight, want, c0, w0)) return 0;  // cannot be: the sum reaches it in this range
      b = (int)s.found[0], c0 = s.found[1], w0 = s.found[2], count = s.found[3];
      hi = hi - ((u64)b << shift);
      const u64 width = (1ull << shift) - 1;
      lo = hi - lo > width ? hi - width : lo;
    }
    // list the tokens of the bin: each CTA its own, then all of them everywhere
    sync_cluster();  // the sums that shared this memory, and earlier lists, are read
    if (tid == 0) s.listed = 0, s.cut = ~0ull, s.kept_weight = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const float v = x[i];
      bool in;
      if (by_bin) {
        in = bin_of(sc, v) == b;
      } else {
        const u64 k = comp(i, v);
        in = k >= lo && k <= hi;
      }
      if (in) s.list.mine[atomicAdd(&s.listed, 1u)] = comp(i, v);
    }
    sync_cluster();
    if (tid < (int)ranks) s.counts[tid] = ld_peer32(&s.listed, tid);
    __syncthreads();
    const uint32_t at = (uint32_t)count;
    if (tid < (int)at) {
      uint32_t p = 0, i = tid;
      while (p + 1 < ranks && i >= s.counts[p]) i -= s.counts[p++];
      const u64 k = ld_peer64(&s.list.mine[min(i, (uint32_t)kList - 1)], p);
      s.list.all[tid] = k;
      s.list.weights[tid] = with_weights ? weight(sc, of_key((uint32_t)(k >> 32))) : 0;
    }
    __syncthreads();
    if (tid < (int)at) {
      const u64 k = s.list.all[tid];
      u64 before = by_weight ? w0 : c0;
      for (uint32_t j = 0; j < at; ++j)
        if (s.list.all[j] > k) before += by_weight ? s.list.weights[j] : 1;
      if (before < want) {
        atomicMin(&s.cut, k);
        if (with_weights) atomicAdd(&s.kept_weight, s.list.weights[tid]);
      }
    }
    __syncthreads();
    if (tid == 0) s.kept_weight += w0;
    __syncthreads();
    return s.cut;
  }
};

// Sort key[0..size) descending, size a power of two up to kShort.
__device__ void sort_down(u64 *key, int size) {
  const int tid = threadIdx.x;
  const bool one = size <= 64;  // one warp's pairs
  if (!one || tid < 32) {
    for (int k = 2; k <= size; k *= 2)
      for (int j = k / 2; j; j /= 2) {
        for (int i = tid; i < size / 2; i += kThreads) {
          const int lo = (i & ~(j - 1)) * 2 | (i & (j - 1)), hi = lo | j;
          const u64 a = key[lo], b = key[hi];
          if ((a < b) == ((lo & k) == 0)) key[lo] = b, key[hi] = a;
        }
        if (one) __syncwarp();
        else __syncthreads();
      }
  }
  __syncthreads();
}

// Sum over the block of the values before this thread's, and of all.
__device__ u64 scan_block(u64 *part, u64 v, u64 &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();  // earlier uses of part
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  u64 w = lane < kWarps ? part[lane] : 0;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const u64 u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, kWarps - 1);
  const u64 prev = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  return (warp ? prev : 0) + incl - v;
}

template <typename T>
__device__ __forceinline__ float widen(T v) {
  const float f = (float)v;
  return f == f ? f : -INFINITY;  // NaN is never chosen
}

__device__ __forceinline__ u64 share_of(float part, u64 total) {  // floor(part * total), part in [0, 1]
  return (u64)((double)part * (double)total);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared &s = *reinterpret_cast<Shared *>(raw);
  float *x = reinterpret_cast<float *>(raw + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.y;
  const int row = blockIdx.x;
  const int base = (int)rank * a.slice, n = a.slice, live = max(0, min(a.vocab - base, n));
  const T *in = static_cast<const T *>(a.logits) + row * a.ld + base;
  const float t = a.temperature ? a.temperature[row] : 1.f;
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.f;
  const float u = fminf(fmaxf(a.u[row], 0.f), 1.f);

  // ---- the row's slice into shared memory, and its maximum
  float high = -INFINITY;
  constexpr int V = 16 / sizeof(T);
  if ((reinterpret_cast<uintptr_t>(in) & 15) == 0) {
    const int full = live / V;
    constexpr int U = 4;
    for (int i = tid; i < full; i += U * kThreads) {
      uint4 w[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i + j * kThreads < full) w[j] = reinterpret_cast<const uint4 *>(in)[i + j * kThreads];
#pragma unroll
      for (int l = 0; l < U; ++l) {
        if (i + l * kThreads >= full) continue;
        const T *e = reinterpret_cast<const T *>(&w[l]);
        float4 *to = reinterpret_cast<float4 *>(x + (i + l * kThreads) * V);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
          const float4 f = make_float4(widen(e[4 * j]), widen(e[4 * j + 1]), widen(e[4 * j + 2]), widen(e[4 * j + 3]));
          to[j] = f;
          high = fmaxf(fmaxf(high, fmaxf(f.x, f.y)), fmaxf(f.z, f.w));
        }
      }
    }
    for (int i = full * V + tid; i < live; i += kThreads) high = fmaxf(high, x[i] = widen(in[i]));
  } else {
    for (int i = tid; i < live; i += kThreads) high = fmaxf(high, x[i] = widen(in[i]));
  }
  for (int i = live + tid; i < n; i += kThreads) x[i] = -INFINITY;
  for (int i = tid; i < 256; i += kThreads) s.pow[i] = make_float2(kPow.hi[i], kPow.lo[i]);
  if (tid == 0) s.listed = 0, s.best = 0xffffffffu;
#pragma unroll
  for (int o = 16; o; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
  if (lane == 0) s.part[0][warp] = __float_as_uint(high);
  __syncthreads();
  if (tid < 32) {
    high = lane < kWarps ? __uint_as_float((uint32_t)s.part[0][lane]) : -INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
    if (lane == 0) s.high = high;
  }
  sync_cluster();
  high = __uint_as_float(ld_peer32(&s.high, lane & (ranks - 1)));  // ranks is a power of two
#pragma unroll
  for (int o = kMaxCluster / 2; o; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));

  const bool none = high == -INFINITY;
  if (none || !(t > 0.f)) {
    // the first token of the highest logit, sent to the first CTA
    uint32_t best = 0xffffffffu;
    for (int i = tid; i < n; i += kThreads)
      if (x[i] == high) best = min(best, (uint32_t)(base + i));
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
    for (int i = tid; i < n; i += kThreads) x[i] = x[i] == high ? 0.f : -INFINITY;
    high = 0.f;
    __syncthreads();
  }
  // c = 2 log2(e) / t as two fp32 numbers (a temperature so small that it is
  // not finite separates all logits that differ all the same)
  constexpr float kLh = 2.8853900432586669922f, kLl = 3.851925982e-8f;
  const float ch = fminf(kLh / t, 3e38f);
  const float cl = ch > 0.f && ch < 3e38f ? (fmaf(-ch, t, kLh) + kLl) / t : 0.f;
  Ctx c = {s, a, x, n, base, rank, ranks, {high, 0.5f * high, ch, cl, ch * (kBins / kOrders), s.pow}};
  if (!(c.sc.cb < 3e38f)) c.sc.cb = 3e38f;
  // min-p: e_i >= min_p, as weights
  const u64 least = mp > 0.f ? max(1ull, (u64)ceilf(fminf(mp, 1.f) * kOne)) : 0;

  // ---- the filters, each as the smallest key it keeps
  u64 cut = 0;
  const bool use_k = k > 0 && k < a.vocab, use_p = p < 1.f;
  if (use_k || use_p) {
    const auto bins = [&](int, float v) { return bin_of(c.sc, v); };
    u64 total = 0;
    c.histogram(s.top, !use_k, bins);
    if (!use_k) {
      u64 w = 0;
      for (int b = tid; b < kBins; b += kThreads) w += s.top.weight[b];
      scan_block(s.part[0], w, total);
      __syncthreads();
    }
    // before < top_p * total, and at least the first token: before < want
    u64 want = use_k ? (u64)k : max(1ull, (u64)ceil((double)fmaxf(p, 0.f) * (double)total));
    const bool reached = c.find(s.top, !use_k, want, 0, 0);
    int b = reached ? (int)s.found[0] : kBins - 1;
    u64 count = reached ? s.found[1] + s.found[3] : 0;
    if (!reached) {  // fewer than k tokens of any weight: all of them
      u64 m = 0;
      for (int i = tid; i < kBins; i += kThreads) m += s.top.count[i];
      scan_block(s.part[0], m, count);
    }
    if (count <= kShort) {
      for (int i = tid; i < n; i += kThreads) {
        const float v = x[i];
        if (bin_of(c.sc, v) <= b) st_peer64(&s.short_list[add_peer32(&s.listed, 0, 1)], 0, c.comp(i, v));
      }
      sync_cluster();
      if (rank != 0) return;
      constexpr int PER = kShort / kThreads;  // tokens per thread, in order
      const int m = (int)count;
      int size = 2;
      while (size < m) size *= 2;
      for (int i = m + tid; i < size; i += kThreads) s.short_list[i] = 0;
      __syncthreads();
      sort_down(s.short_list, size);
      const int kept_k = use_k ? min(m, k) : m;
      u64 w[PER], key[PER], sum = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int i = PER * tid + j;
        key[j] = i < kept_k ? s.short_list[i] : 0;
        w[j] = i < kept_k ? weight(c.sc, of_key((uint32_t)(key[j] >> 32))) : 0;
        sum += w[j];
      }
      u64 all, before = scan_block(s.part[0], sum, all);
      if (use_p && use_k) want = max(1ull, (u64)ceil((double)fmaxf(p, 0.f) * (double)all));
      int mine = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const u64 e = w[j];
        if ((use_p && before >= want) || e < least) w[j] = 0;
        before += e;
        mine += w[j] != 0;
      }
      u64 kept;  // the first `kept` of the order
      scan_block(s.part[1], mine, kept);
      size = 2;
      while (size < (int)kept) size *= 2;
      // by index: ~i high, the place in the order low
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int i = PER * tid + j;
        if (i < size) {
          s.short_weight[i] = w[j];
          s.short_list[i] = w[j] ? key[j] << 32 | (uint32_t)i : 0;
        }
      }
      __syncthreads();
      sort_down(s.short_list, size);
      sum = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int i = PER * tid + j;
        key[j] = i < (int)kept ? s.short_list[i] : 0;
        w[j] = i < (int)kept ? s.short_weight[(uint32_t)key[j]] : 0;
        sum += w[j];
      }
      before = scan_block(s.part[0], sum, all);
      u64 target = share_of(u, all);
      if (target >= all) target = all - 1;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (before <= target && target < before + w[j]) {
          a.token[row] = (int32_t)~(uint32_t)(key[j] >> 32);
          if (a.logp) a.logp[row] = log_share(s.pow, w[j], all);
        }
        before += w[j];
      }
      return;
    }
    if (use_k && use_p) {
      sync_cluster();  // the sums are read
      c.histogram(s.top, true, bins);
    }
    if (use_k) {
      cut = c.select(false, (u64)k, use_p);
      if (use_p) {
        if (cut) {
          total = s.kept_weight;
        } else {  // the top-k set is everything of any weight
          u64 w = 0;
          for (int i = tid; i < kBins; i += kThreads) w += s.top.weight[i];
          scan_block(s.part[0], w, total);
        }
        want = max(1ull, (u64)ceil((double)fmaxf(p, 0.f) * (double)total));
        __syncthreads();
      }
    }
    if (use_p) cut = max(cut, c.select(true, want, true));
  }

  // ---- the draw.  A warp's tokens are contiguous, so the order of the sums is
  // that of the indexes.
  const int run = (n + 2 * kThreads - 1) / (2 * kThreads) * 64, i0 = min(n, warp * run), i1 = min(n, i0 + run);
  const auto kept = [&](int i) -> u64 {  // of tokens i and i + 1, i even
    const float2 v = *reinterpret_cast<const float2 *>(x + i);
    u64 w0, w1;
    weights(c.sc, v.x, v.y, w0, w1);
    if (w0 < least || c.comp(i, v.x) < cut) w0 = 0;
    if (w1 < least || c.comp(i + 1, v.y) < cut) w1 = 0;
    return w0 + w1;
  };
  u64 sum = 0;
  if (cut == 0 && least == 0) {
#pragma unroll kUnroll
    for (int i = i0 + 2 * lane; i < i1; i += 64) {
      const float2 v = *reinterpret_cast<const float2 *>(x + i);
      u64 w0, w1;
      weights(c.sc, v.x, v.y, w0, w1);
      sum += w0 + w1;
    }
  } else {
    for (int i = i0 + 2 * lane; i < i1; i += 64) sum += kept(i);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  u64 mine, before = scan_block(s.part[0], lane == 0 ? sum : 0, mine);
  before = __shfl_sync(0xffffffffu, before, 0);  // before this warp's tokens
  if (tid == 0) s.total = mine;
  sync_cluster();
  u64 total = ld_peer64(&s.total, lane & (ranks - 1));
  {
    u64 less = lane < (int)rank ? total : 0;
    total = lane < (int)ranks ? total : 0;
#pragma unroll
    for (int o = kMaxCluster / 2; o; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      less += __shfl_xor_sync(0xffffffffu, less, o);
    }
    total = __shfl_sync(0xffffffffu, total, 0);
    before += __shfl_sync(0xffffffffu, less, 0);
  }
  sync_cluster();  // all totals are read: from here on the CTAs are on their own
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
  for (int i = j0; i < j1; i += 2) own += kept(i);
  u64 at = s.cut + scan_block(s.part[1], own, mine);
  if (at <= target && target < at + own) {
    for (int i = j0; i < j1; ++i) {
      const u64 e = weight(c.sc, x[i]), w = e < least || c.comp(i, x[i]) < cut ? 0 : e;
      at += w;
      if (at > target) {
        a.token[row] = base + i;
        if (a.logp) a.logp[row] = log_share(s.pow, w, total);
        break;
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const SampleArgs &a, int64_t rows, int ranks, cudaStream_t stream) {
  static bool ready[kMaxDevices];  // the attribute is per device
  const int dev = device_facts()->device;
  if (!ready[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(Shared) + kMaxVocab / kMaxCluster * 4);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows, ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared) + (size_t)a.slice * 4;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = ranks;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
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
  const SampleArgs a = {logits, ld, (int)vocab, slice, u, temperature, top_p, min_p, top_k, token, logp};
  return dtype == Q4K_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, rows, ranks, stream) : launch_t<float>(a, rows, ranks, stream);
}

}  // namespace q4k
