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
// integer rint(2^44 e_i), computed in pairs of fp32 numbers to about 2^-42 (fp64
// has 1/64 of the fp32 rate here and would take over a millisecond for 256 rows
// of 131072).  Integer sums are exact, the same in any order; 2^18 tokens sum
// below 2^62.
//
// Order.  Every filter keeps a prefix of the tokens in the order (logit
// descending, index ascending).  With c_i = (monotone integer image of x_i) <<
// 32 | ~i that order is the descending one of distinct integers, a filter is the
// smallest c_i kept, and the kept set is c_i >= the largest of these.
//
// Selection.  A histogram over (max - x) in kBins equal steps of the 46 binary
// orders in which weights are not 0, with the count and the exact weight of
// each bin, gives the bin in which the k-th token lies, or in which the
// cumulative weight reaches top_p of the total.  The bin's tokens are listed
// and ranked by comparing all pairs.  A bin of more than kList tokens is first
// split further, by histograms over ranges of c_i, whatever the ties.
//
// What bounds it: the logits are read once from memory (a cluster of up to 8
// CTAs holds a row in its shared memory, all passes run from there), then the
// instructions of the weights, about 60 per token and pass that needs them.
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
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024, kList = 512;
constexpr float kOrders = 46.f;
constexpr int kMaxCluster = 8, kMaxVocab = 262144;
constexpr u64 kOne = 1ull << 44;

struct SampleArgs {
  const void *logits;
  int64_t ld;
  int vocab, slice;  // slice: tokens per CTA, a multiple of 32
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

// rint(2^44 exp((x - max) / temperature)) to about 2^-42 relative.
__device__ __forceinline__ u64 weight(const Scale &s, float x) {
  if (x == s.high) return kOne;
  // d = (max - x) / 2 as dh + dl, exactly
  const float b = -0.5f * x, dh = s.half + b, bb = dh - s.half;
  if (!(dh * s.ch < kOrders)) return 0;  // also -infinity, and all but the largest where that is +infinity
  const float dl = (s.half - (dh - bb)) + (b - bb);
  // y = d c in binary orders, as yh + yl
  const float yh = dh * s.ch;
  const float yl = fmaf(dl, s.ch, fmaf(dh, s.cl, fmaf(dh, s.ch, -yh)));
  // y = n / 256 + r, |r| <= 1/512 and a little
  // (conversions by adding 1.5 * 2^23, which leaves an integer in the low bits:
  // the conversion instructions run at a quarter of this rate or less)
  constexpr float kMagic = 12582912.f;
  const float nm = fmaf(yh, 256.f, kMagic), nf = nm - kMagic;
  const int n = __float_as_int(nm) - 0x4B400000;
  const float r0 = fmaf(nf, -1.f / 256.f, yh), r = r0 + yl, rl = yl - (r - r0);
  // 2^-r - 1 = z + z^2/2 + ... as eh + el, z = -r ln 2
  constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.904654323148236017e-9f;
  const float zh = -r * kLn2h;
  const float zl = fmaf(-r, kLn2h, -zh) - fmaf(r, kLn2l, rl * kLn2h);
  const float q = zh * zh * fmaf(zh, fmaf(zh, 1.f / 24.f, 1.f / 6.f), 0.5f);
  const float eh = zh + q, el = (q - (eh - zh)) + zl;
  const float2 p = s.pow[n & 255];
  // 2^-(n mod 256)/256 (1 + eh + el) as wh + wl
  const float ph = p.x * eh;
  const float wh = p.x + ph;
  const float wl = (ph - (wh - p.x)) + (fmaf(p.x, eh, -ph) + fmaf(p.x, el, fmaf(p.y, eh, p.y)));
  // wh in (0.49, 1.01) is its 24-bit mantissa times 2^-25, 2^-24 or 2^-23
  const uint32_t bits = __float_as_uint(wh);
  const uint32_t wi = ((bits & 0x7fffffu) | 0x800000u) << ((bits >> 23) - 125);
  const int64_t m = ((int64_t)wi << 19) + (__float_as_int(fmaf(wl, 17592186044416.f, kMagic)) - 0x4B400000);
  const int e = n >> 8;
  return (u64)(e ? (m + (1ll << (e - 1))) >> e : m);
}

// Bin of a token: 0 for the largest, kBins and above for those of weight 0.
// Not increasing in x.
__device__ __forceinline__ int bin_of(const Scale &s, float x) {
  if (x == s.high) return 0;
  const float t = (s.half + -0.5f * x) * s.cb;
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
  Hist top, split;
  // One use after the other, a cluster barrier between: the CTA's own sums (the
  // weights in three parts of 16 bits or less, so that 32768 tokens add up in 32
  // bits with the native atomics), then the lists.
  union {
    struct {
      uint32_t count[kBins], w[3][kBins];
    } own;
    struct {
      u64 mine[kList], all[kList], weights[kList];
    } list;
  };
  float2 pow[256];
  u64 part[2][kWarps];
  u64 found[4];   // bin, count before, weight before, count in it
  u64 cut, kept_weight, total;
  float high;
  uint32_t listed;
  double c, log_min_p;
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
  __device__ void histogram(Hist &h, bool weights, F bin) {
    const int tid = threadIdx.x;
    uint32_t *zero = reinterpret_cast<uint32_t *>(&s.own);
    for (int i = tid; i < (int)(sizeof(s.own) / 4); i += kThreads) zero[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const float v = x[i];
      const int b = bin(i, v);
      if (b >= kBins) continue;
      atomicAdd(&s.own.count[b], 1u);
      if (weights) {
        const u64 w = weight(sc, v);
        atomicAdd(&s.own.w[0][b], (uint32_t)w & 0xffffu);
        atomicAdd(&s.own.w[1][b], (uint32_t)(w >> 16) & 0xffffu);
        atomicAdd(&s.own.w[2][b], (uint32_t)(w >> 32));
      }
    }
    sync_cluster();
    // CTA r sums bins [r, r + 1) * kBins / ranks of all CTAs, then all exchange
    const int share = kBins / ranks, first = rank * share;
    for (int b = first + tid; b < first + share; b += kThreads) {
      uint32_t c = 0;
      u64 w = 0;
      for (uint32_t p = 0; p < ranks; ++p) {
        c += ld_peer32(&s.own.count[b], p);
        if (weights)
          w += ld_peer32(&s.own.w[0][b], p) + ((u64)ld_peer32(&s.own.w[1][b], p) << 16) +
               ((u64)ld_peer32(&s.own.w[2][b], p) << 32);
      }
      h.count[b] = c;
      h.weight[b] = w;
    }
    sync_cluster();
    for (int b = tid; b < kBins; b += kThreads)
      if ((uint32_t)(b / share) != rank) {
        h.count[b] = ld_peer32(&h.count[b], b / share);
        if (weights) h.weight[b] = ld_peer64(&h.weight[b], b / share);
      }
    if (!weights) {
      for (int b = tid; b < kBins; b += kThreads) h.weight[b] = 0;
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
  __device__ u64 select(bool by_weight, u64 want, bool weights) {
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
      histogram(s.split, weights, [&](int i, float v) {
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
    uint32_t at = 0;
    for (uint32_t p = 0; p < ranks; ++p) {
      const uint32_t m = ld_peer32(&s.listed, p);
      for (uint32_t i = tid; i < m && at + i < kList; i += kThreads) {
        const u64 k = ld_peer64(&s.list.mine[i], p);
        s.list.all[at + i] = k;
        s.list.weights[at + i] = weights ? weight(sc, of_key((uint32_t)(k >> 32))) : 0;
      }
      at += m;
    }
    __syncthreads();
    if (tid < (int)at && tid < kList) {
      const u64 k = s.list.all[tid];
      u64 before = by_weight ? w0 : c0;
      for (uint32_t j = 0; j < at; ++j)
        if (s.list.all[j] > k) before += by_weight ? s.list.weights[j] : 1;
      if (before < want) {
        atomicMin(&s.cut, k);
        if (weights) atomicAdd(&s.kept_weight, s.list.weights[tid]);
      }
    }
    __syncthreads();
    if (tid == 0) s.kept_weight += w0;
    __syncthreads();
    return s.cut;
  }
};

template <typename T>
__device__ __forceinline__ float widen(T v) {
  const float f = (float)v;
  return f == f ? f : -INFINITY;  // NaN is never chosen
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared &s = *reinterpret_cast<Shared *>(raw);
  float *x = reinterpret_cast<float *>(raw + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank(), ranks = gridDim.y;
  const int row = blockIdx.x;
  const int base = (int)rank * a.slice, n = max(0, min(a.vocab - base, a.slice));
  const T *in = static_cast<const T *>(a.logits) + row * a.ld + base;
  const float t = a.temperature ? a.temperature[row] : 1.f;
  const float mp = a.min_p ? a.min_p[row] : 0.f;

  // ---- the row's slice into shared memory, and its maximum
  float high = -INFINITY;
  constexpr int V = 16 / sizeof(T);
  if ((reinterpret_cast<uintptr_t>(in) & 15) == 0) {
    const int full = n / V;
    constexpr int U = 4;
    for (int i = tid; i < full; i += U * kThreads) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kThreads < full) w[u] = reinterpret_cast<const uint4 *>(in)[i + u * kThreads];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u * kThreads >= full) continue;
        const T *e = reinterpret_cast<const T *>(&w[u]);
        float4 *to = reinterpret_cast<float4 *>(x + (i + u * kThreads) * V);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
          const float4 f = make_float4(widen(e[4 * j]), widen(e[4 * j + 1]), widen(e[4 * j + 2]), widen(e[4 * j + 3]));
          to[j] = f;
          high = fmaxf(fmaxf(high, fmaxf(f.x, f.y)), fmaxf(f.z, f.w));
        }
      }
    }
    for (int i = full * V + tid; i < n; i += kThreads) high = fmaxf(high, x[i] = widen(in[i]));
  } else {
    for (int i = tid; i < n; i += kThreads) high = fmaxf(high, x[i] = widen(in[i]));
  }
  for (int i = tid; i < 256; i += kThreads) s.pow[i] = make_float2(kPow.hi[i], kPow.lo[i]);
  if (tid == kThreads - 1) {  // in fp64, once per row
    s.c = 2.0 * 1.4426950408889634074 / (double)t;
    s.log_min_p = mp > 0.f ? (double)t * log((double)fminf(mp, 1.f)) : 0.0;
  }
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
  high = -INFINITY;
  for (uint32_t p = 0; p < ranks; ++p) high = fmaxf(high, __uint_as_float(ld_peer32(&s.high, p)));

  const bool none = high == -INFINITY;
  if (none || !(t > 0.f)) {
    // the first token of the highest logit
    uint32_t best = 0xffffffffu;
    for (int i = tid; i < n; i += kThreads)
      if (x[i] == high) best = min(best, (uint32_t)(base + i));
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) s.part[1][warp] = best;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) best = min(best, (uint32_t)s.part[1][w]);
      s.listed = best;
    }
    sync_cluster();
    if (rank == 0 && tid == 0) {
      for (uint32_t p = 0; p < ranks; ++p) best = min(best, ld_peer32(&s.listed, p));
      a.token[row] = none ? -1 : (int32_t)best;
      if (a.logp) a.logp[row] = none ? -INFINITY : 0.f;
    }
    sync_cluster();  // no CTA leaves while its memory is read
    return;
  }

  const float ch = (float)s.c;
  Ctx c = {s, a, x, n, base, rank, ranks, {high, 0.5f * high, ch, (float)(s.c - (double)ch), ch * (kBins / kOrders), s.pow}};
  if (!(fabsf(ch) < INFINITY)) c.sc.cl = 0.f;

  // ---- the filters, each as the smallest key it keeps
  u64 cut = 0;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.f;
  const bool use_k = k > 0 && k < a.vocab, use_p = p < 1.f;
  if (use_k || use_p) {
    c.histogram(s.top, use_p, [&](int, float v) { return bin_of(c.sc, v); });
    u64 total = 0;
    bool whole = true;  // the top-k set is everything of any weight
    if (use_k) {
      cut = c.select(false, (u64)k, use_p);
      whole = cut == 0;
      total = whole ? 0 : s.kept_weight;
    }
    if (use_p) {
      if (whole) {
        u64 w = 0;
        for (int b = tid; b < kBins; b += kThreads) w += s.top.weight[b];
#pragma unroll
        for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        if (lane == 0) s.part[0][warp] = w;
        __syncthreads();
        for (int v = 0; v < kWarps; ++v) total += s.part[0][v];
        __syncthreads();
      }
      // before < top_p * total, and at least the first token: before < want
      const u64 want = max(1ull, (u64)ceil((double)fmaxf(p, 0.f) * (double)total));
      sync_cluster();  // the lists of the first selection are read
      cut = max(cut, c.select(true, want, true));
    }
  }
  if (mp > 0.f) {
    const float least = high == INFINITY ? high : __double2float_ru((double)high + s.log_min_p);
    cut = max(cut, (u64)key_of(least) << 32);
  }

  // ---- the draw.  A warp's tokens are contiguous, 32 at a time, so the order
  // of the sums is that of the indexes.
  const int run = (n + kThreads - 1) / kThreads * 32, i0 = min(n, warp * run), i1 = min(n, i0 + run);
  const auto kept = [&](int i) -> u64 {
    const float v = x[i];
    return c.comp(i, v) >= cut ? weight(c.sc, v) : 0;
  };
  u64 sum = 0;
  for (int i = i0 + lane; i < i1; i += 32) sum += kept(i);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s.part[0][warp] = sum;
  __syncthreads();
  u64 before = 0, mine = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s.part[0][w];
    mine += s.part[0][w];
  }
  if (tid == 0) s.total = mine;
  sync_cluster();
  u64 total = 0;
  for (uint32_t q = 0; q < ranks; ++q) {
    const u64 w = ld_peer64(&s.total, q);
    if (q < rank) before += w;
    total += w;
  }
  // cumulative > u * total, for an integer: cumulative > floor(u * total)
  const float u = fminf(fmaxf(a.u[row], 0.f), 1.f);
  u64 target = (u64)((double)u * (double)total);
  if (target >= total) target = total - 1;
  // The warp whose tokens reach the target tells the block, which goes through
  // them again together (one warp alone took 6 us for its 1024).
  if (tid == 0) s.listed = 0xffffffffu;
  __syncthreads();
  if (lane == 0 && before <= target && target < before + sum) s.listed = warp, s.cut = before;
  __syncthreads();
  if (s.listed != 0xffffffffu) {
    const int from = min(n, (int)s.listed * run), to = min(n, from + run);
    const int per = (run + kThreads - 1) / kThreads, j0 = min(to, from + tid * per), j1 = min(to, j0 + per);
    u64 own = 0;
    for (int i = j0; i < j1; ++i) own += kept(i);
    u64 incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s.part[1][warp] = incl;
    __syncthreads();
    u64 at = s.cut + incl - own;
    for (int w = 0; w < warp; ++w) at += s.part[1][w];
    if (at <= target && target < at + own) {
      for (int i = j0; i < j1; ++i) {
        const u64 w = kept(i);
        at += w;
        if (at > target) {
          a.token[row] = base + i;
          if (a.logp) a.logp[row] = (float)log((double)w / (double)total);
          break;
        }
      }
    }
  }
  sync_cluster();  // no CTA leaves while its memory is read
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
  // A CTA's slice is at least 4096 tokens; 8 CTAs hold the largest row.
  int ranks = 1;
  while (ranks < kMaxCluster && vocab > ranks * 4096) ranks *= 2;
  const int slice = (int)((vocab + ranks - 1) / ranks + 31) / 32 * 32;
  const SampleArgs a = {logits, ld, (int)vocab, slice, u, temperature, top_p, min_p, top_k, token, logp};
  return dtype == Q4K_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, rows, ranks, stream) : launch_t<float>(a, rows, ranks, stream);
}

}  // namespace q4k
