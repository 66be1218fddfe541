// q4k_rope.cu -- norm of each head and rotation by position (q4k_rope), the same
// with the write of new keys and values into the paged cache
// (q4k_rope_kv_write), and the table of frequencies (q4k_rope_steps).
//
// "spec: specialized model runtimes", section "Architecture": norms and
// attention, and what lies between them, are ops of kernel tier T0.
//
// Mathematics.  A head x of D values: y = x gamma / sqrt(mean x^2 + eps) where
// there is a gamma, then of its first R values the pairs (a, b) turn by the
// position's angle t_i = pos f_i:
//   (a, b) -> A (a cos t - b sin t, b cos t + a sin t).
//
// Angles.  At position 10^6 an fp32 product pos f_i is off by 0.06 radians.  So
// f_i comes as f_i / 2 pi in units of 2^-64 of a turn, an integer: its product
// with the position, modulo 2^64, is the fraction of a turn exactly, to the 2^-65
// that the table's rounding leaves times the position.  Its upper 32 bits, signed,
// are the angle in (-1/2, 1/2] turns.
//
// What bounds it: bytes, each read and written once.  A block takes a few tokens,
// whose angles' cosines and sines it computes once, into shared memory (they are
// the same for all heads), while its first rows are on their way; then groups of
// D / 8 lanes take a row each.
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

constexpr int kThreads = 256;

enum Pairs { kHalf = 0, kAdjacent = 1, kAny = 2 };  // kAny: (i, i + R / 2) where R / 2 is no multiple of 4

struct Args {
  RopeArgs r;
  // [0]: queries, [1]: keys and values.  A block takes some tokens and a group of the
  // heads of one kind; the grid runs over those of queries, of keys, of values.
  uint32_t blocks[2];
  int tokens_per_block[2], heads_per_block[2];
  FastDiv groups[2]{FastDiv{1}, FastDiv{1}};
  FastDiv half{1};     // of the rotated values
  FastDiv page{1};
};

// A lane's 8 values of a row, as two times four: where pairs lie half a rotated
// part apart, 4 values of its first half and their partners in the second, so that
// they turn within the lane; else 8 in a row.
template <typename T>
struct Fours;
template <>
struct Fours<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p, int oa, int ob) {
    a = *reinterpret_cast<const float4 *>(p + oa);
    b = *reinterpret_cast<const float4 *>(p + ob);
  }
  __device__ __forceinline__ void to(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Fours<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, int oa, int ob) {
    if (ob == oa + 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p + oa);
      a = make_uint2(v.x, v.y), b = make_uint2(v.z, v.w);
    } else {
      a = *reinterpret_cast<const uint2 *>(p + oa);
      b = *reinterpret_cast<const uint2 *>(p + ob);
    }
  }
  __device__ __forceinline__ void to(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void store_fours(float *p, int oa, int ob, const float (&v)[8]) {
  *reinterpret_cast<float4 *>(p + oa) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + ob) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_fours(__nv_bfloat16 *p, int oa, int ob, const float (&v)[8]) {
  const uint2 a = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])), b = make_uint2(pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  if (ob == oa + 4) {
    *reinterpret_cast<uint4 *>(p + oa) = make_uint4(a.x, a.y, b.x, b.y);
  } else {
    *reinterpret_cast<uint2 *>(p + oa) = a;
    *reinterpret_cast<uint2 *>(p + ob) = b;
  }
}

template <int LPR, typename T, typename TO, int PAIRS, bool CACHE, bool E4M3>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const Args a) {
  extern __shared__ __align__(16) float table[];
  const RopeArgs &r = a.r;
  constexpr int SLOTS = kThreads / LPR, U = 2;  // rows at a time, of the block and of a thread
  const int c = threadIdx.x % LPR, slot_in = threadIdx.x / LPR, lane = threadIdx.x & 31;
  // the block's kind of heads (0: queries, 1: keys, 2: values), which of them, and its tokens
  const uint32_t x0 = blockIdx.x;
  const int kind = !CACHE || x0 < a.blocks[0] ? 0 : x0 < a.blocks[0] + a.blocks[1] ? 1 : 2, kv = kind ? 1 : 0;
  const uint32_t xk = kind == 0 ? x0 : kind == 1 ? x0 - a.blocks[0] : x0 - a.blocks[0] - a.blocks[1];
  const uint32_t part = a.groups[kv].div(xk);
  const int head0 = (int)(xk - part * a.groups[kv].d) * a.heads_per_block[kv], heads = min(a.heads_per_block[kv], r.heads[kv] - head0);
  const int tpb = a.tokens_per_block[kv], tok0 = (int)part * tpb, toks = min(tpb, (int)(r.tokens - tok0));
  const int half = r.rot / 2, stride = (half + 3) & ~3;
  float *cs = table, *sn = table + tpb * stride;
  const unsigned mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (lane / LPR * LPR);
  const bool mine = c * 8 < r.dim;  // lanes past the row's end only take part in sums
  // this lane's values oa .. oa + 3 and ob .. ob + 3; whether they turn, by the angles 4 c ..
  int oa = 8 * c, ob = oa + 4;
  bool turns = oa < r.rot && kind != 2;
  if (PAIRS == kHalf && 4 * c < half) oa = 4 * c, ob = half + 4 * c;
  if (PAIRS == kHalf) turns = 4 * c < half && kind != 2;

  // Rows (token, head) of the block in a list, heads first; a thread takes every SLOTS-th.
  const int step_t = SLOTS / heads, step_h = SLOTS - step_t * heads, rows = toks * heads;
  const int64_t ld_t = r.ld_token[kind], ld_h = r.ld_head[kind];
  int t = slot_in / heads, h = slot_in - t * heads;
  const T *from = static_cast<const T *>(r.in[kind]) + (int64_t)(tok0 + t) * ld_t + (int64_t)(head0 + h) * ld_h;
  const int64_t step = step_t * ld_t + step_h * ld_h, carry = ld_t - heads * ld_h;
  struct Row {
    int t, h;
    bool on;
    const T *from;
    Fours<T> raw;
  } row[U];
  int next = slot_in;  // its place in the list
  const auto fetch = [&](Row &x) {
    x.t = t, x.h = h, x.on = next < rows, x.from = from;
    if (x.on && mine) x.raw.load(from, oa, ob);
    next += SLOTS;
    t += step_t, h += step_h, from += step;
    if (h >= heads) h -= heads, ++t, from += carry;
  };
#pragma unroll
  for (int u = 0; u < U; ++u) row[u].raw = Fours<T>(), fetch(row[u]);

  const float *gamma = kind == 2 ? nullptr : r.gamma[kind];
  float g[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = 1.f;
  if (mine && gamma) {
    const float4 x = *reinterpret_cast<const float4 *>(gamma + oa), z = *reinterpret_cast<const float4 *>(gamma + ob);
    g[0] = x.x, g[1] = x.y, g[2] = x.z, g[3] = x.w, g[4] = z.x, g[5] = z.y, g[6] = z.z, g[7] = z.w;
  }
  if (kind != 2) {
    for (int i = threadIdx.x; i < toks * half; i += kThreads) {
      const int tt = (int)a.half.div(i), f = i - tt * half;
      const uint64_t turn = (uint64_t)(int64_t)r.pos[tok0 + tt] * r.steps[f];
      float si, co;
      sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &si, &co);  // in units of 2^-31 half turns
      cs[tt * stride + f] = co * r.amplitude, sn[tt * stride + f] = si * r.amplitude;
    }
    __syncthreads();
  }

  const float inv_dim = 1.f / (float)r.dim;
  int pos = -1, slot = -1, at = -1;  // of token `at`
  // of the lane's pairs (p, q): p' = p pc - q qs, q' = q qc + p ps, with gamma in them
  float2 pc[2], qs[2], qc[2], ps[2];
  const auto work = [&](const Row &x) {
    if (x.t != at) {
      at = x.t;
      pos = x.on ? r.pos[tok0 + x.t] : -1;
      slot = CACHE && kind && x.on ? r.slots[tok0 + x.t] : -1;
      if (PAIRS != kAny) {
        float co[4], si[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = turns && x.on && (PAIRS == kHalf || 4 * c + j < half);
          co[j] = in ? cs[x.t * stride + 4 * c + j] : 1.f, si[j] = in ? sn[x.t * stride + 4 * c + j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // kHalf: p in g[0..3], q in g[4..7]; kAdjacent: p, q in turn
          const int p0 = PAIRS == kHalf ? 2 * j : 4 * j, p1 = PAIRS == kHalf ? 2 * j + 1 : 4 * j + 2, q0 = PAIRS == kHalf ? p0 + 4 : p0 + 1, q1 = PAIRS == kHalf ? p1 + 4 : p1 + 1;
          pc[j] = make_float2(g[p0] * co[2 * j], g[p1] * co[2 * j + 1]), qs[j] = make_float2(-g[q0] * si[2 * j], -g[q1] * si[2 * j + 1]);
          qc[j] = make_float2(g[q0] * co[2 * j], g[q1] * co[2 * j + 1]), ps[j] = make_float2(g[p0] * si[2 * j], g[p1] * si[2 * j + 1]);
        }
      }
    }
    float v[8], partner[8];
    x.raw.to(v);
    if (PAIRS == kAny && x.on && mine && kind != 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = c * 8 + j;
        partner[j] = e < r.rot ? (float)x.from[e < half ? e + half : e - half] : 0.f;
      }
    }
    // ---- the norm's factor
    float inv = 1.f;
    if (gamma) {
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 8; j += 2) s2 = __ffma2_rn(make_float2(v[j], v[j + 1]), make_float2(v[j], v[j + 1]), s2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      // (1 / sqrt to 2 units in the last place; infinite for a row of zeros without eps, which gives NaN as 0 / 0 does)
      inv = rsqrtf(fmaf(ss, inv_dim, r.eps));
    }
    // ---- norm and rotation
    if (PAIRS != kAny) {
      if (kind != 2) {
        const float2 i2 = make_float2(inv, inv);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int p0 = PAIRS == kHalf ? 2 * j : 4 * j, p1 = PAIRS == kHalf ? 2 * j + 1 : 4 * j + 2, q0 = PAIRS == kHalf ? p0 + 4 : p0 + 1, q1 = PAIRS == kHalf ? p1 + 4 : p1 + 1;
          const float2 p = __fmul2_rn(make_float2(v[p0], v[p1]), i2), q = __fmul2_rn(make_float2(v[q0], v[q1]), i2);
          const float2 n = __ffma2_rn(p, pc[j], __fmul2_rn(q, qs[j])), m = __ffma2_rn(q, qc[j], __fmul2_rn(p, ps[j]));
          v[p0] = n.x, v[p1] = n.y, v[q0] = m.x, v[q1] = m.y;
        }
      }
    } else {
      if (x.on && mine && kind != 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = c * 8 + j;
          v[j] = v[j] * inv * g[j];
          if (e < r.rot) {
            const int f = x.t * stride + (e < half ? e : e - half);
            const float w = partner[j] * inv * (gamma ? gamma[e < half ? e + half : e - half] : 1.f);
            v[j] = e < half ? v[j] * cs[f] - w * sn[f] : v[j] * cs[f] + w * sn[f];
          }
        }
      }
      __syncwarp();  // partners are read before a row is written in place
    }
    // ---- out
    if (!x.on || pos < 0) return;
    const int tok = tok0 + x.t, head = head0 + x.h;
    if (!CACHE || kind == 0) {
      if (mine) store_fours(static_cast<TO *>(r.out) + tok * r.ldo_token + head * r.ldo_head, oa, ob, v);
    } else if ((uint32_t)slot >= r.n_slots) {
      if (slot != -1 && c == 0) set_device_error(r.err, kDevErrBadPage);
    } else {
      const uint32_t page = a.page.div(slot), off = slot - page * a.page.d;
      const int64_t to = page * r.page_stride + head * r.head_stride + off * r.token_stride;
      if (!E4M3) {
        store_fours(static_cast<__nv_bfloat16 *>(r.cache[kind - 1]) + to, oa, ob, v);
      } else {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
#pragma unroll
        for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o));
        amax = fmaxf(amax, kAmaxFloor);
        float factor;
        const float up = block_factor(amax, c, mask, factor);
        const uint2 w = to_e4m3x8(v, up);
        uint8_t *p = static_cast<uint8_t *>(r.cache[kind - 1]) + to;
        *reinterpret_cast<uint32_t *>(p + oa) = w.x;
        *reinterpret_cast<uint32_t *>(p + ob) = w.y;
        if (c == 0) r.scale[kind - 1][((int64_t)page * r.heads[1] + head) * a.page.d + off] = factor;
      }
    }
  };
  for (int i = 0; i < rows; i += U * SLOTS) {
    Row now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = row[u];
    // the next rows are on their way while these are worked on
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(row[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) work(now[u]);
  }
}

template <int LPR, typename T, typename TO, int PAIRS, bool CACHE, bool E4M3>
cudaError_t go(const Args &a, dim3 grid, size_t smem, cudaStream_t s) {
  rope_kernel<LPR, T, TO, PAIRS, CACHE, E4M3><<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}
template <int LPR, typename T, typename TO, bool CACHE, bool E4M3>
cudaError_t go_pairs(int pairs, const Args &a, dim3 grid, size_t smem, cudaStream_t s) {
  if (pairs == kHalf) return go<LPR, T, TO, kHalf, CACHE, E4M3>(a, grid, smem, s);
  if (pairs == kAdjacent) return go<LPR, T, TO, kAdjacent, CACHE, E4M3>(a, grid, smem, s);
  return go<LPR, T, TO, kAny, CACHE, E4M3>(a, grid, smem, s);
}
template <int LPR, typename T>
cudaError_t go_kind(int pairs, const Args &a, dim3 grid, size_t smem, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (!a.r.cache[0])
    return a.r.out_dtype == Q4K_DTYPE_BF16 ? go_pairs<LPR, T, B, false, false>(pairs, a, grid, smem, s)
                                           : go_pairs<LPR, T, float, false, false>(pairs, a, grid, smem, s);
  return a.r.cache_dtype == Q4K_DTYPE_BF16 ? go_pairs<LPR, T, B, true, false>(pairs, a, grid, smem, s)
                                           : go_pairs<LPR, T, B, true, true>(pairs, a, grid, smem, s);
}
template <typename T>
cudaError_t go_lanes(int lanes, int pairs, const Args &a, dim3 grid, size_t smem, cudaStream_t s) {
  if (lanes <= 8) return go_kind<8, T>(pairs, a, grid, smem, s);
  if (lanes <= 16) return go_kind<16, T>(pairs, a, grid, smem, s);
  return go_kind<32, T>(pairs, a, grid, smem, s);
}

}  // namespace

bool rope_steps(int rot, double base, double factor, int64_t original, double beta_fast,
                double beta_slow, const float *factors, uint64_t *steps, float *amplitude) {
  constexpr double kPi = 3.14159265358979323846;
  const bool ramp = original > 0;
  double low = 0, high = 0;
  if (ramp) {
    // the pair that turns `turns` times over the original context
    const auto at = [&](double turns) { return rot * log((double)original / (turns * 2 * kPi)) / (2 * log(base)); };
    low = fmax(0.0, floor(at(beta_fast)));
    high = fmin((double)rot - 1, ceil(at(beta_slow)));
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot) / (factors ? (double)factors[i] : 1.0);
    const double keep = ramp ? 1.0 - fmin(1.0, fmax(0.0, (i - low) / fmax(0.001, high - low))) : 0.0;
    f = f / factor * (1.0 - keep) + f * keep;
    double turns = f / (2 * kPi);
    if (!(turns - turns == 0.0)) return false;
    turns = (turns - floor(turns)) * 18446744073709551616.0;
    turns = nearbyint(turns);
    steps[i] = turns >= 18446744073709551616.0 ? 0 : (uint64_t)turns;
  }
  *amplitude = ramp ? (float)(1.0 + 0.1 * log(factor)) : 1.f;
  return true;
}

cudaError_t launch_rope(const RopeArgs &r, int dtype, bool interleaved, cudaStream_t stream) {
  const int lanes = (r.dim + 7) / 8, lpr = lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32, slots = kThreads / lpr;
  const int heads = r.heads[0] + (r.cache[0] ? 2 * r.heads[1] : 0), half = r.rot / 2;
  const int pairs = interleaved ? kAdjacent : half % 4 ? kAny : kHalf;
  // Rows per block: one per group of lanes while there are few, so that all SMs
  // take part; of many, 8 or more, of as many tokens as give every thread an angle.
  Args a = {};
  a.r = r, a.half = FastDiv(half > 0 ? half : 1), a.page = FastDiv(r.cache[0] ? r.page : 1);
  const int64_t sms = device_facts()->sm_count;
  const bool few = r.tokens * heads <= sms * 16 * slots;
  int most = 1;
  for (int i = 0; i < (r.cache[0] ? 2 : 1); ++i) {
    int toks = 1, hpb = r.heads[i];
    if (few) hpb = hpb < slots ? hpb : slots;
    else
      while (toks * half < kThreads && toks * hpb < 8 * slots) ++toks;
    const int groups = (r.heads[i] + hpb - 1) / hpb;
    a.tokens_per_block[i] = toks, a.heads_per_block[i] = hpb, a.groups[i] = FastDiv(groups);
    a.blocks[i] = (uint32_t)((r.tokens + toks - 1) / toks * groups);
    most = toks > most ? toks : most;
  }
  const dim3 grid(a.blocks[0] + 2 * a.blocks[1]);
  const size_t smem = (size_t)2 * most * ((half + 3) & ~3) * 4;
  return dtype == Q4K_DTYPE_BF16 ? go_lanes<__nv_bfloat16>(lanes, pairs, a, grid, smem, stream)
                                 : go_lanes<float>(lanes, pairs, a, grid, smem, stream);
}

}  // namespace q4k
