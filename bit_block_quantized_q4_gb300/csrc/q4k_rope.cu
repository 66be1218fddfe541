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
// that the table's rounding leaves times the position (the table is computed in twice
// 64 bits: from doubles alone its values are up to 182 units off, 2^-25 of a turn at
// position 2^31).  Its upper 32 bits, signed, are the angle in (-1/2, 1/2] turns.
//
// What bounds it: bytes, each read and written once; so rows stay in registers, and
// all loads of a thread go out at its start.  D / 8 lanes take a row, and up to R
// heads of the same token.  While the rows are on their way the block computes the
// cosines and sines of its tokens, which are the same for all heads, into shared
// memory: a thread one or a few.  Measured (of the copy rate): 8191 x 64 x 128 bf16 46 us
// (87%), 8191 x 24 x 256 with 64 values rotated 47 us (64%; its tokens take 3 of a block's 8
// groups of lanes each, so that a quarter of the warps have no rows), with the write of an e4m3
// cache 8191 x (64 + 16) x 128 78 us (61%), there with issue slots 65% busy; 16 x 64 heads
// 4.2 us, a launch and two dependent loads.
//
// Cosine and sine of q quarter turns and x more, |x| <= 1/2: Taylor's series of sin
// and cos of x pi / 2 to the terms x^9 and x^10, beyond which there are 2 10^-9, and
// the quadrant's signs.
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
// Heads of a thread: where rows are few, and where they are many.  A prompt block of
// 8191 x 80 x 128 bf16 to e4m3 took 127, 84 and 80 us with 2, 4 and 8; fp32 rows take
// twice the registers.
constexpr int kFew = 1;
template <typename T>
constexpr int kMany = sizeof(T) == 2 ? 8 : 4;

enum Pairs { kHalf = 0, kAdjacent = 1, kAny = 2 };  // kAny: (i, i + R / 2) where R / 2 is no multiple of 4

struct Args {
  RopeArgs r;
  FastDiv per_token[2];  // groups of lanes that share a token: of a block of queries, of keys and values
  int tokens[2];         // tokens of such a block
  int rows[2];           // rows of a thread there, at most R
  uint32_t blocks[2];    // such blocks: head groups of the first tokens, of the next
  FastDiv groups[2];
  FastDiv half, page;
};

// Cosine and sine of turn / 2^32 turns.
__device__ __forceinline__ void cos_sin(uint32_t turn, float &co, float &si) {
  const uint32_t q = (turn + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(turn - (q << 30)) * 9.313225746154785e-10f, z = x * x;  // 2^-30
  float s = fmaf(z, 1.60441184e-4f, -4.68175413e-3f);
  s = fmaf(z, s, 7.96926262e-2f);
  s = fmaf(z, s, -6.45964097e-1f);
  s = fmaf(z, s, 1.57079633f) * x;
  float c = fmaf(z, -2.52020424e-5f, 9.19260274e-4f);
  c = fmaf(z, c, -2.08634807e-2f);
  c = fmaf(z, c, 2.53669508e-1f);
  c = fmaf(z, c, -1.23370055f);
  c = fmaf(z, c, 1.f);
  const auto sign = [](float v, uint32_t bit) { return __int_as_float(__float_as_int(v) ^ (int)((bit & 2u) << 30)); };
  co = sign(q & 1u ? s : c, q + 1u);
  si = sign(q & 1u ? c : s, q);
}
// The upper half of pos * step modulo 2^64: the fraction of a turn.
__device__ __forceinline__ uint32_t turn_of(uint32_t pos, uint64_t step) {
  return __umulhi(pos, (uint32_t)step) + pos * (uint32_t)(step >> 32);
}

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

template <int LPR, typename T, int PAIRS, bool CACHE, int R>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const Args a) {
  // cosines and sines of the block's tokens, [token][R / 2] each
  constexpr int SLOTS = kThreads / LPR;  // rows at a time
  __shared__ __align__(16) float cs[SLOTS * LPR * 4], sn[SLOTS * LPR * 4];
  const RopeArgs &r = a.r;
  const int c = threadIdx.x % LPR, slot_in = threadIdx.x / LPR, lane = threadIdx.x & 31;
  // Blocks of queries first, then of keys and values (heads 0 .. of keys, then of values).
  const int kv = CACHE && blockIdx.x >= a.blocks[0];
  const uint32_t x = blockIdx.x - (kv ? a.blocks[0] : 0u), part = a.groups[kv].div(x);
  const int all = kv ? 2 * r.heads[1] : r.heads[0], per_token = (int)a.per_token[kv].d, rows = a.rows[kv];
  // this group's token, and its heads s, s + per_token, ...
  const int tt = (int)a.per_token[kv].div(slot_in), s = slot_in - tt * per_token + (int)(x - part * a.groups[kv].d) * per_token * rows;
  const int64_t tok = (int64_t)part * a.tokens[kv] + tt;
  const bool there = tt < a.tokens[kv] && tok < r.tokens;
  const int half = r.rot / 2, stride = (half + 3) & ~3;
  const unsigned mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (lane / LPR * LPR);
  const bool mine = c * 8 < r.dim;  // lanes past the row's end only take part in sums
  // this lane's values oa .. oa + 3 and ob .. ob + 3; whether they turn, by the angles 4 c ..
  int oa = 8 * c, ob = oa + 4;
  bool turns = oa < r.rot;
  if (PAIRS == kHalf) {
    turns = 4 * c < half;
    if (turns) oa = 4 * c, ob = half + 4 * c;
  }
  const int pos = there ? r.pos[tok] : -1;
  const int slot = kv && there ? r.slots[tok] : -1;

  // ---- all rows of this thread
  const T *from = static_cast<const T *>(r.in[kv]) + tok * r.ld_token[kv] + s * r.ld_head[kv];
  const int64_t step = per_token * r.ld_head[kv];
  // values lie so far from keys, and their heads begin again
  const int64_t to_v = kv ? (static_cast<const T *>(r.in[2]) - static_cast<const T *>(r.in[1])) - r.heads[1] * r.ld_head[1] : 0;
  Fours<T> raw[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    raw[k] = Fours<T>();
    const int h = s + k * per_token;
    if (k < rows && there && h < all && mine) raw[k].load(from + k * step + (kv && h >= r.heads[1] ? to_v : 0), oa, ob);
  }

  // ---- the block's angles
  const int64_t tok0 = (int64_t)part * a.tokens[kv];
  const int toks = (int)min((int64_t)a.tokens[kv], r.tokens - tok0);
  for (int i = threadIdx.x; i < toks * half; i += kThreads) {
    const int ti = (int)a.half.div(i), f = i - ti * half;
    float co, si;
    cos_sin(turn_of((uint32_t)max(r.pos[tok0 + ti], 0), r.steps[f]), co, si);
    cs[ti * stride + f] = co * r.amplitude, sn[ti * stride + f] = si * r.amplitude;
  }
  __syncthreads();

  // ---- its pairs (p, q): p' = p pc + q qs, q' = q qc + p ps, with
  // gamma in them; values that do not turn keep their size
  const float *gamma = r.gamma[kv];
  float g[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = 1.f;
  if (mine && gamma) {
    const float4 y = *reinterpret_cast<const float4 *>(gamma + oa), z = *reinterpret_cast<const float4 *>(gamma + ob);
    g[0] = y.x, g[1] = y.y, g[2] = y.z, g[3] = y.w, g[4] = z.x, g[5] = z.y, g[6] = z.z, g[7] = z.w;
  }
  // kHalf: p in values 0..3, q in 4..7; kAdjacent: p, q in turn
  constexpr int P0[2] = {0, PAIRS == kHalf ? 2 : 4}, S1 = PAIRS == kHalf ? 1 : 2, Q = PAIRS == kHalf ? 4 : 1;
  float2 pc[2], qs[2], qc[2], ps[2];
  if (PAIRS != kAny) {
    float4 co4 = make_float4(1.f, 1.f, 1.f, 1.f), si4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turns && tt < a.tokens[kv]) {
      const float4 y = *reinterpret_cast<const float4 *>(cs + tt * stride + 4 * c), z = *reinterpret_cast<const float4 *>(sn + tt * stride + 4 * c);
      co4.x = y.x, si4.x = z.x;
      if (PAIRS == kHalf || 4 * c + 1 < half) co4.y = y.y, si4.y = z.y;
      if (PAIRS == kHalf || 4 * c + 2 < half) co4.z = y.z, si4.z = z.z;
      if (PAIRS == kHalf || 4 * c + 3 < half) co4.w = y.w, si4.w = z.w;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 co = j ? make_float2(co4.z, co4.w) : make_float2(co4.x, co4.y), si = j ? make_float2(si4.z, si4.w) : make_float2(si4.x, si4.y);
      const float2 gp = make_float2(g[P0[j]], g[P0[j] + S1]), gq = make_float2(g[P0[j] + Q], g[P0[j] + S1 + Q]);
      pc[j] = __fmul2_rn(gp, co), qc[j] = __fmul2_rn(gq, co), ps[j] = __fmul2_rn(gp, si);
      qs[j] = __fmul2_rn(gq, make_float2(-si.x, -si.y));
    }
  }
  const float inv_dim = 1.f / (float)r.dim;
  // ---- where the first row goes, in bytes; the next ones lie steps further, values elsewhere
  const bool e4m3 = CACHE && r.cache_dtype != Q4K_DTYPE_BF16, wide = !CACHE && r.out_dtype == Q4K_DTYPE_FP32;
  const bool valid = !kv || (uint32_t)slot < r.n_slots;
  uint8_t *to = nullptr;
  int64_t to_step = 0, to_value = 0;
  float *scale = nullptr;
  int64_t scale_value = 0;
  if (!kv) {
    const int shift = wide ? 2 : 1;
    to = static_cast<uint8_t *>(r.out) + ((tok * r.ldo_token + s * r.ldo_head) << shift);
    to_step = (per_token * r.ldo_head) << shift;
  } else if (valid) {
    const int shift = e4m3 ? 0 : 1;
    const uint32_t page = a.page.div(slot), off = slot - page * a.page.d;
    to = static_cast<uint8_t *>(r.cache[0]) + ((page * r.page_stride + s * r.head_stride + off * r.token_stride) << shift);
    to_step = (per_token * r.head_stride) << shift;
    to_value = (static_cast<uint8_t *>(r.cache[1]) - static_cast<uint8_t *>(r.cache[0])) - ((r.heads[1] * r.head_stride) << shift);
    if (e4m3) {
      scale = r.scale[0] + ((int64_t)page * r.heads[1] + s) * a.page.d + off;
      scale_value = (r.scale[1] - r.scale[0]) - (int64_t)r.heads[1] * a.page.d;
    }
  }
  if (kv && !valid && slot != -1 && pos >= 0 && c == 0) set_device_error(r.err, kDevErrBadPage);

#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (k >= rows) break;
    const int h = s + k * per_token;
    const bool on = there && h < all, value = kv && h >= r.heads[1];
    float v[8], partner[8];
    raw[k].to(v);
    if (PAIRS == kAny && on && mine && !value) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = c * 8 + j;
        partner[j] = e < r.rot ? (float)from[k * step + (e < half ? e + half : e - half)] : 0.f;
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
      if (!value) {
        const float2 i2 = make_float2(inv, inv);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 p = __fmul2_rn(make_float2(v[P0[j]], v[P0[j] + S1]), i2), q = __fmul2_rn(make_float2(v[P0[j] + Q], v[P0[j] + S1 + Q]), i2);
          const float2 n = __ffma2_rn(p, pc[j], __fmul2_rn(q, qs[j])), m = __ffma2_rn(q, qc[j], __fmul2_rn(p, ps[j]));
          v[P0[j]] = n.x, v[P0[j] + S1] = n.y, v[P0[j] + Q] = m.x, v[P0[j] + S1 + Q] = m.y;
        }
      }
    } else {
      if (on && mine && !value) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {  // (r.rot is even, so both turn or none)
          const int e = c * 8 + j;
          v[j] = v[j] * inv * g[j], v[j + 1] = v[j + 1] * inv * g[j + 1];
          if (e < r.rot) {
            const bool lo0 = e < half, lo1 = e + 1 < half;
            const int o0 = lo0 ? e + half : e - half, o1 = lo1 ? e + 1 + half : e + 1 - half;  // partners
            const int f0 = tt * stride + min(e, o0), f1 = tt * stride + min(e + 1, o1);
            const float w0 = partner[j] * inv * (gamma ? gamma[o0] : 1.f), w1 = partner[j + 1] * inv * (gamma ? gamma[o1] : 1.f);
            v[j] = v[j] * cs[f0] + (lo0 ? -w0 : w0) * sn[f0];
            v[j + 1] = v[j + 1] * cs[f1] + (lo1 ? -w1 : w1) * sn[f1];
          }
        }
      }
      __syncwarp();  // partners are read before a row is written in place
    }
    // ---- out
    if (!on || pos < 0 || !valid) continue;
    uint8_t *p = to + k * to_step + (value ? to_value : 0);
    if (!kv || !e4m3) {
      if (!mine) continue;
      if (wide) store_fours(reinterpret_cast<float *>(p), oa, ob, v);
      else store_fours(reinterpret_cast<__nv_bfloat16 *>(p), oa, ob, v);
      continue;
    }
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o));
    amax = fmaxf(amax, kAmaxFloor);
    // (a reciprocal and products, each off by half a unit, where q4k_kv_write divides: 60 instructions fewer)
    const uint2 w = to_e4m3x8(v, 448.f * __frcp_rn(amax));
    *reinterpret_cast<uint32_t *>(p + oa) = w.x;
    *reinterpret_cast<uint32_t *>(p + ob) = w.y;
    if (c == 0) scale[k * per_token * (int)a.page.d + (value ? scale_value : 0)] = amax * (1.f / 448.f);
  }
}

template <int LPR, typename T, int PAIRS, bool CACHE>
cudaError_t go(const RopeArgs &r, cudaStream_t s) {
  constexpr int SLOTS = kThreads / LPR;
  // Heads of a thread: one while that leaves SMs without work; else kMany, for which
  // its angles are computed once, of as many tokens as a block has room for.  Measured,
  // 64 heads x 128, us with one / kMany: 512 tokens 9.0 / 7.6, 1024 tokens 14.6 / 12.4, and
  // up to 256 tokens the same (6.3).
  const bool many = r.tokens * (r.heads[0] + (CACHE ? 2 * r.heads[1] : 0)) > (int64_t)device_facts()->sm_count * 8 * SLOTS;
  Args a = {r, {FastDiv(1), FastDiv(1)}, {}, {}, {}, {FastDiv(1), FastDiv(1)}, FastDiv(r.rot > 0 ? r.rot / 2 : 1), FastDiv(CACHE ? r.page : 1)};
  for (int i = 0; i < (CACHE ? 2 : 1); ++i) {
    const int heads = i ? 2 * r.heads[1] : r.heads[0], most = many ? kMany<T> : kFew, least = (heads + most - 1) / most;
    const int per_token = least < SLOTS ? least : SLOTS, each = (heads + per_token - 1) / per_token;
    const int groups = (each + most - 1) / most;
    a.per_token[i] = FastDiv(per_token), a.tokens[i] = SLOTS / per_token, a.rows[i] = (each + groups - 1) / groups, a.groups[i] = FastDiv(groups);
    a.blocks[i] = (uint32_t)((r.tokens + a.tokens[i] - 1) / a.tokens[i] * groups);
  }
  if (many) rope_kernel<LPR, T, PAIRS, CACHE, kMany<T>><<<a.blocks[0] + a.blocks[1], kThreads, 0, s>>>(a);
  else rope_kernel<LPR, T, PAIRS, CACHE, kFew><<<a.blocks[0] + a.blocks[1], kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <int LPR, typename T, int PAIRS>
cudaError_t go_kind(const RopeArgs &r, cudaStream_t s) {
  return r.cache[0] ? go<LPR, T, PAIRS, true>(r, s) : go<LPR, T, PAIRS, false>(r, s);
}
template <int LPR, typename T>
cudaError_t go_pairs(int pairs, const RopeArgs &r, cudaStream_t s) {
  if (pairs == kHalf) return go_kind<LPR, T, kHalf>(r, s);
  if (pairs == kAdjacent) return go_kind<LPR, T, kAdjacent>(r, s);
  return go_kind<LPR, T, kAny>(r, s);
}
template <typename T>
cudaError_t go_lanes(int pairs, const RopeArgs &r, cudaStream_t s) {
  if (r.dim <= 64) return go_pairs<8, T>(pairs, r, s);
  if (r.dim <= 128) return go_pairs<16, T>(pairs, r, s);
  return go_pairs<32, T>(pairs, r, s);
}

}  // namespace

namespace {
// A number as the exact sum of two doubles, the second at most half a unit in the
// last place of the first: about 104 bits.  (Dekker 1971, Knuth: the error of a sum or
// a product of two doubles is a double.)
struct Two {
  double hi, lo;
};
Two two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Two times(Two a, Two b) {
  volatile const double rounded = a.hi * b.hi;  // (not fused with the sum below)
  const double p = rounded;
  return two_sum(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Two plus(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}
Two over(Two a, double b) {  // the quotient, and what it leaves over b
  const double q = a.hi / b;
  return two_sum(q, (fma(-q, b, a.hi) + a.lo) / b);
}
// base^(-i / n) for 0 <= i < n: the root r of r^n base^i = 1 near pow's.  With e = r^n base^i - 1,
// of n times pow's error, the root is r (1 - e / n) to e^2.  The factors alternate, so that
// the product stays within a factor of base.
Two root_of(double base, int i, int n) {
  const double r = pow(base, -(double)i / n);
  Two p = {1.0, 0.0};
  for (int j = 0, k = 0; j < n; ++j) {
    p = times(p, {r, 0.0});
    for (; k * n < (j + 1) * i; ++k) p = times(p, {base, 0.0});
  }
  const Two e = over(plus(p, {-1.0, 0.0}), (double)n);
  return times({r, 0.0}, plus({1.0, 0.0}, {-e.hi, -e.lo}));
}
}  // namespace

bool rope_steps(int rot, double base, double factor, int64_t original, double beta_fast,
                double beta_slow, const float *factors, uint64_t *steps, float *amplitude) {
  constexpr double kPi = 3.14159265358979323846;
  constexpr Two kTurn = {0.15915494309189535, -9.839338337591243e-18};  // 1 / 2 pi
  const bool ramp = original > 0;
  double low = 0, high = 0;
  if (ramp) {
    // the pair that turns `turns` times over the original context
    const auto at = [&](double turns) { return rot * log((double)original / (turns * 2 * kPi)) / (2 * log(base)); };
    low = fmax(0.0, floor(at(beta_fast)));
    high = fmin((double)rot - 1, ceil(at(beta_slow)));
  }
  for (int i = 0; i < rot / 2; ++i) {
    // (in twice the bits: a position multiplies the table's error by up to 2^31)
    Two f = over(root_of(base, i, rot / 2), factors ? (double)factors[i] : 1.0);
    const Two slow = over(f, factor);
    const double width = fmax(0.001, high - low), from = i - low;
    if (!ramp || from >= width) f = slow;
    else if (from > 0) f = plus(times(f, over({width - from, 0.0}, width)), times(slow, over({from, 0.0}, width)));
    const Two turns = times(f, kTurn);
    if (!(turns.hi - turns.hi == 0.0)) return false;
    // modulo 1, in units of 2^-64: both parts without their whole turns, which come off exactly
    const Two part = two_sum(turns.hi - floor(turns.hi), turns.lo - nearbyint(turns.lo));
    const double upper = part.hi * 4294967296.0, whole = floor(upper);
    const double lower = nearbyint(((upper - whole) + part.lo * 4294967296.0) * 4294967296.0);
    steps[i] = ((uint64_t)(int64_t)whole << 32) + (uint64_t)(int64_t)lower;
  }
  *amplitude = ramp ? (float)(1.0 + 0.1 * log(factor)) : 1.f;
  return true;
}

cudaError_t launch_rope(const RopeArgs &r, int dtype, bool interleaved, cudaStream_t stream) {
  const int pairs = interleaved ? kAdjacent : (r.rot / 2) % 4 ? kAny : kHalf;
  return dtype == Q4K_DTYPE_BF16 ? go_lanes<__nv_bfloat16>(pairs, r, stream) : go_lanes<float>(pairs, r, stream);
}

}  // namespace q4k
