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

enum Pairs { kHalf = 0, kAdjacent = 1, kAny = 2 };  // kAny: (i, i + R / 2) where R / 2 is no multiple of 8

struct Args {
  RopeArgs r;
  int heads;           // rows of a token: q, k, v heads
  int tokens_per_block, heads_per_block;
  FastDiv rows_div;    // by heads_per_block
  FastDiv page;
};

template <int LPR, typename T, typename TO, int PAIRS, bool CACHE, bool E4M3>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Args a) {
  extern __shared__ __align__(16) float table[];
  const RopeArgs &r = a.r;
  const int c = threadIdx.x % LPR, slot_in = threadIdx.x / LPR, lane = threadIdx.x & 31;
  const int tok0 = blockIdx.x * a.tokens_per_block, head0 = blockIdx.y * a.heads_per_block;
  const int toks = min(a.tokens_per_block, (int)(r.tokens - tok0)), heads = min(a.heads_per_block, a.heads - head0);
  const int rows = toks * heads, half = r.rot / 2;
  float *cs = table, *sn = table + a.tokens_per_block * ((half + 3) & ~3);
  const unsigned mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (lane / LPR * LPR);
  const bool mine = c * 8 < r.dim;  // lanes past the row's end only take part in sums

  struct Row {
    int tok, kind, head;  // kind 0: q, 1: k, 2: v
    bool on;
    const T *from;
  };
  const auto row_at = [&](int i) {
    Row x;
    x.on = i < rows;
    const int t = heads == a.heads_per_block ? (int)a.rows_div.div(x.on ? i : 0) : (x.on ? i : 0) / heads;
    const int h = (x.on ? i : 0) - t * heads + head0;
    x.tok = tok0 + t;
    x.kind = !CACHE || h < r.heads[0] ? 0 : h < r.heads[0] + r.heads[1] ? 1 : 2;
    x.head = x.kind == 0 ? h : h - r.heads[0] - (x.kind == 2 ? r.heads[1] : 0);
    x.from = static_cast<const T *>(r.in[x.kind]) + x.tok * r.ld_token[x.kind] + x.head * r.ld_head[x.kind] + c * 8;
    return x;
  };
  Row x = row_at(slot_in);
  Raw8<T> raw = {};
  if (x.on && mine) raw.load(x.from);
  {
    const int stride = (half + 3) & ~3;
    for (int i = threadIdx.x; i < toks * half; i += kThreads) {
      const int t = i / half, f = i - t * half;
      const uint64_t turn = (uint64_t)(int64_t)r.pos[tok0 + t] * r.steps[f];
      float s, co;
      sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &co);  // in units of 2^-31 half turns
      cs[t * stride + f] = co * r.amplitude, sn[t * stride + f] = s * r.amplitude;
    }
  }
  __syncthreads();

  for (int i = slot_in; i - slot_in < rows; i += kThreads / LPR) {
    const Row next = row_at(i + kThreads / LPR);
    Raw8<T> ahead = {};
    if (next.on && mine) ahead.load(next.from);
    float v[8];
    raw.to(v);
    const int pos = x.on ? r.pos[x.tok] : -1;
    const int slot = CACHE && x.kind && pos >= 0 ? r.slots[x.tok] : -1;
    float partner[8];
    if (PAIRS == kAny && x.on && mine && x.kind != 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = c * 8 + j;
        partner[j] = e < r.rot ? (float)x.from[e < half ? j + half : j - half] : 0.f;
      }
    }
    // ---- norm
    const float *gamma = r.gamma[CACHE && x.kind == 1];
    if (r.gamma[0] || r.gamma[1]) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (gamma && x.kind != 2 && mine) {
        const float inv = 1.f / sqrtf(ss / (float)r.dim + r.eps);
        float g[8];
        load8(gamma + c * 8, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= inv * g[j];
        if (PAIRS == kAny) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = c * 8 + j;
            if (e < r.rot) partner[j] *= inv * gamma[e < half ? e + half : e - half];
          }
        }
      }
    }
    // ---- rotation
    const int t = x.tok - tok0;
    const float *ct = cs + t * ((half + 3) & ~3), *st = sn + t * ((half + 3) & ~3);
    if (PAIRS == kHalf) {
      // values c * 8 .. c * 8 + 7 pair with those of the lane half / 8 before or after
      const bool first = c * 8 < half, in = c * 8 < r.rot;
      const int other = (lane & ~(LPR - 1)) + (in ? (first ? c + half / 8 : c - half / 8) : c);
#pragma unroll
      for (int j = 0; j < 8; ++j) partner[j] = __shfl_sync(0xffffffffu, v[j], other);
      if (in && x.kind != 2) {
        const int f = first ? c * 8 : c * 8 - half;
        float co[8], si[8];
        load8(ct + f, co);
        load8(st + f, si);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = first ? v[j] * co[j] - partner[j] * si[j] : v[j] * co[j] + partner[j] * si[j];
      }
    } else if (PAIRS == kAdjacent) {
      if (x.kind != 2) {
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          if (c * 8 + j < r.rot) {
            const float co = ct[c * 4 + j / 2], si = st[c * 4 + j / 2], p = v[j], q = v[j + 1];
            v[j] = p * co - q * si;
            v[j + 1] = q * co + p * si;
          }
      }
    } else if (x.on && mine && x.kind != 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = c * 8 + j;
        if (e < r.rot) {
          const int f = e < half ? e : e - half;
          v[j] = e < half ? v[j] * ct[f] - partner[j] * st[f] : v[j] * ct[f] + partner[j] * st[f];
        }
      }
    }
    if (PAIRS == kAny) __syncwarp();  // partners are read before a row is written in place
    // ---- out
    if (x.on && pos >= 0) {
      if (!CACHE || x.kind == 0) {
        if (mine) store8(static_cast<TO *>(r.out) + x.tok * r.ldo_token + x.head * r.ldo_head + c * 8, v);
      } else if ((uint32_t)slot >= r.n_slots) {
        if (slot != -1 && c == 0) set_device_error(r.err, kDevErrBadPage);
      } else {
        const uint32_t page = a.page.div(slot), off = slot - page * a.page.d;
        const int64_t to = page * r.page_stride + x.head * r.head_stride + off * r.token_stride + c * 8;
        if (!E4M3) {
          store8(static_cast<__nv_bfloat16 *>(r.cache[x.kind - 1]) + to, v);
        } else {
          float amax = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o));
          amax = fmaxf(amax, kAmaxFloor);
          float factor;
          const float inv = block_factor(amax, c, mask, factor);
          *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(r.cache[x.kind - 1]) + to) = to_e4m3x8(v, inv);
          if (c == 0) r.scale[x.kind - 1][((int64_t)page * r.heads[1] + x.head) * a.page.d + off] = factor;
        }
      }
    }
    x = next;
    raw = ahead;
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
  const int pairs = interleaved ? kAdjacent : half % 8 ? kAny : kHalf;
  // Rows per block: one per group of lanes while there are few, so that all SMs
  // take part; of many, all heads of as many tokens as give every thread an angle.
  const int64_t sms = device_facts()->sm_count;
  int toks = 1, hpb = heads;
  if (r.tokens * heads <= sms * 16 * slots) {
    hpb = heads < slots ? heads : slots;
  } else {
    while (toks * half < kThreads && toks * heads < 8 * slots) ++toks;
  }
  const Args a = {r, heads, toks, hpb, FastDiv(hpb), FastDiv(r.cache[0] ? r.page : 1)};
  const dim3 grid((unsigned)((r.tokens + toks - 1) / toks), (unsigned)((heads + hpb - 1) / hpb));
  const size_t smem = (size_t)2 * toks * ((half + 3) & ~3) * 4;
  return dtype == Q4K_DTYPE_BF16 ? go_lanes<__nv_bfloat16>(lanes, pairs, a, grid, smem, stream)
                                 : go_lanes<float>(lanes, pairs, a, grid, smem, stream);
}

}  // namespace q4k
