// q4k_attn.cu -- attention of one new token per request over the paged cache
// (q4k_paged_attn).
//
// "spec: specialized model runtimes", section "Architecture": attention is an
// op of kernel tier T0.
//
// Mathematics.  One pass over the keys with the running maximum m and sum l of
// a softmax, all in base 2 (scores carry log2 e):
//   m' = max(m, z_j),  l' = l 2^(m-m') + 2^(z_j-m'),
//   o' = o 2^(m-m') + 2^(z_j-m') v_j,  out = o / l;
// two parts of a key range are joined by the same rule.
//
// What bounds it: bytes.  At 8 query heads per key head a bf16 cache gives 8
// operations per byte, an e4m3 cache 16: far below the tensor rate, so the
// design is about keeping bytes in flight.  mma.sync suffices for the arithmetic; with one new token the
// scores of a group fill the 8 columns of its N side exactly, where a
// tcgen05.mma would want 64 or 128 rows.
//
// Work split.  The (request, key head) items, each a run of tiles of TILE
// tokens, form one list; every warp of a persistent grid takes an equal run of
// it, whatever the requests' lengths.  The lengths are on the device, so each
// CTA sums them itself.  An item inside one warp's run is written out directly;
// the pieces of the others go to the workspace and a second launch joins them.
//
// A warp streams its own ring of tiles: one TMA tile copy per page and buffer
// (5-D map: 128 bytes of a row, token, part of the row, head, page; 128-byte
// swizzle), issued by its lane 0 STAGES tiles ahead across item boundaries.
// Warps never wait for one another inside the loop.
//
// Products, transposed so that the query heads are the 8 columns:
//   S^T[16 keys, 8 heads] += K[16 keys, 16 d] Q^T     (ldmatrix)
//   O^T[16 d, 8 heads]    += V^T[16 d, 16 keys] P^T   (ldmatrix.trans; P^T from
//                                                      S^T by movmatrix)
// bf16 cache: P enters as two bf16 terms (hi + lo, 16 bits), because one
// rounding of P to 8 bits would be as large as the output's own.  e4m3 cache:
// K and V are converted exactly to fp16; q is scaled by a power of two per head
// into fp16 (exact down to 2^-31 of the head's largest value, to within 2^-39 of
// it below); and P times the row's V scale enters as one fp16 term.  Its running
// maximum is that of z + log2(scale), which keeps this term at most 1 whatever the
// scales; it is stored times 2^15, fp16's upper half, so that it has its 11 bits
// down to 2^-29 of the largest and an error of 2^-40 of it below.  (Stored as it
// is, terms below 2^-14 lost bits and those below 2^-25 were 0, while the sum of
// weights held them: the part of 31 tokens 20 binary orders below another came out
// wrong by 1%.  The multiplications cost 1%: 4 requests of 90..131 thousand tokens,
// 16 heads per key head, 95.9 -> 96.8 us.)
//
// Groups of more query heads than an item holds (8 at dim 256, else 16) are
// several items, each over all of the cache: at dim 256 and 1 GB of cache 8 heads
// take 177 us, 12 and 16 take 330.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

constexpr int kMaxSms = 160;   // SMs and warps per SM that the workspace is
constexpr int kMaxWarps = 12;  // sized for

template <int D, bool E4M3>
struct Cfg {
  static constexpr int kEs = E4M3 ? 1 : 2;
  static constexpr int kTile = D * kEs >= 512 ? 16 : 32;    // tokens per tile
  static constexpr int kRow = D * kEs >= 128 ? 128 : 64;    // bytes of a row per swizzled part
  static constexpr int kParts = D * kEs / kRow;
  static constexpr int kSide = kTile * D * kEs;             // bytes of K (or V) per tile
  static constexpr int kScales = E4M3 ? kTile * 4 : 0;      // bytes of K (or V) scales per tile
  static constexpr int kWarps = kSide >= 8192 ? 6 : 12;
  static constexpr int kStages = kSide >= 4096 ? 2 : 3;
  // per warp STAGES x (K | V), 1024-byte aligned as the swizzle wants it; then
  // per warp STAGES x (K scales | V scales)
  static constexpr int kRing = kStages * 2 * kSide, kScaleRing = kStages * 2 * kScales;
  static constexpr int kSmem = kWarps * (kRing + kScaleRing) + 1024;
  static_assert(kWarps <= kMaxWarps, "the workspace has two slots for each of kMaxWarps warps");
  static_assert(kSide % 1024 == 0, "tile buffers keep the swizzle's alignment");
};

struct Params {
  AttnArgs a;
  int groups;      // query-head groups per key head
  int items;       // items per request: kv_heads * groups
  int group_size;  // query heads per key head
  int heads_per_item;  // of them in an item: 8 per n-tile
  int box_rows, box_shift, page_shift;
  int64_t warps;   // of the whole grid
  int64_t *prefix;  // [n + 1] tiles per head before a request
  float *slots;
};

// Tiles per warp.  Even a run of one tile pays: for 22 tiles per head (one
// request of 700 tokens) runs of 1, 2, 4 and 8 took 9.6, 10.9, 14.0 and 19.7 us.
__device__ __forceinline__ int64_t run_of(int64_t tiles, int64_t warps) {
  const int64_t c = (tiles + warps - 1) / warps;
  return c < 1 ? 1 : c;
}

// A request's tokens start .. len - 1 and their tiles t0 .. t1 - 1.  The window
// ends at lens[r] itself; tokens past the table are absent, so that a request
// far longer than its table may have none.
template <int TILE>
__device__ __forceinline__ void span_of(const AttnArgs &a, int r, int &len, int &start, int &t0, int &t1) {
  const int told = a.lens[r], cap = a.max_pages * a.page;
  len = told < 0 ? 0 : told > cap ? cap : told;
  start = a.window > 0 && told > a.window ? told - a.window : 0;
  t0 = start / TILE;
  t1 = start < len ? (len + TILE - 1) / TILE : t0;
}

// What the e4m3 path stores its weights times, and o with them; l stays as it is.
constexpr float kUp = 32768.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// Four e4m3 values to two fp16 pairs (the lower two, the upper two), exact.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// The state of a piece in registers.  Thread (g = lane / 4, t = lane % 4) has
// of every n-tile j the heads 8 j + 2t and 8 j + 2t + 1; o[dt][j] holds, of the
// 16 values 16 dt .. 16 dt + 15 of a row, rows (d0, d1) x these two heads:
// d0 = g, d1 = g + 8 (bf16) or d0 = 2g, d1 = 2g + 1 (e4m3).
template <int D, int NQ>
struct State {
  float o[D / 16][NQ][4];
  float m[NQ][2], l[NQ][2];
};

// Writes D values of a head's row of `row` values, from d0 on, for the heads of
// n-tiles j0 .. j0 + NQ - 1 of an item.  No token: l is 0.
template <int D, bool E4M3, int NQ>
__device__ __forceinline__ void write_out(const Params &p, const State<D, NQ> &s, int r, int item, int j0, int d0, int row, bool lse) {
  const AttnArgs &a = p.a;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kvh = item / p.groups, q0 = (item - kvh * p.groups) * p.heads_per_item + 8 * j0;
#pragma unroll
  for (int j = 0; j < NQ; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int q = q0 + 8 * j + 2 * t + c;
      if (q >= p.group_size) continue;
      const float l = s.l[j][c], inv = l == 0.f ? 0.f : (E4M3 ? 1.f / kUp : 1.f) / l;
      const int head = kvh * p.group_size + q;
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + r * a.ldo + (int64_t)head * row + d0;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
        const float v0 = s.o[dt][j][c] * inv, v1 = s.o[dt][j][2 + c] * inv;
        if (E4M3) {
          *reinterpret_cast<uint32_t *>(out + 16 * dt + 2 * g) = pack_bf16(v0, v1);
        } else {
          out[16 * dt + g] = __float2bfloat16(v0);
          out[16 * dt + 8 + g] = __float2bfloat16(v1);
        }
      }
      if (lse && a.lse && g == 0)
        a.lse[(int64_t)r * a.q_heads + head] = l == 0.f ? -INFINITY : (s.m[j][c] + log2f(l)) * 0.6931471805599453f;
    }
}

// Floats of one workspace slot: the o registers and m, l of every lane.
template <int D, int NQ>
constexpr int slot_floats() {
  return 32 * NQ * (D / 16 * 4 + 4);
}

template <int D, bool E4M3, int NQ>
__global__ void __launch_bounds__(Cfg<D, E4M3>::kWarps * 32, 1)
    paged_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, E4M3>;
  constexpr int TILE = C::kTile, MT = TILE / 16, W = C::kWarps, ST = C::kStages, T = W * 32;
  constexpr int KS = D / 16;                  // k16 steps of S^T, and 16-row tiles of O^T
  constexpr int LD = E4M3 ? D / 32 : D / 16;  // ldmatrix.x4 per 16 rows
  constexpr int LPP = C::kRow / 32;           // of these, per 128-byte part
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[W][ST];
  __shared__ int4 head[W][ST];
  __shared__ int64_t sums[T];
  __shared__ int64_t wsum[W];
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  grid_launch_dependents();
  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();
    if (warp == 0) prefetch_tmap(&kmap), prefetch_tmap(&vmap);
  }

  // Sum the tiles of all requests: thread i takes requests [i*per, (i+1)*per).
  const int per = (a.n + T - 1) / T, r_lo = min(tid * per, a.n), r_hi = min(r_lo + per, a.n);
  int64_t mine = 0;
  bool bad = false;
  for (int r = r_lo; r < r_hi; ++r) {
    int len, start, t0, t1;
    span_of<TILE>(a, r, len, start, t0, t1);
    mine += t1 - t0;
    bad |= a.lens[r] > len;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) incl += wsum[w];
    total += wsum[w];
  }
  sums[tid] = incl;
  if (blockIdx.x == 0) {
    if (bad) set_device_error(a.err, kDevErrBadPage);
    int64_t at = incl - mine;
    for (int r = r_lo; r < r_hi; ++r) {
      int len, start, t0, t1;
      span_of<TILE>(a, r, len, start, t0, t1);
      p.prefix[r] = at;
      at += t1 - t0;
    }
    if (tid == T - 1) p.prefix[a.n] = total;
  }
  __syncthreads();

  // This warp's run of tiles [first, first + todo).
  const int64_t tiles = total * p.items, run = run_of(tiles, p.warps);
  const int64_t gw = (int64_t)blockIdx.x * W + warp, first = gw * run;
  if (first >= tiles) return;
  int64_t to_issue = min(run, tiles - first), to_do = to_issue;
  int r, item, t, t0, t1, start, len;
  {
    const int64_t y = first / p.items;
    int lo = 0, hi = T - 1;  // the first thread whose inclusive sum exceeds y
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] > y) hi = mid;
      else lo = mid + 1;
    }
    int64_t at = lo ? sums[lo - 1] : 0;
    for (r = lo * per;; ++r) {
      span_of<TILE>(a, r, len, start, t0, t1);
      if (at + (t1 - t0) > y) break;
      at += t1 - t0;
    }
    const int64_t rem = first - at * p.items;
    item = (int)(rem / (t1 - t0));
    t = t0 + (int)(rem - (int64_t)item * (t1 - t0));
  }

  uint8_t *ring = smem + warp * C::kRing;
  uint8_t *scales = smem + W * C::kRing + warp * C::kScaleRing;  // used for e4m3 only

  // ---- producer: every lane tracks the next tile, lane 0 issues its copies.
  // Lanes hold 32 table entries from page index tb on, and the 32 after them.
  int tb = 0, entry = 0, entry2 = 0;
  const auto table_at = [&](int i) {
    return i < a.max_pages ? a.table[r * a.ldt + i] : 0;
  };
  const auto fetch_table = [&]() {
    tb = (t * TILE) >> p.page_shift;
    entry = table_at(tb + lane);
    entry2 = table_at(tb + 32 + lane);
  };
  fetch_table();
  bool piece_new = true, from_start = false;
  const int box_bytes = p.box_rows * D * C::kEs;
  const auto issue = [&](int slot) {
    const int pos0 = t * TILE;
    const int hd = item / p.groups;
    if (piece_new) from_start = t == t0;
    const int lo = max(start - pos0, 0), hi = max(min(len - pos0, TILE), 0);
    uint32_t valid = (hi >= 32 ? 0xffffffffu : (1u << hi) - 1u) & (0xffffffffu << lo);
    const bool end = t + 1 == t1, last = end || to_issue == 1;
    uint8_t *k = ring + slot * 2 * C::kSide, *v = k + C::kSide;
    uint8_t *ks = scales + slot * 2 * C::kScales, *vs = ks + C::kScales;
    // the boxes that hold a token, and their pages
    const int boxes = TILE >> p.box_shift;
    uint32_t bytes = 0;
    int page[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      page[b] = -1;
      if (b >= boxes) continue;
      const uint32_t mask = (p.box_rows == 32 ? 0xffffffffu : (1u << p.box_rows) - 1u) << (b << p.box_shift);
      if (!(valid & mask)) continue;
      const int i = ((pos0 + (b << p.box_shift)) >> p.page_shift) - tb;
      const int pg = __shfl_sync(0xffffffffu, i < 32 ? entry : entry2, i & 31);
      if (pg < 0 || pg >= a.n_pages) {
        valid &= ~mask;
        if (lane == 0) set_device_error(a.err, kDevErrBadPage);
        continue;
      }
      page[b] = pg;
      bytes += 2 * (box_bytes + (E4M3 ? p.box_rows * 4 : 0));
    }
    if (lane == 0) {
      const bool whole = from_start && end;
      head[warp][slot] = make_int4(r, item | (piece_new ? 1 << 16 : 0) | (last ? 1 << 17 : 0) |
                                          (whole ? 1 << 18 : 0) | (from_start ? 1 << 19 : 0),
                                   (int)valid, 0);
      uint64_t *bar = &full[warp][slot];
      mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (page[b] < 0) continue;
        const int off = (pos0 + (b << p.box_shift)) & (a.page - 1);
        tma_load_5d(k + b * box_bytes, &kmap, bar, 0, off, 0, hd, page[b]);
        tma_load_5d(v + b * box_bytes, &vmap, bar, 0, off, 0, hd, page[b]);
        if (E4M3) {
          const int64_t at = ((int64_t)page[b] * a.kv_heads + hd) * a.page + off;
          bulk_load(ks + b * p.box_rows * 4, a.scale[0] + at, p.box_rows * 4, bar);
          bulk_load(vs + b * p.box_rows * 4, a.scale[1] + at, p.box_rows * 4, bar);
        }
      }
    }
    // next tile
    --to_issue;
    piece_new = end;
    if (!end) {
      ++t;
      if (((t * TILE) >> p.page_shift) - tb >= 32) {
        tb += 32;
        entry = entry2;
        entry2 = table_at(tb + 32 + lane);
      }
    } else if (to_issue > 0) {
      if (++item == p.items) {
        item = 0;
        t0 = t1;
        while (t0 >= t1 && r + 1 < a.n) {
          ++r;
          span_of<TILE>(a, r, len, start, t0, t1);
        }
      }
      t = t0;
      fetch_table();
    }
  };

  // ---- consumer
  const int g = lane >> 2, tq = lane & 3;
  uint32_t qf[KS][NQ][2];
  float qs[NQ][2];  // score factor of the thread's two heads per n-tile
  State<D, NQ> s;
  int cur_r = 0, cur_item = 0;
  const auto start_piece = [&]() {
    const int kvh = cur_item / p.groups, q0 = (cur_item - kvh * p.groups) * 8 * NQ;
    const float f = a.softmax_scale * 1.4426950408889634f;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const int q = q0 + 8 * j + g;
      const bool in = q < p.group_size;
      const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + cur_r * a.ldq +
                                 (int64_t)(kvh * p.group_size + (in ? q : 0)) * a.ldq_head;
      if (!E4M3) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            qf[ks][j][h] = in ? *reinterpret_cast<const uint32_t *>(src + 16 * ks + 8 * h + 2 * tq) : 0u;
        qs[j][0] = qs[j][1] = f;
      } else {
        // values 16 ks + 4t .. + 3 of the row: the order in which ldmatrix on
        // 8-bit rows and the conversions give K
        uint2 w[KS];
        float amax = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          w[ks] = in ? *reinterpret_cast<const uint2 *>(src + 16 * ks + 4 * tq) : make_uint2(0u, 0u);
          amax = fmaxf(fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[ks].x << 16)), fabsf(__uint_as_float(w[ks].x & 0xffff0000u)))),
                       fmaxf(fabsf(__uint_as_float(w[ks].y << 16)), fabsf(__uint_as_float(w[ks].y & 0xffff0000u))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^(14 - exponent of amax): the row's largest value lands in [2^14, 2^15)
        const int e = (int)((__float_as_uint(amax) >> 23) & 255);
        const int up = min(max(127 + 14 - (e - 127), 1), 254);
        const float scale = amax > 0.f && e < 255 ? __uint_as_float((uint32_t)up << 23) : 1.f;
        const float back = f / scale;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[ks][j][0] = pack_f16(__uint_as_float(w[ks].x << 16) * scale, __uint_as_float(w[ks].x & 0xffff0000u) * scale);
          qf[ks][j][1] = pack_f16(__uint_as_float(w[ks].y << 16) * scale, __uint_as_float(w[ks].y & 0xffff0000u) * scale);
        }
        qs[j][0] = __shfl_sync(0xffffffffu, back, 8 * tq);
        qs[j][1] = __shfl_sync(0xffffffffu, back, 8 * tq + 4);
      }
      s.m[j][0] = s.m[j][1] = -INFINITY;
      s.l[j][0] = s.l[j][1] = 0.f;
#pragma unroll
      for (int dt = 0; dt < KS; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s.o[dt][j][i] = 0.f;
    }
  };

  // ldmatrix row of this lane: token (lane & 7) + 8 ((lane >> 3) & 1) of 16,
  // 16-byte chunk 2 i + (lane >> 4) of the row, swizzled by the token.
  const int row = lane & 15;
  const uint32_t swz = C::kRow == 128 ? (lane & 7) : ((lane >> 1) & 3);
  uint32_t chunk[LPP];
#pragma unroll
  for (int i = 0; i < LPP; ++i) chunk[i] = (uint32_t)row * C::kRow + (((2 * i + (lane >> 4)) ^ swz) << 4);
  const uint32_t part_stride = p.box_rows * C::kRow;
  const uint32_t mt_stride = p.box_rows == 16 ? 16 * D * C::kEs : 16 * C::kRow;

  for (int i = 0; i < ST && to_issue > 0; ++i) issue(i);
  __syncwarp();
  int slot = 0;
  uint32_t phase = 0;
  for (; to_do > 0; --to_do) {
    const int4 hd = head[warp][slot];
    const uint32_t valid = (uint32_t)hd.z;
    if (hd.y & (1 << 16)) {  // a piece begins: its q is fetched while its first tile arrives
      cur_r = hd.x, cur_item = hd.y & 0xffff;
      start_piece();
    }
    if (!mbar_wait(&full[warp][slot], phase, a.err)) {
      // copies still under way get the same time to land before the CTA ends
      if (lane == 0) drain_ring(full[warp], ST, slot, phase, (int)min(to_do - to_issue, (int64_t)ST));
      __syncwarp();
      return;
    }
    uint8_t *kt = ring + slot * 2 * C::kSide;
    const uint32_t kb = smem_u32(kt), vb = kb + C::kSide;

    // S^T, each 16 x 8 tile as the sum of CH chains of products (a chain waits
    // for its previous product; four chains in all keep the tensor pipe fed)
    constexpr int CH = MT * NQ >= 4 ? 1 : 4 / (MT * NQ);
    float z[MT][NQ][4];
    {
      float zc[CH][MT][NQ][4];
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < NQ; ++j) zc[c][mt][j][0] = zc[c][mt][j][1] = zc[c][mt][j][2] = zc[c][mt][j][3] = 0.f;
#pragma unroll
      for (int i = 0; i < LD; ++i)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t k4[4];
          ldsm(k4, kb + mt * mt_stride + (i / LPP) * part_stride + chunk[i % LPP]);
          if (!E4M3) {
#pragma unroll
            for (int j = 0; j < NQ; ++j)
              mma_bf16(zc[i % CH][mt][j], k4[0], k4[1], k4[2], k4[3], qf[i][j][0], qf[i][j][1]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_f16(k4[2 * h], a0, a2);
              e4m3x4_f16(k4[2 * h + 1], a1, a3);
#pragma unroll
              for (int j = 0; j < NQ; ++j)
                mma_f16(zc[(2 * i + h) % CH][mt][j], a0, a1, a2, a3, qf[2 * i + h][j][0], qf[2 * i + h][j][1]);
            }
          }
        }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            z[mt][j][x] = zc[0][mt][j][x];
#pragma unroll
            for (int c = 1; c < CH; ++c) z[mt][j][x] += zc[c][mt][j][x];
          }
    }

    // scores in base 2; tokens that are not there get -infinity
    const bool partial = valid != (TILE == 32 ? 0xffffffffu : 0xffffu);
    float lv[MT][2], rv[MT][2];
    const float *ksc = reinterpret_cast<const float *>(scales + slot * 2 * C::kScales), *vsc = ksc + TILE;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float ks = 1.f;
        if (E4M3) {
          ks = ksc[mt * 16 + 8 * h + g];
          // (a floor of 2^-96 keeps the sum of 1 / scale finite for any number of tokens)
          const float vs = fmaxf(vsc[mt * 16 + 8 * h + g], 1.2621774e-29f);
          lv[mt][h] = lg2(vs);
          rv[mt][h] = rcp_approx(vs);
        }
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float &x = z[mt][j][2 * h + c];
            x = E4M3 ? fmaf(x * qs[j][c], ks, lv[mt][h]) : x * qs[j][c];
          }
      }
    if (partial) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!(valid >> (mt * 16 + 8 * h + g) & 1u)) {
#pragma unroll
            for (int j = 0; j < NQ; ++j) z[mt][j][2 * h] = z[mt][j][2 * h + 1] = -INFINITY;
          }
      // zero the V rows that are not there: 0 * (whatever they hold) must be 0
      for (int i = lane; i < C::kSide / 16; i += 32) {
        const int in_box = i % (box_bytes / 16);
        const int tok = (i / (box_bytes / 16) << p.box_shift) + (in_box * 16 / C::kRow & (p.box_rows - 1));
        if (!(valid >> tok & 1u)) *reinterpret_cast<uint4 *>(kt + C::kSide + i * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
    }

    // running maximum
    bool grew = false;
    float mn[NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = fmaxf(z[0][j][c], z[0][j][2 + c]);
#pragma unroll
        for (int mt = 1; mt < MT; ++mt) x = fmaxf(x, fmaxf(z[mt][j][c], z[mt][j][2 + c]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        mn[j][c] = fmaxf(s.m[j][c], x);
        grew |= mn[j][c] > s.m[j][c];
      }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float f = mn[j][c] == s.m[j][c] ? 1.f : ex2(s.m[j][c] - mn[j][c]);
          s.m[j][c] = mn[j][c];
          s.l[j][c] *= f;
#pragma unroll
          for (int dt = 0; dt < KS; ++dt) s.o[dt][j][c] *= f, s.o[dt][j][2 + c] *= f;
        }
    }

    // weights, and the P^T fragments
    uint32_t ph[MT][NQ][2], pl[MT][NQ][2];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const float m0 = s.m[j][0] == -INFINITY ? 0.f : s.m[j][0], m1 = s.m[j][1] == -INFINITY ? 0.f : s.m[j][1];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float w0 = ex2(z[mt][j][2 * h] - m0), w1 = ex2(z[mt][j][2 * h + 1] - m1);
          if (E4M3) {
            s.l[j][0] = fmaf(w0, rv[mt][h], s.l[j][0]);
            s.l[j][1] = fmaf(w1, rv[mt][h], s.l[j][1]);
            ph[mt][j][h] = transpose8(pack_f16(w0 * kUp, w1 * kUp));
          } else {
            s.l[j][0] += w0;
            s.l[j][1] += w1;
            const uint32_t hi = pack_bf16(w0, w1);
            ph[mt][j][h] = transpose8(hi);
            pl[mt][j][h] = transpose8(pack_bf16(w0 - __uint_as_float(hi << 16), w1 - __uint_as_float(hi & 0xffff0000u)));
          }
        }
    }

    // O^T.  The products of two d-tiles are interleaved: hi and lo of one tile
    // add to the same registers.
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (!E4M3) {
#pragma unroll
        for (int i = 0; i < LD; i += 2) {
          uint32_t v4[2][4];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            ldsm_t(v4[x], vb + mt * mt_stride + ((i + x) / LPP) * part_stride + chunk[(i + x) % LPP]);
#pragma unroll
          for (int lo = 0; lo < 2; ++lo)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int j = 0; j < NQ; ++j)
                mma_bf16(s.o[i + x][j], v4[x][0], v4[x][2], v4[x][1], v4[x][3],
                         lo ? pl[mt][j][0] : ph[mt][j][0], lo ? pl[mt][j][1] : ph[mt][j][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < LD; ++i) {
          uint32_t v4[4];
          ldsm_t(v4, vb + mt * mt_stride + (i / LPP) * part_stride + chunk[i % LPP]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // bytes (key 2t: d 2g, 2g + 1; key 2t + 1: the same) to fp16 pairs
            // of the two keys for d 2g and for d 2g + 1
            uint32_t a0, a1, a2, a3;
            e4m3x4_f16(__byte_perm(v4[2 * h], 0, 0x3120), a0, a1);
            e4m3x4_f16(__byte_perm(v4[2 * h + 1], 0, 0x3120), a2, a3);
#pragma unroll
            for (int j = 0; j < NQ; ++j) mma_f16(s.o[2 * i + h][j], a0, a1, a2, a3, ph[mt][j][0], ph[mt][j][1]);
          }
        }
      }
    }
    __syncwarp();
    if (to_issue > 0) issue(slot);
    __syncwarp();  // the tile's header, written by lane 0, is read before its barrier
    if (++slot == ST) slot = 0, phase ^= 1u;

    if (hd.y & (1 << 17)) {  // the piece ends
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          s.l[j][c] += __shfl_xor_sync(0xffffffffu, s.l[j][c], 4);
          s.l[j][c] += __shfl_xor_sync(0xffffffffu, s.l[j][c], 8);
          s.l[j][c] += __shfl_xor_sync(0xffffffffu, s.l[j][c], 16);
        }
      if (hd.y & (1 << 18)) {
        write_out<D, E4M3, NQ>(p, s, cur_r, cur_item, 0, 0, D, true);
      } else {
        float4 *to = reinterpret_cast<float4 *>(p.slots + (2 * gw + (hd.y >> 19 & 1)) * (int64_t)slot_floats<D, NQ>()) + lane;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
#pragma unroll
          for (int dt = 0; dt < KS; ++dt)
            to[(dt * NQ + j) * 32] = make_float4(s.o[dt][j][0], s.o[dt][j][1], s.o[dt][j][2], s.o[dt][j][3]);
          to[(KS * NQ + j) * 32] = make_float4(s.m[j][0], s.m[j][1], s.l[j][0], s.l[j][1]);
        }
      }
    }
  }
}

// Joins the pieces of the items that several warps share, and writes the items
// without tokens.  A warp joins one unit, 16 of an item's D values of 8 heads;
// `ways` warps of a CTA take a unit's pieces in turn.  Item i covers tiles [A, B)
// of the list, so its pieces are those of warps A / run .. (B-1) / run; the
// first of them is its warp's slot 1 (it starts the item), the others are slot 0.
constexpr int kJoinWarps = 8;

template <int D, bool E4M3, int NQ>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ Params p, int ways) {
  constexpr int KS = D / 16;
  __shared__ float4 part[kJoinWarps][2][32];
  const AttnArgs &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = kJoinWarps / ways, way = warp / units;
  const int64_t unit = (int64_t)blockIdx.x * units + warp % units;
  const int64_t it = unit / (KS * NQ);
  const int dj = (int)(unit - it * (KS * NQ)), dt = dj / NQ, j = dj % NQ;
  const int r = (int)(it / p.items), item = (int)(it - (int64_t)r * p.items);
  grid_dependency_wait();
  int64_t w0 = 0, w1 = 0, nt = 1;  // what is left so has nothing to join
  if (r < a.n) {
    const int64_t before = p.prefix[r], total = p.prefix[a.n] * p.items;
    nt = p.prefix[r + 1] - before;
    const int64_t A = before * p.items + item * nt, run = run_of(total, p.warps);
    if (total <= INT32_MAX) {  // 64-bit divisions take as long as the loads
      w0 = (uint32_t)A / (uint32_t)run;
      w1 = nt ? (uint32_t)(A + nt - 1) / (uint32_t)run : w0;
    } else {
      w0 = A / run;
      w1 = nt ? (A + nt - 1) / run : w0;
    }
  }
  const bool joined = w1 > w0 || nt == 0;
  if (ways == 1 && !joined) return;
  State<16, 1> s;
  s.m[0][0] = s.m[0][1] = -INFINITY;
  s.l[0][0] = s.l[0][1] = 0.f;
  s.o[0][0][0] = s.o[0][0][1] = s.o[0][0][2] = s.o[0][0][3] = 0.f;
  const auto add = [&](float4 o, float4 ml) {
    const float m2[2] = {ml.x, ml.y}, l2[2] = {ml.z, ml.w}, o2[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float m = fmaxf(s.m[0][c], m2[c]);
      const float f = s.m[0][c] == m ? 1.f : ex2(s.m[0][c] - m), f2 = m2[c] == m ? 1.f : ex2(m2[c] - m);
      s.m[0][c] = m;
      s.l[0][c] = s.l[0][c] * f + l2[c] * f2;
      s.o[0][0][c] = s.o[0][0][c] * f + o2[c] * f2;
      s.o[0][0][2 + c] = s.o[0][0][2 + c] * f + o2[2 + c] * f2;
    }
  };
  if (w1 > w0) {
    constexpr int U = 4;  // pieces loaded at a time
    for (int64_t w = w0 + way; w <= w1; w += U * ways) {
      float4 o[U], ml[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t x = min(w + u * ways, w1);
        const float4 *from = reinterpret_cast<const float4 *>(p.slots + (2 * x + (x == w0)) * (int64_t)slot_floats<D, NQ>()) + lane;
        o[u] = from[(dt * NQ + j) * 32], ml[u] = from[(KS * NQ + j) * 32];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (w + u * ways <= w1) add(o[u], ml[u]);
    }
  }
  for (int half = ways / 2; half; half /= 2) {  // the upper half of the ways to the lower
    if (way >= half && way < 2 * half) {
      part[warp][0][lane] = make_float4(s.o[0][0][0], s.o[0][0][1], s.o[0][0][2], s.o[0][0][3]);
      part[warp][1][lane] = make_float4(s.m[0][0], s.m[0][1], s.l[0][0], s.l[0][1]);
    }
    __syncthreads();
    if (way < half) add(part[warp + half * units][0][lane], part[warp + half * units][1][lane]);
  }
  if (!joined || way) return;
  write_out<16, E4M3, 1>(p, s, r, item, j, dt * 16, D, dt == 0);
}

int query_tiles(int dim, int group) { return group > 8 && dim <= 128 ? 2 : 1; }
size_t slot_bytes(int dim, int nq) { return (size_t)32 * nq * (dim / 16 * 4 + 4) * 4; }
size_t prefix_bytes(int n) { return ((size_t)(n + 1) * 8 + 255) / 256 * 256; }

template <int D, bool E4M3, int NQ>
cudaError_t launch_cfg(Params &p, cudaStream_t stream) {
  using C = Cfg<D, E4M3>;
  const AttnArgs &a = p.a;
  const DeviceFacts *f = device_facts();
  static SmemLimit limit;
  cudaError_t e = raise_smem_limit(limit, paged_attn_kernel<D, E4M3, NQ>, C::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap maps[2];
  p.box_rows = a.page < C::kTile ? a.page : C::kTile;
  p.box_shift = p.box_rows == 32 ? 5 : 4;
  p.page_shift = 31 - __builtin_clz((unsigned)a.page);
  const int inner = C::kRow / C::kEs;
  const uint64_t dims[5] = {(uint64_t)inner, (uint64_t)a.page, (uint64_t)C::kParts, (uint64_t)a.kv_heads, (uint64_t)a.n_pages};
  const uint64_t strides[4] = {(uint64_t)a.token_stride * C::kEs, (uint64_t)C::kRow, (uint64_t)a.head_stride * C::kEs,
                               (uint64_t)a.page_stride * C::kEs};
  const uint32_t box[5] = {(uint32_t)inner, (uint32_t)p.box_rows, (uint32_t)C::kParts, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (encode_tiled(&maps[i], E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                     const_cast<void *>(a.cache[i]), dims, strides, box,
                     C::kRow == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  const int grid = f->sm_count < kMaxSms ? f->sm_count : kMaxSms;
  p.warps = (int64_t)grid * C::kWarps;
  paged_attn_kernel<D, E4M3, NQ><<<grid, C::kWarps * 32, C::kSmem, stream>>>(p, maps[0], maps[1]);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // An item has about warps / items pieces; a warp takes up to 8 of them.  (With
  // one CTA per item the join of 16 items of 114 pieces alone took 11 us; 16 ways
  // for every item took 40 us for 256 items of 4.  With up to 4 a warp, 96
  // items of 9 at D 256 took 62.6 us in all, with up to 8 61.1; other shapes the
  // same within 0.6 us.)
  const int64_t items = (int64_t)a.n * p.items, pieces = p.warps / items;
  int ways = 1;
  while (ways < kJoinWarps && ways * 8 < pieces) ways *= 2;
  const int units = kJoinWarps / ways;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((items * (D / 16) * NQ + units - 1) / units));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, join_kernel<D, E4M3, NQ>, p, ways);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, bool E4M3>
cudaError_t launch_nq(Params &p, int nq, cudaStream_t s) {
  if constexpr (D <= 128) {
    if (nq == 2) return launch_cfg<D, E4M3, 2>(p, s);
  }
  return launch_cfg<D, E4M3, 1>(p, s);
}

}  // namespace

size_t paged_attn_workspace_size(int32_t n, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  const int nq = query_tiles(dim, q_heads / (kv_heads < q_heads ? kv_heads : q_heads));
  return prefix_bytes(n) + (size_t)kMaxSms * kMaxWarps * 2 * slot_bytes(dim, nq);
}

cudaError_t launch_paged_attn(const AttnArgs &a, cudaStream_t s) {
  Params p = {};
  p.a = a;
  p.group_size = a.q_heads / a.kv_heads;
  const int nq = query_tiles(a.dim, p.group_size);
  p.heads_per_item = 8 * nq;
  p.groups = (p.group_size + 8 * nq - 1) / (8 * nq);
  p.items = a.kv_heads * p.groups;
  p.prefix = static_cast<int64_t *>(a.workspace);
  p.slots = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + prefix_bytes(a.n));
  const bool e = a.cache_dtype == Q4K_DTYPE_E4M3;
  if (a.dim == 64) return e ? launch_nq<64, true>(p, nq, s) : launch_nq<64, false>(p, nq, s);
  if (a.dim == 128) return e ? launch_nq<128, true>(p, nq, s) : launch_nq<128, false>(p, nq, s);
  return e ? launch_nq<256, true>(p, nq, s) : launch_nq<256, false>(p, nq, s);
}

}  // namespace q4k
