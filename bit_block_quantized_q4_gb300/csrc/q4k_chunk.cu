// q4k_chunk.cu -- attention of each request's new tokens, one or many, over the
// paged cache (q4k_paged_attn_chunk).
//
// "spec: specialized model runtimes", section "Architecture": attention is an
// op of kernel tier T0.
//
// Mathematics.  Token i of a request's m new ones stands at position p = len - m
// + i and sees the tokens max(0, p + 1 - window) .. p.  One pass over the keys
// with a running reference M and sum l, in base 2 (scores carry log2 e):
//   w_j = 2^(z_j - M),  l += w_j,  o += w_j v_j,  out = o / l.
// M is the running maximum, but it follows only when the maximum has grown by
// more than 2^kLazy; then l and o are multiplied by 2^(M - M').  A sum of powers is
// the same whatever its reference, so this costs nothing but kLazy of fp32's
// exponent, and o, which lives in tensor memory, is rarely touched.
//
// Rows.  The query heads of one key head share its keys, so the rows of a
// product are (token, head) pairs: row = token * group + head.  128 of them are a
// query tile; a decode step's single tokens fill a part of one, a prompt all.
//
// Products, both by tcgen05.mma with fp32 accumulators in tensor memory:
//   S[128 rows, TILE keys] = Q K^T    (Q, K from shared memory)
//   O[128 rows, D]        += P V      (P in tensor memory beside S, V from shared memory)
//
// Roles of a CTA's 16 warps, connected by mbarriers:
//   0..3, 4..7  softmax of query tile 0 and 1: a thread owns a row of S
//   8, 10       issue the products, Q K^T and P V.  (Issuing and the waits before it
//               take one warp about as long as the tensor cores take for both.)
//   9, 11       find the work and issue the copies of K; issue the copies of V (TMA, a
//               page each)
//   12..15      fetch Q and prepare what was copied: rows of V that no query sees
//               become zeros (their weights are 0, but 0 times a NaN is not); an e4m3
//               cache is converted to fp16 in place
//
// Work split.  An item is (request, key head, block of rows), its cost its key
// tiles and a fixed cost; every CTA of a persistent grid takes an equal run of the
// list of all items' tiles.  The lengths are on the device, so each CTA sums them
// itself.  A CTA has at most two pieces of items that it shares with others; they
// go to the workspace and a second launch joins them.
//
// What bounds it, measured on replays of a graph (one call after another takes prompts and
// windows 3 to 5% longer).  A prompt of 8191 tokens, 64 / 8 heads x 128, bf16: 750 to 770 us,
// 1449 TFLOP/s, 74% of the library product's rate; the tensor pipe is busy half of the
// time, and the softmax warps take longer for a tile than the products do.  4 chunks
// of 2049 with a window of 4096, 24 / 4 x 256: 606 to 625 us, 62%, the tensor pipe busy 53% of the
// time with tiles of 64 keys, the most that fit beside Q.  8 requests of up to 60000 tokens, 5
// new ones each: 220 us, 92% of the copy rate.  e4m3, 60 requests of up to 16001 tokens,
// three of them with 700 new ones: 914 us; the conversion's warps share the softmax's
// instruction caches and pipes.  45 tokens behind 700: 21 to 22.5 us, a chain of lengths, table,
// tile, products and the join.
// The e4m3 kernels are sensitive to what stands beside their loops (of 120 KB): code that runs
// once per item takes thousands of cycles for its instructions alone, and two such blocks
// more in the softmax took a prompt at head size 64 from 1013 to 1318 us with the same
// registers, warps without an instruction from 1.16 to 2.19 per issue.  So what is rare there
// is kept short and rolled.
//
// Weights as one term.  A second bf16 term would double the products P V and the weights'
// columns, and tensor memory is full at head size 128; the result is rounded to the same
// 8 bits.  (The single-token kernel has two, its products cost nothing there.)
// Tried: scores in halves of 64 columns (prompt 1157 us, not 1036: the shared score buffer
// is free later); four more warps for e4m3 that convert V beside K (1375 us, not 1184);
// two groups of softmax warps for the one query tile of head size 256, its key tiles in turn
// (625 us, not 622).  Kept: K and V copied by a warp each (the 8 requests 233 us, not
// 260; the window 708, not 765); scores of tiles that all rows see entirely do not wait
// for V (220 and 618).
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

constexpr int kMaxSms = 160;     // CTAs that the workspace is sized for
constexpr int kThreads = 512;
constexpr float kLazy = 8.f;     // binary orders that a maximum may grow before M follows
constexpr float kUpBits = 7.f;   // e4m3: weights are stored times 2^7, so that the largest, 2^kLazy more, are below 2^16
// e4m3: no tile's values are divided by less than 2^kLeastLog (rows of zeros have scales of 2^-109).  The sum of weights
// is that of stored ones over this power, at most 2^15 2^80 for each of 2^30 tokens: finite.
// (2^-v_log is a normal number up to 2^kMostLog, where the largest scale becomes 2^6 .. 2^7.)
constexpr int kLeastLog = -80, kMostLog = 121;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr int kRing = 4;         // items on their way

template <int D, bool E4M3>
struct Cfg {
  static constexpr int kNq = D == 256 ? 1 : 2;        // query tiles per block
  // Buffers in tensor memory: O of each query tile; scores, of each query tile (dim
  // 64), of both in turn (128), or of a key tile and the next (256); weights, of
  // each query tile, or of a key tile and the next (256).
  static constexpr int kSBufs = D == 128 ? 1 : 2, kPBufs = 2;
  static constexpr int kTile = D == 256 ? 64 : 128;   // tokens per key tile
  // Registers of a softmax thread; the others have 256 less these.  Measured: dim 128, bf16, 184
  // or 176: prompt 976 or 1040 us; e4m3, 176, 184 or 192: mixed step 926, 910, 920; dim 256, 152
  // or 176: 797 or 808.
  static constexpr int kMoreRegs = D == 256 ? 152 : 184;
  // Cost of an item's start and end, in key tiles, for the shares of the CTAs.  Measured on
  // an 8191-token prompt, bf16, head size 128: 1: 972 us, 2: 916, 4: 813, 5: 786, 6: 807,
  // 8: 835; on 60 requests of e4m3, whose tiles cost more: 1: 929, 2: 926, 3: 922.  (Head sizes
  // 64 and 256 use what was measured at 128.)
  static constexpr int kItemCost = E4M3 ? 3 : 5;
  static constexpr int kParts = D / 64;               // 128-byte parts of a row
  static constexpr int kSide = kTile * D * 2;         // bytes of a tile of K or V
  static constexpr int kStages = D == 64 ? 4 : 2;     // of K, and of V
  static constexpr int kQ = 128 * D * 2;              // bytes of a query tile
  static constexpr int kRows = 128 * kNq;             // rows of a block
  static constexpr int kSCol = kNq * D;               // first columns of scores, of weights
  static constexpr int kPCol = kSCol + kSBufs * kTile;
  static constexpr int kCols = 512;
  static constexpr int kEs = E4M3 ? 1 : 2;
  // Rows of Q that a lane fetches at once, and pieces that it converts (e4m3).  This runs once
  // per item, and its instructions push out others'.  Prompt, size 64: 4 and all 8: 1260 us, 4
  // and 2: 1181, 1 and 1: 1095; size 128: 4 and all 16: 1357, 4 and 2: 1261, 1 and 1: 1265; window,
  // size 256: 4 and 2: 1284, 1 and 1: 1340.
  static constexpr int kQRows = E4M3 && D == 64 ? 1 : 4, kQPieces = D == 64 ? 1 : 2;
  static constexpr int kRaw = kTile * D;              // bytes of an e4m3 tile
  static constexpr int kRawParts = D == 256 ? 2 : 1;  // in which its rows are copied
  // Q | K stages | V stages | e4m3: per stage of V the scales of K and V
  static constexpr int kKAt = kNq * kQ, kVAt = kKAt + kStages * kSide;
  static constexpr int kScaleAt = kVAt + kStages * kSide;
  static constexpr int kSmem = kScaleAt + (E4M3 ? kStages * 2 * kTile * 4 : 0) + 1024;
  static_assert(kPCol + kPBufs * kTile / 2 <= kCols, "O, S and P fit tensor memory");
};

struct Params {
  AttnArgs a;
  int64_t tokens;     // of q and out
  const int64_t *cu;
  int group;          // query heads per key head
  FastDiv by_group;
  int box_rows, box_shift, page_shift;
  int slot_rows;      // rows of a workspace slot, a multiple of 32
  int4 *desc;         // per CTA: the item that it starts and does not end
  float *slots;
};

// ------------------------------------------------------------------ work list

// A request's geometry.
struct Req {
  int tok0, m, pos0, rows;  // first token of the step, their number, position of the first, rows per key head
};
__device__ __forceinline__ Req request(const Params &p, int r, bool &bad) {
  const int64_t c0 = p.cu[r], c1 = p.cu[r + 1];
  const bool ok = c0 >= 0 && c1 >= c0 && c1 <= p.tokens;
  const int told = max(p.a.lens[r], 0);
  Req q;
  q.tok0 = ok ? (int)c0 : 0;
  q.m = ok ? (int)(c1 - c0) : 0;
  q.pos0 = told - q.m;
  q.rows = q.m * p.group;
  bad |= !ok || (q.m > 0 && told > p.a.max_pages * p.a.page);
  return q;
}
// First token that a position sees; what follows its last one.  Tokens past the
// table are absent.
__device__ __forceinline__ int first_seen(const AttnArgs &a, int pos) {
  return a.window > 0 && pos >= a.window ? pos + 1 - a.window : 0;
}
__device__ __forceinline__ int end_seen(const AttnArgs &a, int pos) {
  return min(max(pos + 1, 0), a.max_pages * a.page);
}
// The key tiles [t0, t1) of rows [row0, row0 + rows) of a request.
template <int TILE>
__device__ __forceinline__ void tiles_of(const Params &p, const Req &q, int row0, int rows, int &t0, int &t1) {
  const int lo = first_seen(p.a, q.pos0 + (int)p.by_group.div(row0));
  const int hi = end_seen(p.a, q.pos0 + (int)p.by_group.div(row0 + rows - 1));
  t0 = lo / TILE;
  t1 = hi > lo ? (hi + TILE - 1) / TILE : t0;
}
template <int TILE, int ROWS, int ITEM_COST>
__device__ __forceinline__ int block_cost(const Params &p, const Req &q, int b) {
  int t0, t1;
  tiles_of<TILE>(p, q, b * ROWS, min(ROWS, q.rows - b * ROWS), t0, t1);
  return t1 - t0 + ITEM_COST;
}

// What all roles know of an item.
struct Item {
  int r, head, row0, rows;  // rows < 0: there are no more items
  int tok0, pos0;
  int t0, n;                // its first key tile here, and their number
  int lo, hi;               // tokens that any of its rows sees
  int full_lo, full_hi;     // tokens in between are seen by all rows
  int kind;                 // 0: whole, 1: starts the item (slot 1), 2: does not (slot 0)
};

// ---------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// D[tmem] (+)= A[smem desc or tmem] * B[smem desc], kind::f16, issued by the lanes
// whose `lead` is not 0.  (A predicate and not a branch, so that the descriptors
// stay uniform values: 8 products with both operands in shared memory issue in 126
// cycles, in a branch of one lane in 365; with one in tensor memory 60 and 244.
// They run for 512.)
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
// tc_commit by the lanes whose `lead` is not 0.
__device__ __forceinline__ void tc_commit_if(uint64_t *bar, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)), "r"(lead)
      : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p;
}
#define Q4K_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define Q4K_V8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 lanes x 32 bits, 32 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld_x32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : Q4K_R8(r, 0), Q4K_R8(r, 8), Q4K_R8(r, 16), Q4K_R8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(addr),
      Q4K_V8(r, 0), Q4K_V8(r, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st_x4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// A wait by a whole warp, whose lanes stay together; false after the time limit.
// (Without a call, which would cost every role its registers.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned *err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  do {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  } while (!__any_sync(0xffffffffu, global_ns() - t0 > kWaitLimitNs));
  set_device_error(err, kDevErrTimeout);
  return false;
}
// Two waits, whose first polls go out together.
__device__ __forceinline__ bool warp_wait2(uint64_t *bar, uint32_t parity, uint64_t *bar2, uint32_t parity2, unsigned *err) {
  const bool x = mbar_try_wait(bar, parity), y = mbar_try_wait(bar2, parity2);
  if (__all_sync(0xffffffffu, x && y)) return true;
  return warp_wait(bar, parity, err) && warp_wait(bar2, parity2, err);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// A barrier of the 128 threads of a warpgroup; true if `ok` was true for all.
// (Every warp passes it whatever happened to it, so that none is left behind.)
__device__ __forceinline__ bool group_and(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(all)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return all != 0;
}
// Descriptor of V as the second operand: [token][64 values] rows of 128 bytes,
// swizzled, 8 tokens per 1024 bytes; the next 64 values of D `part` bytes on.
__device__ __forceinline__ uint64_t sdesc_v(uint32_t addr, uint32_t part) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)((part >> 4) & 0x3FFFu) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
// Instruction descriptor: fp32 accumulators, operands bf16 or fp16, the second
// one with its rows along N (K-major) or along K (transposed).
__host__ __device__ constexpr uint32_t idesc_of(bool bf16, bool transposed, int n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (transposed ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Four e4m3 values to two fp16 pairs, exact.
__device__ __forceinline__ uint2 e4m3x4_f16(uint32_t w) {
  uint2 d;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(d.x), "=r"(d.y) : "r"(w));
  return d;
}

// ------------------------------------------------------------------- the kernel

struct Bars {
  uint64_t item_full[kRing], item_empty[kRing];
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[4], k_ready[4], k_empty[4], v_full[4], v_known[4], v_ready[4], v_empty[4];
  uint64_t s_full[2], s_free[2];  // scores: of a query tile (dim 256: of a buffer); buffers
  uint64_t p_full[2], o_done[2];  // weights and their products, by buffer of weights
};
// Of a stage of V: 16-token pieces that are absent, tokens whose values are not
// finite; e4m3: the binary logarithm of what the values were divided by (and kOwn in absent where
// some tokens' were divided by more or less), and the largest one so far of tokens that all rows see.
struct __align__(16) VInfo {
  uint32_t bad[4], absent;
  float v_log, v_run;
};
constexpr uint32_t kOwn = 0x80000000u;

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, E4M3>;
  constexpr int TILE = C::kTile, ROWS = C::kRows, ST = C::kStages, NQ = C::kNq;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars bars;
  __shared__ VInfo vinfo[4];
  __shared__ uint32_t gone[8];  // 16-token pieces that are absent, of the last eight tiles of K
  __shared__ uint32_t v_absent[4], e_max[2][4];  // of a stage of V; largest exponents of a tile's scales by warp, two tiles in turn
  __shared__ __align__(16) int16_t v_own[E4M3 ? 4 : 1][128];  // of a stage of V: orders by which a token's values were divided besides
  __shared__ Item items[kRing];
  __shared__ float q_scale[kRing][ROWS];  // e4m3: what the rows' scores are multiplied by, of the items on their way
  __shared__ int64_t sums[kThreads], wsum[kThreads / 32];
  __shared__ uint32_t tmem_slot;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  grid_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(&bars.item_full[i], 1), mbar_init(&bars.item_empty[i], 2 + 4 * NQ + 1 + 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 4), mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.s_full[i], 1), mbar_init(&bars.s_free[i], 4), mbar_init(&bars.p_full[i], 4), mbar_init(&bars.o_done[i], 1);
    }
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.k_full[i], 1), mbar_init(&bars.k_ready[i], 4), mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 1), mbar_init(&bars.v_known[i], 4), mbar_init(&bars.v_ready[i], 4), mbar_init(&bars.v_empty[i], 1);
    }
    fence_mbar_init();
    prefetch_tmap(&kmap), prefetch_tmap(&vmap);
  }
  if (warp == 8) {
    tmem_alloc(&tmem_slot, C::kCols);
    tmem_relinquish();
  }

  // Sum the costs of all requests: thread i takes requests [i * per, (i + 1) * per).
  const int per = (a.n + kThreads - 1) / kThreads, r_lo = min(tid * per, a.n), r_hi = min(r_lo + per, a.n);
  bool bad = false;
  int64_t mine = 0;
  const auto cost_of = [&](int r) {
    const Req q = request(p, r, bad);
    int64_t c = 0;
    for (int b = 0; b * ROWS < q.rows; ++b) c += block_cost<TILE, ROWS, C::kItemCost>(p, q, b);
    return c * a.kv_heads;
  };
  for (int r = r_lo; r < r_hi; ++r) mine += cost_of(r);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) incl += wsum[w];
    total += wsum[w];
  }
  sums[tid] = incl;
  if (blockIdx.x == 0 && bad) set_device_error(a.err, kDevErrBadPage);
  __syncthreads();
  const uint32_t tmem = tmem_slot;
  const int64_t run = max((total + gridDim.x - 1) / gridDim.x, (int64_t)1);
  const int64_t u0 = min((int64_t)blockIdx.x * run, total), u1 = min(u0 + run, total);
  bool ok = true;

  // The ring of items, as every role but the copying one reads it.
  int it = 0;
  const auto next_item = [&](Item &x) {  // false: there are no more, or the wait ran out
    ok = warp_wait(&bars.item_full[it % kRing], (uint32_t)(it / kRing) & 1u, a.err);
    if (ok) x = items[it % kRing];
    return ok && x.rows >= 0;
  };
  const auto free_item = [&]() {  // by one lane of the warp
    mbar_arrive(&bars.item_empty[it % kRing]);
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kMoreRegs));
    // ---------------------------------------------------------------- softmax
    const int t = warp >> 2, row_in = 32 * (warp & 3) + lane, row_t = 128 * t + row_in;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t o_at = tmem + lanes + t * D, s_col = tmem + lanes + C::kSCol, p_col = tmem + lanes + C::kPCol;
    // scores are multiplied by -1 or 0 first where the scale is not positive (e4m3: q was)
    const float scale = (a.softmax_scale == 0.f ? 1.f : fabsf(a.softmax_scale)) * kLog2e;
    const float sign = a.softmax_scale < 0.f ? -1.f : 0.f;
    const bool positive = a.softmax_scale > 0.f;
    int tiles = 0, mine_t = 0, taken = 0;  // key tiles of this CTA so far, those of query tile t, and its items
    // The g-th product P V of this query tile is complete.  A wait tells phases apart
    // by their parity alone, so it must not come when the phase before may be missing
    // or the one after be there.  Each tile waits for the product that used its buffer
    // of weights last; and the next one in that buffer waits for weights that this
    // warp has not written yet.
    const auto values_done = [&](int g) {
      return warp_wait(&bars.o_done[NQ == 1 ? g & 1 : t], (uint32_t)(NQ == 1 ? g >> 1 : g) & 1u, a.err);
    };
    const auto weights_free = [&](int g) { return g < (NQ == 1 ? 2 : 1) || values_done(g - (NQ == 1 ? 2 : 1)); };
    Item x;
    while (t < NQ && ok && next_item(x)) {
      const bool active = x.rows > 128 * t, used = x.rows > 128 * t + 32 * (warp & 3), live = row_t < x.rows;
      // this row's token, its head in the group, and the tokens that it sees
      const int row = x.row0 + row_t, tok = (int)p.by_group.div(row), at_pos = x.pos0 + tok;
      const int seen_lo = live ? first_seen(a, at_pos) : x.lo, seen_hi = live ? end_seen(a, at_pos) : x.hi;
      float m = -INFINITY, l = 0.f;
      bool poisoned = false;
      float sc = scale;
      float v_seen = -1000.f;  // e4m3: the largest v_log of this row's where tokens have ones of their own
      uint32_t wide = 0u;      // kOwn once that, of a row of this warp, is so large that another tile's may need it
      for (int j = 0; active && j < x.n && ok; ++j) {
        const int g = mine_t + j, buf = NQ == 1 ? g & 1 : t;
        const int vs = (tiles + j) % ST;
        if (!(ok = warp_wait(&bars.s_full[buf], (uint32_t)(NQ == 1 ? g >> 1 : g) & 1u, a.err))) break;
        tc_fence_after();
        const uint32_t s_at = s_col + (C::kSBufs == 1 ? 0 : buf) * TILE, at = p_col + buf * (TILE / 2);
        uint32_t s[TILE];
        if (used) {
#pragma unroll
          for (int c = 0; c < TILE; c += 32) tmem_ld_x32(s_at + c, s + c);
          tmem_ld_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_free[C::kSBufs == 1 ? 0 : buf]);
        // The buffer of weights is free, and O complete but for this tile; and what VInfo
        // says of V is there, where it is needed: bf16 tiles that all rows see entirely are
        // only multiplied.
        const int pos = (x.t0 + j) * TILE;
        const bool whole = !E4M3 && pos >= x.full_lo && pos + TILE <= x.full_hi && gone[(tiles + j) & 7] == 0;
        if (!(ok = weights_free(g) && (whole || warp_wait(E4M3 ? &bars.v_known[vs] : &bars.v_ready[vs], (uint32_t)((tiles + j) / ST) & 1u, a.err)))) break;
        if (used) {
          if (E4M3 && j == 0) sc = scale * q_scale[taken % kRing][row_t];
          if (!E4M3 && !positive) {
#pragma unroll
            for (int c = 0; c < TILE; ++c) s[c] = __float_as_uint(__uint_as_float(s[c]) * sign);
          }
          if (E4M3) {  // the keys' scales: the same for all rows
            const float4 *ks = reinterpret_cast<const float4 *>(smem + C::kScaleAt + vs * 2 * TILE * 4);
#pragma unroll
            for (int c = 0; c < TILE; c += 4) {
              const float4 k4 = ks[c / 4];
              const float2 x0 = __fmul2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), make_float2(k4.x, k4.y));
              const float2 x1 = __fmul2_rn(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), make_float2(k4.z, k4.w));
              s[c] = __float_as_uint(x0.x), s[c + 1] = __float_as_uint(x0.y), s[c + 2] = __float_as_uint(x1.x), s[c + 3] = __float_as_uint(x1.y);
            }
          }
          const uint32_t absent = whole ? 0u : vinfo[vs].absent;
          const int lo = seen_lo - pos, hi = seen_hi - pos;
          const uint32_t *bad_words = vinfo[vs].bad;
          uint32_t some = absent;
#pragma unroll
          for (int w = 0; w < TILE / 32; ++w) some |= whole ? 0u : bad_words[w];
          if (!whole && __any_sync(0xffffffffu, lo > 0 || hi < TILE || some)) {
#pragma unroll
            for (int w = 0; w < TILE / 32; ++w) {  // the tokens that this row sees, as bits
              const int lo_w = min(max(lo - 32 * w, 0), 32), hi_w = min(max(hi - 32 * w, 0), 32);
              uint32_t sees = (hi_w == 32 ? 0xffffffffu : (1u << hi_w) - 1u) & (lo_w == 32 ? 0u : 0xffffffffu << lo_w);
              if (absent >> 2 * w & 1u) sees &= 0xffff0000u;
              if (absent >> (2 * w + 1) & 1u) sees &= 0x0000ffffu;
              poisoned |= (bad_words[w] & sees) != 0;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(sees >> c & 1u)) s[32 * w + c] = 0xff800000u;
            }
          }
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < TILE; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) tops[k] = max3(tops[k], __uint_as_float(s[c + k]), __uint_as_float(s[c + k + 4]));
          const float top = max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]);
          // z = S sc (+ v_log: e4m3 weights carry what the tile's values were divided by).
          // m starts as the maximum itself: the weight of a row's only token is 1, exactly.
          const float unit = fmaxf(sc, 1e-37f);
          float v_log = E4M3 ? vinfo[vs].v_log : 0.f;
          if (E4M3 && (absent | wide) & kOwn) {
            // Tokens whose values were divided by 2^(v_log + own): the weights carry the largest of
            // those that this row sees.  (Tiles without such tokens come here once a row has seen
            // ones so large that what it keeps to, 2^-90 of them, may be above the tile's.)
            if (absent & kOwn) {
              int own = -1000;
#pragma unroll 1
              for (int c = max(lo, 0); c < min(hi, TILE); ++c) own = max(own, (int)v_own[vs][c]);
              v_log = fmaxf(v_log + (float)own, (float)kLeastLog);
              v_seen = fmaxf(v_seen, v_log);
              wide |= __any_sync(0xffffffffu, v_log > (float)(kLeastLog + 90)) ? kOwn : 0u;
            }
            v_log = fmaxf(v_log, fmaxf(v_seen, vinfo[vs].v_run) - 90.f);
          }
          const float top_z = top == -INFINITY ? top : fmaf(top, unit, v_log);
          const bool grew = m != -INFINITY && top_z > m + kLazy;
          if (m == -INFINITY) m = top_z;
          if (__any_sync(0xffffffffu, grew)) {
            // (e4m3: m may grow by the 200 orders between two tiles' v_log, of which l, which has none of
            // them, keeps its part: half of them at a time, none of which underflows)
            const float half = grew ? ex2(E4M3 ? 0.5f * (m - top_z) : m - top_z) : 1.f, f = E4M3 ? half * half : half;
            if (grew) m = top_z;
            l = E4M3 ? l * half * half : l * f;
            if (NQ == 1 && !(ok = g == 0 || values_done(g - 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld_x16(o_at + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st_x16(o_at + c, o);
            }
            tmem_st_wait();
          }
          const float ref = m == -INFINITY ? 0.f : (v_log - m) + (E4M3 ? kUpBits : 0.f);
          const float2 unit2 = make_float2(unit, unit), ref2 = make_float2(ref, ref);
          float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < TILE; c += 32) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float2 z0 = make_float2(__uint_as_float(s[c + i]), __uint_as_float(s[c + i + 1])), z1 = make_float2(__uint_as_float(s[c + i + 2]), __uint_as_float(s[c + i + 3]));
              const float2 y0 = __ffma2_rn(z0, unit2, ref2), y1 = __ffma2_rn(z1, unit2, ref2);
              const float2 e0 = make_float2(ex2(y0.x), ex2(y0.y)), e1 = make_float2(ex2(y1.x), ex2(y1.y));
              l2[0] = __fadd2_rn(l2[0], e0), l2[1] = __fadd2_rn(l2[1], e1);
              w[i / 2] = E4M3 ? pack_f16(e0.x, e0.y) : pack_bf16(e0.x, e0.y);
              w[i / 2 + 1] = E4M3 ? pack_f16(e1.x, e1.y) : pack_bf16(e1.x, e1.y);
            }
            tmem_st_x16(at + c / 2, w);
          }
          const float more = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
          l += E4M3 ? more * ex2(-v_log) : more;
          tmem_st_wait();
          if (E4M3 && (absent | wide) & kOwn) {  // weights times what their tokens' values were divided by, over what is in v_log
            const int rest = (int)vinfo[vs].v_log - (int)v_log;
#pragma unroll 1
            for (int c = 0; c < TILE / 2; c += 4) {
              uint32_t w[4];
              tmem_ld_x4(at + c, w);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const short2 own = absent & kOwn ? reinterpret_cast<const short2 *>(v_own[vs])[c + i] : make_short2(0, 0);
                const auto factor = [&](int o) { return __int_as_float((127 + min(max(rest + o, -126), 0)) << 23); };  // (of tokens that are not seen at most 1)
                const float2 e = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                w[i] = pack_f16(e.x * factor(own.x), e.y * factor(own.y));
              }
              tmem_st_x4(at + c, w);
            }
            tmem_st_wait();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[buf]);
      }
      // ---- the piece ends: O is complete once its last product is
      if (active && x.n > 0 && ok) {
        const int g = mine_t + x.n - 1;
        ok = values_done(g);
        tc_fence_after();
      }
      if (used && ok) {
        const int i = tok, head = x.head * p.group + (row - tok * p.group);
        const int64_t token = (int64_t)x.tok0 + i;
        float *slot = p.slots + (2 * (int64_t)blockIdx.x + (x.kind == 1)) * (int64_t)(D + 2) * p.slot_rows + row_t;
        const float f = poisoned ? __int_as_float(0x7fc00000) : x.kind ? 1.f : l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + token * a.ldo + (int64_t)head * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (x.n > 0) {
            tmem_ld_x32(o_at + c, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (live && x.kind) {
#pragma unroll
            for (int k = 0; k < 32; ++k) slot[(int64_t)(c + k) * p.slot_rows] = __uint_as_float(o[k]) * f;
          } else if (live) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[k + e]) * f;
              store8(out + c + k, v);
            }
          }
          __syncwarp();
        }
        if (live && x.kind) {
          slot[(int64_t)D * p.slot_rows] = m;
          slot[(int64_t)(D + 1) * p.slot_rows] = l;
        } else if (live && a.lse) {
          a.lse[token * a.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l) - (E4M3 ? kUpBits : 0.f)) * kLn2;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) free_item();
      tiles += x.n;
      if (active && x.n > 0) mine_t += x.n, ++taken;
      ++it;
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(256 - C::kMoreRegs));
    if (warp == 8 || warp == 10) {
      // ------------------------------------------------------------- products
      // A whole warp runs each half, so that descriptors are uniform values; one lane issues.
      const uint32_t leader = elect_one();
      const uint32_t base = smem_u32(smem);
      uint32_t count0 = 0, count1 = 0;  // key tiles of query tiles 0 and 1
      Item x;
      if (warp == 8) {
        constexpr uint32_t id_qk = idesc_of(!E4M3, false, TILE);
        const uint64_t q_desc = sdesc_sw128(base, 1024), k_desc = sdesc_sw128(base + C::kKAt, 1024);
        uint64_t *k_ready = E4M3 ? bars.k_ready : bars.k_full;
        int ks = 0;         // next stage of K
        uint32_t kph = 0, q_seen0 = 0, q_seen1 = 0;
        uint32_t used = 0;  // times that the one score buffer was used (dim 128)
        // Scores of query tile t with the key tile in stage ks, the g-th of this query tile
        const auto qk = [&](int t, uint32_t g, bool first_key, bool last_key, bool last_q) {
          const uint32_t buf = NQ == 1 ? g & 1u : t, sb = C::kSBufs == 1 ? 0u : buf;
          const uint32_t use = C::kSBufs == 1 ? used++ : NQ == 1 ? g >> 1 : g;
          // the key tile is there, and the scores that were in this buffer have been read
          const uint32_t sp = (use & 1u) ^ 1u;
          if (!(first_key ? warp_wait2(&k_ready[ks], kph, &bars.s_free[sb], sp, a.err) : warp_wait(&bars.s_free[sb], sp, a.err))) return false;
          tc_fence_after();
          const uint64_t qd = q_desc + (uint64_t)((uint32_t)t * (C::kQ >> 4)), kd = k_desc + (uint64_t)((uint32_t)ks * (C::kSide >> 4));
          const uint32_t d = tmem + C::kSCol + sb * TILE;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_ss(d, qd + (uint64_t)((k / 4) * (128 * 128 >> 4) + (k % 4) * 2), kd + (uint64_t)((k / 4) * (TILE * 128 >> 4) + (k % 4) * 2), id_qk, k != 0, leader);
          tc_commit_if(&bars.s_full[buf], leader);
          tc_commit_if(&bars.k_empty[ks], last_key ? leader : 0u);
          tc_commit_if(&bars.q_empty[t], last_q ? leader : 0u);
          if (last_key && ++ks == ST) ks = 0, kph ^= 1u;
          return true;
        };
        while (ok && next_item(x)) {
          const int n = __shfl_sync(0xffffffffu, x.n, 0), act = NQ == 1 || __shfl_sync(0xffffffffu, x.rows, 0) <= 128 ? 1 : 2;
          for (int j = 0; j < n; ++j) {
            if (j == 0 && !(ok = warp_wait(&bars.q_full[0], q_seen0++ & 1u, a.err))) break;
            if (!(ok = qk(0, count0 + j, true, act == 1, j + 1 == n))) break;
            if (act == 1) continue;
            if (j == 0 && !(ok = warp_wait(&bars.q_full[1], q_seen1++ & 1u, a.err))) break;
            if (!(ok = qk(1, count1 + j, false, true, j + 1 == n))) break;
          }
          if (!ok) break;
          count0 += n;
          if (act == 2) count1 += n;
          __syncwarp();
          if (leader) free_item();
          ++it;
        }
      } else {
        constexpr uint32_t id_pv = idesc_of(!E4M3, true, D);
        const uint64_t v_desc = sdesc_v(base + C::kVAt, TILE * 128);
        int vs = 0;  // next stage of V
        uint32_t vph = 0;
        // The weights of query tile t times the values in stage vs.
        const auto pv = [&](int t, uint32_t g, bool fresh, bool last_value) {
          const uint32_t buf = NQ == 1 ? g & 1u : t;
          const uint32_t pp = (NQ == 1 ? g >> 1 : g) & 1u;
          if (!(t == 0 ? warp_wait2(&bars.v_ready[vs], vph, &bars.p_full[buf], pp, a.err) : warp_wait(&bars.p_full[buf], pp, a.err))) return false;
          tc_fence_after();
          const uint64_t vd = v_desc + (uint64_t)((uint32_t)vs * (C::kSide >> 4));
          const uint32_t d = tmem + t * D, pa = tmem + C::kPCol + buf * (TILE / 2);
#pragma unroll
          for (int k = 0; k < TILE / 16; ++k) tc_mma_ts(d, pa + k * 8, vd + (uint64_t)(k * (16 * 128 >> 4)), id_pv, k != 0 || !fresh, leader);
          tc_commit_if(&bars.o_done[buf], leader);
          tc_commit_if(&bars.v_empty[vs], last_value ? leader : 0u);
          if (last_value && ++vs == ST) vs = 0, vph ^= 1u;
          return true;
        };
        while (ok && next_item(x)) {
          const int n = __shfl_sync(0xffffffffu, x.n, 0), act = NQ == 1 || __shfl_sync(0xffffffffu, x.rows, 0) <= 128 ? 1 : 2;
          for (int j = 0; j < n; ++j) {
            if (!(ok = pv(0, count0 + j, j == 0, act == 1))) break;
            if (act == 2 && !(ok = pv(1, count1 + j, j == 0, true))) break;
          }
          if (!ok) break;
          count0 += n;
          if (act == 2) count1 += n;
          __syncwarp();
          if (leader) free_item();
          ++it;
        }
      }
    } else {
      // --------------------------------- work list, copies of K (warp 9), copies of V (11)
      const bool values = warp == 11;
      int tiles = 0, made = 0;
      const auto put = [&](const Item &x) {
        if (!warp_wait(&bars.item_empty[made % kRing], ((uint32_t)(made / kRing) & 1u) ^ 1u, a.err)) return false;
        if (lane == 0) {
          items[made % kRing] = x;
          mbar_arrive(&bars.item_full[made % kRing]);
        }
        __syncwarp();
        ++made;
        return true;
      };
      int4 open = make_int4(-1, 0, 0, 0);  // the item that this CTA starts and does not end
      int open_rows = 0;
      // Where the search stands: request r (its key heads take `unit` units each),
      // key head, the first of 32 blocks, the units before each lane's block, and
      // which of these blocks are still to come.
      int r = 0, head = 0, b0 = 0, blocks = 0;
      int64_t at = 0, unit = 0, u = 0, before = 0, upto = 0;
      unsigned todo = 0;
      Req q = {};
      bool ignore = false, fresh = true;
      if (u0 < u1) {
        int lo = 0, hi = kThreads - 1;  // the first thread whose inclusive sum exceeds u0
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (sums[mid] > u0) hi = mid;
          else lo = mid + 1;
        }
        at = lo ? sums[lo - 1] : 0;  // units before the request
        r = lo * per;
      } else {
        r = a.n;
      }
      const auto blocks_at = [&]() {  // the costs of 32 blocks, and the units before each
        const int cost = b0 + lane < blocks ? block_cost<TILE, ROWS, C::kItemCost>(p, q, b0 + lane) : 0;
        upto = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        before = u + upto - cost;
        todo = __ballot_sync(0xffffffffu, cost && before + cost > u0 && before < u1);
      };
      const auto find = [&](Item &x) {  // this CTA's next piece; false: there is none
        for (;;) {
          while (todo) {
            const int src = __ffs(todo) - 1;
            todo &= todo - 1;
            const int64_t ub = __shfl_sync(0xffffffffu, before, src);
            x.r = r, x.head = head, x.row0 = (b0 + src) * ROWS, x.rows = min(ROWS, q.rows - x.row0);
            x.tok0 = q.tok0, x.pos0 = q.pos0;
            int t0, t1;
            tiles_of<TILE>(p, q, x.row0, x.rows, t0, t1);
            const int nt = t1 - t0;
            // tile k of the item is unit ub + item cost + k
            const int ta = (int)min(max(u0 - ub - C::kItemCost, (int64_t)0), (int64_t)nt), tb = (int)min(max(u1 - ub - C::kItemCost, (int64_t)0), (int64_t)nt);
            if (nt == 0 ? ub < u0 : ta == tb) continue;  // another CTA's
            const int first = q.pos0 + (int)p.by_group.div(x.row0), last = q.pos0 + (int)p.by_group.div(x.row0 + x.rows - 1);
            x.lo = first_seen(a, first), x.hi = end_seen(a, last);
            x.full_lo = first_seen(a, last), x.full_hi = end_seen(a, first);
            x.t0 = t0 + ta, x.n = tb - ta;
            x.kind = x.n == nt ? 0 : ta == 0 ? 1 : 2;
            if (x.kind == 1) {
              open = make_int4(r, head, x.row0, (int)((ub + C::kItemCost + nt - 1) / run));
              open_rows = x.rows;
            }
            return true;
          }
          if (fresh) {  // a request
            if (r >= a.n || at >= u1) return false;
            q = request(p, r, ignore);
            blocks = (q.rows + ROWS - 1) / ROWS;
            unit = 0;  // of a key head: lanes take blocks in turn
            for (int b = lane; b < blocks; b += 32) unit += block_cost<TILE, ROWS, C::kItemCost>(p, q, b);
#pragma unroll
            for (int o = 16; o; o >>= 1) unit += __shfl_xor_sync(0xffffffffu, unit, o);
            if (!blocks || at + unit * a.kv_heads <= u0) {
              at += unit * a.kv_heads;
              ++r;
              continue;
            }
            head = at < u0 ? (int)((u0 - at) / unit) : 0;
            u = at + head * unit;  // units before the key head, then before block b0
            b0 = 0, fresh = false;
            blocks_at();
            continue;
          }
          u += __shfl_sync(0xffffffffu, upto, 31);
          b0 += 32;
          if (b0 >= blocks) {
            b0 = 0;
            if (++head == a.kv_heads || u >= u1) {
              fresh = true;
              at += unit * a.kv_heads;
              ++r;
              continue;
            }
          }
          blocks_at();
        }
      };
      Item x = {}, y = {};  // (no tiles yet)
      for (bool more = true; more && ok; x = y) {
        if (values) {
          if (!next_item(x)) break;
        } else {
          // the others know of an item before the copies of the one before it
          more = find(y);
          if (more && !(ok = put(y))) break;
        }
        // ---- its tiles.  Lanes hold 32 table entries from page tb0 on, and the 32 after them.
        // Boxes of a tile: a lane copies a part of one of them.
        const int boxes = TILE >> p.box_shift, part = lane >> ((TILE == 64 ? 6 : 7) - p.box_shift);
        static_assert(TILE / 16 * C::kParts <= 32 && C::kRawParts <= C::kParts);
        int tb0 = (x.t0 * TILE) >> p.page_shift;
        const auto table_at = [&](int i) { return i < a.max_pages ? a.table[x.r * a.ldt + i] : -1; };
        int entry = 0, entry2 = 0;
        if (x.n > 0) entry = table_at(tb0 + lane), entry2 = table_at(tb0 + 32 + lane);
        for (int j = 0; j < x.n; ++j, ++tiles) {
          const int s = tiles % ST;
          const uint32_t ph = ((uint32_t)(tiles / ST) & 1u) ^ 1u;
          const int pos = (x.t0 + j) * TILE;
          while (((pos + TILE - 1) >> p.page_shift) - tb0 >= 64) {
            tb0 += 32;
            entry = entry2;
            entry2 = table_at(tb0 + 32 + lane);
          }
          // box `lane % boxes` of the tile, its page; the lanes after the first `boxes` take the other parts
          const int b = lane & (boxes - 1), box_pos = pos + (b << p.box_shift), i = (box_pos >> p.page_shift) - tb0;
          const int e1 = __shfl_sync(0xffffffffu, entry, i & 31), e2 = __shfl_sync(0xffffffffu, entry2, i & 31);
          const int page = i < 32 ? e1 : e2;
          const bool wanted = box_pos < x.hi && box_pos + p.box_rows > x.lo;
          const bool there = wanted && page >= 0 && page < a.n_pages;
          const unsigned need = __ballot_sync(0xffffffffu, wanted && lane < boxes), have = __ballot_sync(0xffffffffu, there && lane < boxes);
          if (need != have && !values && lane == 0) set_device_error(a.err, kDevErrBadPage);
          const uint32_t box_bytes = (uint32_t)p.box_rows * D * C::kEs, loaded = __popc(have) * box_bytes;
          const int in_page = box_pos & (a.page - 1);
          uint64_t *full = values ? &bars.v_full[s] : &bars.k_full[s];
          if (!(ok = warp_wait(values ? &bars.v_empty[s] : &bars.k_empty[s], ph, a.err))) break;
          if (lane == 0) {
            uint32_t pieces = 0;  // 16-token pieces that are absent
            for (unsigned w = need & ~have; w; w &= w - 1) {
              const int at16 = (__ffs(w) - 1) << (p.box_shift - 4);
              pieces |= ((1u << (p.box_rows >> 4)) - 1u) << at16;  // (a box has at most 128 rows)
            }
            if (values) v_absent[s] = pieces;
            else gone[tiles & 7] = pieces;
            mbar_arrive_expect_tx(full, loaded + (E4M3 && values ? __popc(have) * p.box_rows * 8 : 0));
          }
          __syncwarp();
          uint8_t *dst = smem + (values ? C::kVAt : C::kKAt) + s * C::kSide + (E4M3 ? C::kSide - C::kRaw : 0);
          if (there && part < (E4M3 ? C::kRawParts : C::kParts))
            tma_load_5d(dst + part * TILE * 128 + (b << p.box_shift) * (E4M3 ? D / C::kRawParts : 128), values ? &vmap : &kmap, full, 0, in_page, part, x.head, page);
          if (E4M3 && values && there && lane < boxes) {
            float *ks = reinterpret_cast<float *>(smem + C::kScaleAt) + s * 2 * TILE + (b << p.box_shift);
            const int64_t from = ((int64_t)page * a.kv_heads + x.head) * a.page + in_page;
            bulk_load(ks, a.scale[0] + from, p.box_rows * 4, full);
            bulk_load(ks + TILE, a.scale[1] + from, p.box_rows * 4, full);
          }
          __syncwarp();
        }
        if (values) {
          if (!ok) break;
          if (lane == 0) free_item();
          ++it, y = x;
        }
      }
      if (!values && lane == 0) {
        p.desc[2 * blockIdx.x] = open;
        p.desc[2 * blockIdx.x + 1] = make_int4(open_rows, 0, 0, 0);
      }
      if (!values && ok) {
        Item end;
        end.rows = -1;
        ok = put(end);
      }
      // copies in flight land before the CTA may end
      const int left = min(tiles, ST);
      for (int j = tiles - left; !ok && j < tiles; ++j) {
        warp_wait(values ? &bars.v_full[j % ST] : &bars.k_full[j % ST], (uint32_t)(j / ST) & 1u, a.err);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(256 - C::kMoreRegs));
    // ---------------------------------------------------------------- prepare
    const int th = tid - 384;  // 0..127
    int tiles = 0, count[2] = {0, 0};
    Item x;
    for (;;) {
      const bool more = next_item(x);
      if (!group_and(1, ok) || !more) break;
      // ---- Q: a warp takes 32 rows of a query tile, a lane knows where one lies (-1: not of this item, zeros)
      for (int t = 0; t < NQ && x.n > 0 && x.rows > 128 * t; ++t) {
        const int c = count[t]++, first = 32 * (warp - 12), rr = 128 * t + first + lane, rw = x.row0 + rr, tok = (int)p.by_group.div(rw);
        const int64_t where = rr < x.rows ? ((int64_t)x.tok0 + tok) * a.ldq + (int64_t)(x.head * p.group + (rw - tok * p.group)) * a.ldq_head : -1;
        uint8_t *dst = smem + t * C::kQ;
        constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces of a row, rows of an iteration
        if (!(ok = warp_wait(&bars.q_empty[t], ((uint32_t)c & 1u) ^ 1u, a.err))) break;
#pragma unroll C::kQRows
        for (int i = 0; i < 32 / RPI; ++i) {
          const int r = i * RPI + lane / CH, row = first + r, ch = lane % CH;
          const int64_t from = __shfl_sync(0xffffffffu, where, r);
          cp_async16(dst + (ch / 8) * 128 * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), static_cast<const __nv_bfloat16 *>(a.q) + max(from, (int64_t)0) + ch * 8, from >= 0 ? 16 : 0);
        }
        cp_async_commit();
        cp_async_wait<0>();
        if (E4M3) {
          // rows to fp16, times a power of two that brings their largest value to 2^14..2^15
          __syncwarp();
          const int row = first + lane;
          uint8_t *r0 = dst + row * 128;
          uint32_t top = 0;
#pragma unroll C::kQPieces
          for (int ch = 0; ch < CH; ++ch) {
            const uint4 v = *reinterpret_cast<const uint4 *>(r0 + (ch / 8) * 128 * 128 + (((ch & 7) ^ (row & 7)) << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(w[e] >> 16 & 0x7fffu, w[e] & 0x7fffu));
          }
          const int ex = (int)(top >> 7) - 127;         // of the largest value
          const int up = min(max(14 - ex, -113), 126);  // factor 2^up
          const float f = __int_as_float((up + 127) << 23) * (a.softmax_scale > 0.f ? 1.f : a.softmax_scale < 0.f ? -1.f : 0.f);
#pragma unroll C::kQPieces
          for (int ch = 0; ch < CH; ++ch) {
            uint4 *at = reinterpret_cast<uint4 *>(r0 + (ch / 8) * 128 * 128 + (((ch & 7) ^ (row & 7)) << 4));
            const uint4 v = *at;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
            *at = make_uint4(w[0], w[1], w[2], w[3]);
          }
          q_scale[c % kRing][128 * t + row] = __int_as_float((127 - up) << 23);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.q_full[t]);
      }
      if (!group_and(1, ok)) break;
      int v_run = -1000;  // largest v_log so far, of tokens that all rows see
      for (int j = 0; j < x.n; ++j, ++tiles) {
        const int s = tiles % ST;
        const uint32_t ph = (uint32_t)(tiles / ST) & 1u;
        constexpr int RC = D / 16, PER = C::kRaw / 16 / 128;  // e4m3: 16-byte pieces of a row, and of a thread
        // This thread's 16-byte pieces (16 e4m3 values) of a tile lie in rows row0 + i
        // (128 / RC), a multiple of 8 apart, at place ch of the row; they become two pieces
        // of fp16 at their swizzled places.  Pieces 0..3 of a row and 4..7 lie in the same
        // banks: the latter write their second half first.
        const int row0 = th / RC, ch = th % RC, sw = (ch >> 2) & 1, c0 = 2 * (ch & 3);
        const uint32_t at0 = (uint32_t)((ch / 4) * TILE * 128 + row0 * 128);
        const uint32_t first = at0 + (uint32_t)(((c0 + sw) ^ (row0 & 7)) << 4), second = at0 + (uint32_t)(((c0 + 1 - sw) ^ (row0 & 7)) << 4);
        const auto place = [&](uint8_t *side, int i, const uint4 &v, bool scaled, __half2 f) {
          uint2 h[4] = {e4m3x4_f16(v.x), e4m3x4_f16(v.y), e4m3x4_f16(v.z), e4m3x4_f16(v.w)};
          if (scaled) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 lo = __hmul2(*reinterpret_cast<const __half2 *>(&h[e].x), f), hi = __hmul2(*reinterpret_cast<const __half2 *>(&h[e].y), f);
              h[e] = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            }
          }
          const uint4 w0 = make_uint4(h[0].x, h[0].y, h[1].x, h[1].y), w1 = make_uint4(h[2].x, h[2].y, h[3].x, h[3].y);
          *reinterpret_cast<uint4 *>(side + first + i * (128 / RC) * 128) = sw ? w1 : w0;
          *reinterpret_cast<uint4 *>(side + second + i * (128 / RC) * 128) = sw ? w0 : w1;
        };
        // What a token's values are divided by besides 2^v_log, where that does not fit its scale.
        const auto own_of = [](float scale, int v_log) {
          const int e = (int)(__float_as_uint(scale) >> 23), off = e - 127 - v_log;
          return e > 20 && e < 255 && (off < -14 || off > 6) ? min(max(off, kLeastLog - v_log), kMostLog - v_log) : 0;  // (e above 255: negative)
        };
        // Rows are converted one after the other by a short loop.  (Unrolled, these warps
        // wait for their instructions, which the others' push out: 60 requests, three of
        // them chunks, head size 128, 1183 us, unrolled by 4 1072, by 2 945, not 927.)
        // Head sizes 128 and 256: 128 values of a row lie where their later half goes, and a
        // row belongs to one warp.  Size 64: row r goes where rows 2 r - 128 and 2 r - 127 lay,
        // so that all warps have read up to r before one of them writes.
        const uint32_t raw_at = (uint32_t)(C::kSide - C::kRaw + (D == 256 ? (ch / 8) * TILE * 128 + row0 * 128 + (ch & 7) * 16 : th * 16));
        const auto convert = [&](uint8_t *side, const auto &put) {
#pragma unroll 1
          for (int i = 0; i < PER; ++i) {
            const uint4 raw = *reinterpret_cast<const uint4 *>(side + raw_at + i * (128 / RC) * (D == 64 ? 64 : 128));
            if (D == 64) ok = group_and(1, ok);
            else __syncwarp();
            put(i, raw);
          }
        };
        const int pos = (x.t0 + j) * TILE;
        if (E4M3) {
          ok = warp_wait(&bars.k_full[s], ph, a.err);
          uint8_t *k = smem + C::kKAt + s * C::kSide;
          convert(k, [&](int i, const uint4 &w) { place(k, i, w, false, __half2()); });
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.k_ready[s]);
        }
        ok = warp_wait(&bars.v_full[s], ph, a.err) && ok;  // (the group leaves as one, below)
        uint8_t *v = smem + C::kVAt + s * C::kSide;
        const uint32_t absent = v_absent[s];
        const auto dead = [&](int row) { return pos + row < x.lo || pos + row >= x.hi || (absent >> (row / 16) & 1u); };
        // tokens that some row does not see, beside those that all rows see
        const bool partial = pos < x.full_lo || pos + TILE > x.full_hi || absent;
        const float *v_scales = reinterpret_cast<const float *>(smem + C::kScaleAt) + (2 * s + 1) * TILE;
        float mine = 1.f;
        if (E4M3) {
          mine = th < TILE ? v_scales[th] : 0.f;
          // the largest exponent of this warp's scales, of tokens that all rows see; after the barrier that of all is known
          const uint32_t e = th < TILE && !dead(th) && pos + th >= x.full_lo && pos + th < x.full_hi && mine - mine == 0.f && mine > 0.f ? __float_as_uint(mine) >> 23 : 0u, top = __reduce_max_sync(0xffffffffu, e);
          if (lane == 0) e_max[tiles & 1][warp - 12] = top;
          if (th == 0) vinfo[s].absent = absent;
        }
        if (th < 4) vinfo[s].bad[th] = 0;
        if (!(ok = group_and(1, ok))) break;
        if (E4M3) {
          // Values enter as fp16 times their scale over 2^v_log, by which the largest scale
          // becomes 2^6 .. 2^7 (times 448 still fp16); below 2^(kLeastLog + 6) they are less.  A
          // tile whose scales are all far below an earlier one's keeps to 2^-90 of it: a weight
          // that underflows with its scale would be missing in the sum of weights.
          const uint32_t *tops = e_max[tiles & 1], e = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
          int v_log = max((int)e - 133, kLeastLog);
          if (!partial) {
            v_run = max(v_run, v_log);
            v_log = max(v_log, v_run - 90);
          } else {
            // A token that a row does not see must not decide how its own are rounded.  So where
            // some rows see tokens that others do not, v_log goes by those that all see (here,
            // or else before), whose largest scale becomes 1 .. 2.  A token whose scale does not
            // fit beside that (2^-14 .. 2^7; below 2^-106 it counts as 0) is divided by a power of
            // its own, which the rows that see it put into their weights.
            if (e) v_run = max(v_run, v_log);
            v_log = min(max(max(e ? (int)e - 127 : v_run + 6, kLeastLog), v_run - 90), kMostLog);
            const int own = own_of(mine, v_log);
            v_own[s][th] = (int16_t)(dead(th) ? -1000 : own);
            if (!dead(th) && own) atomicOr(&vinfo[s].absent, kOwn);
          }
          const float down = __int_as_float((127 - v_log) << 23);
          if (th == 0) vinfo[s].v_log = (float)v_log, vinfo[s].v_run = (float)v_run;
          // tokens whose scale is not finite
          if (th < TILE) {
            const uint32_t odd = __ballot_sync(0xffffffffu, !dead(th) && !(mine - mine == 0.f));
            if (odd && lane == 0) atomicOr(&vinfo[s].bad[th >> 5], odd);
          }
          if (!partial) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.v_known[s]);
          }
          if (!partial) {
            convert(v, [&](int i, const uint4 &w) {
              const float f = v_scales[row0 + i * (128 / RC)] * down;
              place(v, i, w, true, __float2half2_rn(fabsf(f) <= 128.f ? f : 0.f));
            });
          } else {
            convert(v, [&](int i, uint4 w) {
              const int row = row0 + i * (128 / RC);
              const auto nan4 = [](uint32_t y) { return __vcmpeq4(y & 0x7f7f7f7fu, 0x7f7f7f7fu); };
              const bool gone = dead(row), nan = (nan4(w.x) | nan4(w.y) | nan4(w.z) | nan4(w.w)) != 0;
              if (!gone && nan) atomicOr(&vinfo[s].bad[row >> 5], 1u << (row & 31));
              if (gone || nan) w = make_uint4(0, 0, 0, 0);
              const float scale = v_scales[row], f = scale * 0.5f * __int_as_float((128 - v_log - own_of(scale, v_log)) << 23);  // (the power itself may be too small)
              place(v, i, w, true, __float2half2_rn(fabsf(f) <= 128.f ? f : 0.f));
            });
          }
          fence_proxy_async_smem();
        } else {
          if (th == 0) vinfo[s].absent = absent;
          if (partial) {
            constexpr int CH = D / 8;
            for (int i = th; i < TILE * CH; i += 128) {
              const int row = i / CH, ch = i % CH;
              uint4 *at = reinterpret_cast<uint4 *>(v + (ch / 8) * TILE * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
              const uint4 w = *at;
              const auto odd2 = [](uint32_t y) { return (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u; };
              const bool gone = dead(row), odd = odd2(w.x) || odd2(w.y) || odd2(w.z) || odd2(w.w);
              if (!gone && odd) atomicOr(&vinfo[s].bad[row >> 5], 1u << (row & 31));
              if (gone || odd) *at = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) {
          if (E4M3 && partial) mbar_arrive(&bars.v_known[s]);
          mbar_arrive(&bars.v_ready[s]);
        }
      }
      if (!ok) break;
      if (lane == 0) free_item();
      ++it;
    }
  }

  // Every warp comes here, whatever happened to it.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// Joins the pieces of the items that several CTAs share: that of the CTA that
// starts the item (slot 1) and of all after it up to the last (slot 0).  A lane
// owns a row, a warp 8 of its values, so all loads are of 128 contiguous bytes.
// Blocks are small, because most of them find that their CTA starts no such item:
// with all of a row's values in one block, 745 tokens x 16 heads x 256 took 28.7 us in
// all and not 22.6, 100000 tokens x 32 heads x 128 93.5 and not 89.2.
template <int D, bool E4M3>
__global__ void __launch_bounds__(128) chunk_join_kernel(const __grid_constant__ Params p) {
  const AttnArgs &a = p.a;
  const int lane = threadIdx.x & 31, c0 = blockIdx.z * 32 + threadIdx.x / 32 * 8, cta = blockIdx.x;
  grid_dependency_wait();
  const int4 d = p.desc[2 * cta];
  const int rows = p.desc[2 * cta + 1].x;
  const int row_t = blockIdx.y * 32 + lane;
  if (d.x < 0 || (int)blockIdx.y * 32 >= rows) return;
  float m = -INFINITY, l = 0.f, o[8] = {};
  const int64_t size = (int64_t)(D + 2) * p.slot_rows;
  bool ignore = false;
  const Req q = request(p, d.x, ignore);
  constexpr int kAtOnce = 4;  // pieces whose loads are on their way together (100000 tokens: with 1 103.9 us, with 4 93.5, with 8 94.5)
  for (int c = cta; c <= d.w; c += kAtOnce) {
    float pm[kAtOnce], pl[kAtOnce], v[kAtOnce][8];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const float *slot = p.slots + (2 * (int64_t)(c + u) + (c + u == cta)) * size + row_t;
      const bool there = c + u <= d.w;
      pm[u] = there ? slot[(int64_t)D * p.slot_rows] : -INFINITY, pl[u] = there ? slot[(int64_t)(D + 1) * p.slot_rows] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = there ? slot[(int64_t)(c0 + i) * p.slot_rows] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      // (e4m3: the sums' factors half at a time, as where a tile's reference grows)
      constexpr float kPart = E4M3 ? 0.5f : 1.f;
      const float mn = fmaxf(m, pm[u]), hf = m == mn ? 1.f : ex2(kPart * (m - mn)), hg = pm[u] == mn ? 1.f : ex2(kPart * (pm[u] - mn));
      const float f = E4M3 ? hf * hf : hf, g = E4M3 ? hg * hg : hg;
      m = mn;
      l = E4M3 ? l * hf * hf + pl[u] * hg * hg : l * f + pl[u] * g;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = o[i] * f + v[u][i] * g;
    }
  }
  if (row_t >= rows) return;
  const int row = d.z + row_t, tok = (int)p.by_group.div(row), head = d.y * p.group + (row - tok * p.group);
  const int64_t token = (int64_t)q.tok0 + tok;
  const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = l == 0.f && o[i] == o[i] ? 0.f : o[i] * f;
  store8(static_cast<__nv_bfloat16 *>(a.out) + token * a.ldo + (int64_t)head * D + c0, o);
  if (c0 == 0 && a.lse)
    a.lse[token * a.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l) - (E4M3 ? kUpBits : 0.f)) * kLn2;
}

int slot_rows(int64_t tokens, int group, int dim) {
  const int64_t rows = (tokens * group + 31) / 32 * 32, most = dim == 256 ? 128 : 256;
  return (int)(rows < most ? rows : most);
}
size_t desc_bytes() { return (size_t)kMaxSms * 2 * sizeof(int4); }

template <int D, bool E4M3>
cudaError_t launch_cfg(Params &p, cudaStream_t stream) {
  using C = Cfg<D, E4M3>;
  const AttnArgs &a = p.a;
  static SmemLimit limit;
  cudaError_t e = raise_smem_limit(limit, chunk_kernel<D, E4M3>, C::kSmem);
  if (e != cudaSuccess) return e;
  p.box_rows = a.page < C::kTile ? a.page : C::kTile;
  p.box_shift = 31 - __builtin_clz((unsigned)p.box_rows);
  p.page_shift = 31 - __builtin_clz((unsigned)a.page);
  // (values of a part of a row, token, part, head, page): a bf16 row in 128-byte
  // parts, swizzled; an e4m3 row in parts of 64 or 128 bytes
  const int parts = E4M3 ? C::kRawParts : C::kParts, inner = D / parts;
  const uint64_t dims[5] = {(uint64_t)inner, (uint64_t)a.page, (uint64_t)parts, (uint64_t)a.kv_heads, (uint64_t)a.n_pages};
  const uint64_t strides[4] = {(uint64_t)a.token_stride * C::kEs, (uint64_t)inner * C::kEs, (uint64_t)a.head_stride * C::kEs,
                               (uint64_t)a.page_stride * C::kEs};
  const uint32_t box[5] = {(uint32_t)inner, (uint32_t)p.box_rows, 1, 1, 1};
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i)
    if (encode_tiled(&maps[i], E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                     const_cast<void *>(a.cache[i]), dims, strides, box,
                     E4M3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  const int sms = device_facts()->sm_count, grid = sms < kMaxSms ? sms : kMaxSms;
  chunk_kernel<D, E4M3><<<grid, kThreads, C::kSmem, stream>>>(p, maps[0], maps[1]);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)(p.slot_rows / 32), D / 32);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, chunk_join_kernel<D, E4M3>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t paged_attn_chunk_workspace_size(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  const int group = q_heads / (kv_heads < q_heads ? kv_heads : q_heads);
  return desc_bytes() + (size_t)kMaxSms * 2 * (dim + 2) * slot_rows(tokens, group, dim) * 4;
}

cudaError_t launch_paged_attn_chunk(const AttnArgs &a, int64_t tokens, const int64_t *cu, cudaStream_t s) {
  const int group = a.q_heads / a.kv_heads;
  Params p = {a, tokens, cu, group, FastDiv(group), 0, 0, 0, slot_rows(tokens, group, a.dim), static_cast<int4 *>(a.workspace),
              reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + desc_bytes())};
  const bool e = a.cache_dtype == Q4K_DTYPE_E4M3;
  if (a.dim == 64) return e ? launch_cfg<64, true>(p, s) : launch_cfg<64, false>(p, s);
  if (a.dim == 128) return e ? launch_cfg<128, true>(p, s) : launch_cfg<128, false>(p, s);
  return e ? launch_cfg<256, true>(p, s) : launch_cfg<256, false>(p, s);
}

}  // namespace q4k
