// q4k_kv.cu -- the paged key-value cache: block tables and slot maps from
// request lengths (q4k_kv_plan), and the write of new rows (q4k_kv_write).
//
// "PRD: Performant Concurrent Distributed GGUF Runtime": hot KV state per
// session, and batching of decode steps (DGR-012): several requests' tokens
// share one step, each with its own cached context.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/q4k.h"
#include "q4k_device.cuh"
#include "q4k_internal.h"
#include "q4k_step.cuh"
#include "q4k_step.h"

namespace q4k {
namespace {

// ---------------------------------------------------------------------- plan
//
// Per request r with len tokens cached and add to come (add -1: finished),
// page size ps:
//   have = ceil(len / ps), need = ceil((len + add) / ps) - have,
//   cu   = exclusive prefix of max(add, 0): the step's token offsets,
//   P    = inclusive prefix of need; granted if need == 0 or P <= count,
//   new pages pool[(head + P - need + j) mod size], j < need.
// Pages of finished requests go to the ring's tail, in request order, and are
// handed out by later calls only.  So the call reads and writes disjoint parts
// of the ring and of the table, and repeating it on the same lens, add and
// state gives the same result.
//
// What bounds it: latency (a few hundred KB at most).  One cluster of 1..8
// CTAs: every CTA scans all requests, a block's width at a time (cheaper than
// passing sums between CTAs), and the requests' writes are divided among them.
// A cluster barrier between the reads and the writes of a chunk is what allows
// lens_out == lens and state_out == state; without requests there is no chunk,
// and one barrier of its own before the outputs that are defined all the same.

constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int32_t *lens, *add;
  int32_t *table;
  int64_t ldt;
  int32_t *pool;
  const int32_t *state;
  int32_t *lens_out;
  int64_t *cu;
  int32_t *slots, *pos, *status, *state_out;
  int64_t n_slots;
  int n, capacity;  // capacity: tokens of a table row, < 2^31
  uint32_t pool_size;
  FastDiv page;
  unsigned *err;
};

// Inclusive sum over the block, and the block's total.  `part` holds one value
// per warp; the caller's barriers separate its uses.
__device__ __forceinline__ int64_t warp_scan(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ int64_t before_warp(const int64_t *part, int warps, int warp, int64_t &total) {
  const int lane = threadIdx.x & 31;
  const int64_t incl = warp_scan(lane < warps ? part[lane] : 0);
  total = __shfl_sync(0xffffffffu, incl, 31);
  const int64_t prev = __shfl_sync(0xffffffffu, incl, warp ? warp - 1 : 0);
  return warp ? prev : 0;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanArgs a) {
  __shared__ int64_t part[3][32];
  __shared__ unsigned taken_max;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int rank = (int)cluster_ctarank(), ranks = (int)gridDim.x;
  const uint32_t size = a.pool_size, ps = a.page.d;
  const int64_t head_in = a.state[0] % (int64_t)size;
  const uint32_t head = (uint32_t)(head_in < 0 ? head_in + size : head_in);
  const uint32_t count = (uint32_t)min(max((int64_t)a.state[1], (int64_t)0), (int64_t)size);
  const auto ring = [&](uint32_t i) {  // i < 2 size: head + an offset into the ring
    return i >= size ? i - size : i;
  };
  if (tid == 0) taken_max = 0;
  int64_t tokens0 = 0, need0 = 0, back0 = 0;  // of the chunks before
  bool bad_page = false;

  for (int r0 = 0; r0 < a.n; r0 += blockDim.x) {
    const int r = r0 + tid;
    const bool in = r < a.n;
    const int len = in ? a.lens[r] : 0, add = in ? a.add[r] : 0, more = max(add, 0);
    const bool bad = len < 0 || add < -1 || (int64_t)len + more > a.capacity;
    const bool done = add == -1;
    const int have = bad ? 0 : (int)a.page.div(len + ps - 1);
    // tokens first: a request whose tokens do not fit the slot map asks for no pages
    int64_t t = warp_scan(more);
    if (lane == 31) part[0][warp] = t;
    __syncthreads();
    int64_t chunk_tokens, chunk_need, chunk_back;
    t += before_warp(part[0], warps, warp, chunk_tokens);
    const int64_t cu1 = tokens0 + t, cu0 = cu1 - more;
    const bool lng = !bad && more > 0 && cu1 > a.n_slots;
    const int need = bad || done || lng ? 0 : (int)a.page.div(len + more + ps - 1) - have;
    const int back = done && !bad ? have : 0;
    int64_t p = warp_scan(need), q = warp_scan(back);
    if (lane == 31) part[1][warp] = p, part[2][warp] = q;
    // every lens, add and state value of this chunk has been read by every CTA
    // before any CTA writes outputs that may be the same buffers
    cluster_sync();
    p += before_warp(part[1], warps, warp, chunk_need);
    q += before_warp(part[2], warps, warp, chunk_back);
    const int64_t upto = need0 + p, given = back0 + q - back;
    const bool granted = !bad && !lng && !done && (need == 0 || upto <= count);
    if (granted && need > 0) atomicMax(&taken_max, (unsigned)upto);
    // ring index of its first new page; only used where upto <= count <= size
    const uint32_t first = granted && need ? ring(head + (uint32_t)(upto - need)) : 0u;
    // tokens that the slot map has room for
    const int room = (int)max(min((int64_t)more, a.n_slots - cu0), (int64_t)0);

    // Small outputs of the warp's 32 requests: one CTA of the cluster.
    if (in && warp % ranks == rank) {
      a.status[r] = bad ? Q4K_KV_BAD_LENGTH : lng ? Q4K_KV_NO_SLOTS : granted || done ? Q4K_KV_OK : Q4K_KV_NO_PAGES;
      a.lens_out[r] = granted ? len + more : done && !bad ? 0 : len;
      a.cu[r] = cu0;
      if (r == a.n - 1) a.cu[a.n] = cu1;
    }
    // Tokens and pages.  Requests with at most 4 tokens or pages to move are
    // written by their own lane; the others by the warp together, their
    // elements divided among the CTAs of the cluster.
    const auto token = [&](int i, int64_t at, int ln, int hv, uint32_t fst, int64_t row, bool ok) {
      int32_t slot = -1, where = -1;
      if (ok) {
        const uint32_t pp = ln + i, pg = a.page.div(pp);
        const int32_t id = (int)pg < hv ? a.table[row * a.ldt + pg] : a.pool[ring(fst + (pg - hv))];
        where = (int32_t)pp;
        if ((uint32_t)id < size) slot = id * ps + (pp - pg * ps);
        else bad_page = true;
      }
      a.slots[at] = slot;
      a.pos[at] = where;
    };
    const auto fresh = [&](int j, int hv, uint32_t fst, int64_t row) {
      a.table[row * a.ldt + hv + j] = a.pool[ring(fst + j)];
    };
    const auto give = [&](int j, int64_t b0, int64_t row) {
      // the ring has size - count entries left; the rest is dropped
      if (b0 + j < size - count) a.pool[ring(ring(head + count) + (uint32_t)(b0 + j))] = a.table[row * a.ldt + j];
      else bad_page = true;
    };
    const int pages = granted ? need : 0;
    const bool small = in && max(max(room, pages), back) <= 4;
    if (small && warp % ranks == rank) {
      for (int i = 0; i < room; ++i) token(i, cu0 + i, len, have, first, r, granted);
      for (int j = 0; j < pages; ++j) fresh(j, have, first, r);
      for (int j = 0; j < back; ++j) give(j, given, r);
    }
    unsigned big = __ballot_sync(0xffffffffu, in && !small);
    while (big) {
      const int src = __ffs(big) - 1;
      big &= big - 1;
      const int64_t rr = r0 + warp * 32 + src;
      const int m = __shfl_sync(0xffffffffu, room, src), nd = __shfl_sync(0xffffffffu, pages, src);
      const int bk = __shfl_sync(0xffffffffu, back, src), ln = __shfl_sync(0xffffffffu, len, src);
      const int hv = __shfl_sync(0xffffffffu, have, src), ok = __shfl_sync(0xffffffffu, (int)granted, src);
      const int64_t c0 = __shfl_sync(0xffffffffu, cu0, src), b0 = __shfl_sync(0xffffffffu, given, src);
      const uint32_t fs = __shfl_sync(0xffffffffu, first, src);
      const int step = 32 * ranks, i0 = rank * 32 + lane;
      for (int i = i0; i < m; i += step) token(i, c0 + i, ln, hv, fs, rr, ok);
      for (int j = i0; j < nd; j += step) fresh(j, hv, fs, rr);
      for (int j = i0; j < bk; j += step) give(j, b0, rr);
    }
    tokens0 += chunk_tokens, need0 += chunk_need, back0 += chunk_back;
    __syncthreads();  // part[] is rewritten in the next chunk
  }
  if (a.n == 0) {
    cluster_sync();  // every CTA has read the state
    if (rank == 0 && tid == 0) a.cu[0] = 0;
  }
  for (int64_t t = tokens0 + rank * blockDim.x + tid; t < a.n_slots; t += (int64_t)ranks * blockDim.x)
    a.slots[t] = -1, a.pos[t] = -1;
  if (rank == 0 && tid == 0) {
    a.state_out[0] = (int32_t)ring(head + taken_max);
    a.state_out[1] = (int32_t)(count - taken_max + min(back0, (int64_t)(size - count)));
  }
  if (bad_page) set_device_error(a.err, kDevErrBadPage);
}

// --------------------------------------------------------------------- write
//
// A token's rows of K and V of one head: D/8 lanes of 8 values each; a block
// takes tokens of one head.  Bound by bytes (inputs read once, cache rows written
// once), with the instructions of a row close behind: the 16001 x 8 x 128 bf16 ->
// e4m3 write took 71 us with the token and the page from 64-bit divisions, 42
// with 32-bit ones, 21.3 without and with two rows of K or of V per lane, and
// 18.1 us (5.5 TB/s) now that K and V share the slot and the place.  6 blocks
// per SM: 19.9 us.  Two tokens per lane: 18.3, and 64-wide fp32 rows 8.9 -> 12.6.

struct WriteArgs {
  const void *in[2];
  void *cache[2];
  float *scale[2];
  const int32_t *slots;
  int64_t ld_token, ld_head, page_stride, head_stride, token_stride;
  uint32_t tokens, heads, n_slots;
  FastDiv page;
  unsigned *err;
};

template <int D, typename TI, bool E4M3>
__global__ void __launch_bounds__(256, 8) kv_write_kernel(const WriteArgs a) {
  constexpr int LPR = D / 8, TPB = 256 / LPR;  // lanes per row, tokens per block
  const int c = threadIdx.x % LPR;
  const uint32_t h = blockIdx.y, t = blockIdx.x * TPB + threadIdx.x / LPR;
  // all lanes of a row leave together, so the shuffles below are complete
  if (t >= a.tokens) return;
  const int32_t slot = a.slots[t];
  const int64_t from = t * a.ld_token + h * a.ld_head + c * 8;
  Raw8<TI> raw[2];  // K and V
  raw[0].load(static_cast<const TI *>(a.in[0]) + from);
  raw[1].load(static_cast<const TI *>(a.in[1]) + from);
  if ((uint32_t)slot >= a.n_slots) {
    if (slot != -1 && c == 0) set_device_error(a.err, kDevErrBadPage);
    return;
  }
  const uint32_t page = a.page.div(slot), off = slot - page * a.page.d;
  const int64_t to = page * a.page_stride + h * a.head_stride + off * a.token_stride + c * 8;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float v[8];
    raw[kv].to(v);
    if (!E4M3) {
      store8(static_cast<__nv_bfloat16 *>(a.cache[kv]) + to, v);
    } else {
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
      const unsigned mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << ((threadIdx.x & 31) / LPR * LPR);
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o));
      amax = fmaxf(amax, kAmaxFloor);
      float factor;
      const float inv = block_factor(amax, c, mask, factor);
      *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.cache[kv]) + to) = to_e4m3x8(v, inv);
      if (c == 0) a.scale[kv][((int64_t)page * a.heads + h) * a.page.d + off] = factor;
    }
  }
}

template <int D>
void launch_write_d(const WriteArgs &a, bool bf16_in, bool e4m3, cudaStream_t s) {
  constexpr uint32_t kTokens = 256 / (D / 8);
  const dim3 grid((a.tokens + kTokens - 1) / kTokens, a.heads);
  if (bf16_in && e4m3) kv_write_kernel<D, __nv_bfloat16, true><<<grid, 256, 0, s>>>(a);
  else if (bf16_in) kv_write_kernel<D, __nv_bfloat16, false><<<grid, 256, 0, s>>>(a);
  else if (e4m3) kv_write_kernel<D, float, true><<<grid, 256, 0, s>>>(a);
  else kv_write_kernel<D, float, false><<<grid, 256, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_kv_plan(const int32_t *lens, const int32_t *add, int32_t n, int32_t *table,
                           int64_t ldt, int32_t width, int32_t page, int32_t *pool,
                           int32_t pool_size, const int32_t *state, int32_t *lens_out, int64_t *cu,
                           int32_t *slots, int32_t *pos, int64_t n_slots, int32_t *status,
                           int32_t *state_out, cudaStream_t stream) {
  const PlanArgs a = {lens, add, table, ldt, pool, state, lens_out, cu, slots, pos, status, state_out,
                      n_slots, n, width * page, (uint32_t)pool_size, FastDiv(page), device_error_word()};
  const int ranks = n_slots <= 4096 ? 1 : n_slots <= 16384 ? 4 : 8;
  // a block as wide as the requests, and wide enough for the slots; a warp at least
  const int64_t most = n > n_slots / 8 ? n : n_slots / 8, wide = most > 0 ? most : 1;
  const int threads = wide >= kPlanThreads ? kPlanThreads : ((int)wide + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_plan_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_write(const void *k, const void *v, int in_dtype, int64_t ld_token,
                            int64_t ld_head, const int32_t *slots, int64_t tokens, int32_t heads,
                            int32_t dim, void *k_cache, void *v_cache, int cache_dtype,
                            int64_t n_pages, int32_t page, int64_t page_stride, int64_t head_stride,
                            int64_t token_stride, float *k_scale, float *v_scale,
                            cudaStream_t stream) {
  const WriteArgs a = {{k, v}, {k_cache, v_cache}, {k_scale, v_scale}, slots, ld_token, ld_head,
                       page_stride, head_stride, token_stride, (uint32_t)tokens, (uint32_t)heads,
                       (uint32_t)(n_pages * page), FastDiv(page), device_error_word()};
  const bool b = in_dtype == Q4K_DTYPE_BF16, e = cache_dtype == Q4K_DTYPE_E4M3;
  if (dim == 64) launch_write_d<64>(a, b, e, stream);
  else if (dim == 128) launch_write_d<128>(a, b, e, stream);
  else launch_write_d<256>(a, b, e, stream);
  return cudaGetLastError();
}

}  // namespace q4k
