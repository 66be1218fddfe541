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
// CTAs: every CTA scans all requests, 1024 at a time (cheaper than passing
// sums between CTAs), and the requests' writes are divided among them.  A
// cluster barrier between the reads and the writes of a chunk is what allows
// lens_out == lens and state_out == state.

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
  int n, width, page, pool_size;
  unsigned *err;
};

struct Sums {
  int64_t tokens, need, back;
};
__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) {
  return {a.tokens + b.tokens, a.need + b.need, a.back + b.back};
}
__device__ __forceinline__ Sums shfl_up(const Sums &s, int o) {
  return {__shfl_up_sync(0xffffffffu, s.tokens, o), __shfl_up_sync(0xffffffffu, s.need, o),
          __shfl_up_sync(0xffffffffu, s.back, o)};
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanArgs a) {
  __shared__ Sums warp_sums[32];
  __shared__ unsigned long long taken_max;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_ctarank(), ranks = (int)gridDim.x;
  const int64_t size = a.pool_size;
  const int64_t head = ((a.state[0] % size) + size) % size;
  const int64_t count = min(max((int64_t)a.state[1], (int64_t)0), size);
  const int ps = a.page;
  if (tid == 0) taken_max = 0;
  Sums carry = {0, 0, 0};
  bool bad_page = false;

  for (int r0 = 0; r0 < a.n; r0 += kPlanThreads) {
    const int r = r0 + tid;
    const bool in = r < a.n;
    const int64_t len = in ? a.lens[r] : 0, add = in ? a.add[r] : 0;
    const int64_t more = max(add, (int64_t)0);
    const bool bad = len < 0 || add < -1 || len + more > (int64_t)a.width * ps;
    const bool done = add == -1;
    const int64_t have = bad ? 0 : (len + ps - 1) / ps;
    // prefix of the tokens first: a request whose tokens do not fit the slot
    // map asks for no pages
    int64_t t = more;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    if (lane == 31) warp_sums[warp].tokens = t;
    __syncthreads();
    int64_t chunk_tokens = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) t += warp_sums[w].tokens;
      chunk_tokens += warp_sums[w].tokens;
    }
    const int64_t cu1 = carry.tokens + t, cu0 = cu1 - more;
    const bool lng = !bad && more > 0 && cu1 > a.n_slots;
    const int64_t need = bad || done || lng ? 0 : (len + more + ps - 1) / ps - have;
    const int64_t back = done && !bad ? have : 0;
    int64_t p = need, q = back;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, p, o), v = __shfl_up_sync(0xffffffffu, q, o);
      if (lane >= o) p += u, q += v;
    }
    if (lane == 31) warp_sums[warp].need = p, warp_sums[warp].back = q;
    // every lens, add and state value of this chunk has been read by every CTA
    // before any CTA writes outputs that may be the same buffers
    cluster_sync();
    Sums chunk = {chunk_tokens, 0, 0};
    for (int w = 0; w < 32; ++w) {
      if (w < warp) p += warp_sums[w].need, q += warp_sums[w].back;
      chunk.need += warp_sums[w].need, chunk.back += warp_sums[w].back;
    }
    const int64_t upto = carry.need + p, first = upto - need, back0 = carry.back + q - back;
    const bool granted = !bad && !lng && !done && (need == 0 || upto <= count);
    if (granted && need > 0) atomicMax(&taken_max, (unsigned long long)upto);

    // Small outputs of the warp's 32 requests: one CTA of the cluster.
    if (in && warp % ranks == rank) {
      a.status[r] = bad ? Q4K_KV_BAD_LENGTH : lng ? Q4K_KV_NO_SLOTS : granted || done ? Q4K_KV_OK : Q4K_KV_NO_PAGES;
      a.lens_out[r] = (int32_t)(granted ? len + more : done && !bad ? 0 : len);
      a.cu[r] = cu0;
      if (r == a.n - 1) a.cu[a.n] = cu1;
    }
    // Tokens and pages.  Requests with at most 4 tokens or pages to move are
    // written by their own lane; the others by the warp together, their
    // elements divided among the CTAs of the cluster.
    const int64_t work = max(max(more, granted ? need : (int64_t)0), back);
    const bool small = in && work <= 4;
    auto token = [&](int64_t i, int64_t at, int64_t ln, int64_t hv, int64_t fst, int64_t row, bool ok) {
      if (at >= a.n_slots) return;
      int32_t slot = -1, where = -1;
      if (ok) {
        const int64_t pp = ln + i, pg = pp / ps;
        const int32_t id = pg < hv ? a.table[row * a.ldt + pg] : a.pool[(head + fst + pg - hv) % size];
        where = (int32_t)pp;
        if (id >= 0 && id < a.pool_size) slot = id * ps + (int32_t)(pp - pg * ps);
        else bad_page = true;
      }
      a.slots[at] = slot;
      a.pos[at] = where;
    };
    auto fresh = [&](int64_t j, int64_t hv, int64_t fst, int64_t row) {
      a.table[row * a.ldt + hv + j] = a.pool[(head + fst + j) % size];
    };
    auto give = [&](int64_t j, int64_t b0, int64_t row) {
      if (b0 + j < size - count) a.pool[(head + count + b0 + j) % size] = a.table[row * a.ldt + j];
      else bad_page = true;
    };
    if (small && warp % ranks == rank) {
      for (int64_t i = 0; i < more; ++i) token(i, cu0 + i, len, have, first, r, granted);
      if (granted)
        for (int64_t j = 0; j < need; ++j) fresh(j, have, first, r);
      for (int64_t j = 0; j < back; ++j) give(j, back0, r);
    }
    unsigned big = __ballot_sync(0xffffffffu, in && !small);
    while (big) {
      const int src = __ffs(big) - 1;
      big &= big - 1;
      const int64_t rr = r0 + warp * 32 + src;
      const int64_t m = __shfl_sync(0xffffffffu, more, src), nd = __shfl_sync(0xffffffffu, granted ? need : 0, src);
      const int64_t bk = __shfl_sync(0xffffffffu, back, src), c0 = __shfl_sync(0xffffffffu, cu0, src);
      const int64_t ln = __shfl_sync(0xffffffffu, len, src), hv = __shfl_sync(0xffffffffu, have, src);
      const int64_t fs = __shfl_sync(0xffffffffu, first, src), b0 = __shfl_sync(0xffffffffu, back0, src);
      const bool ok = __shfl_sync(0xffffffffu, (int)granted, src);
      const int64_t m_in = min(m, max(a.n_slots - c0, (int64_t)0));
      for (int64_t i = rank * 32 + lane; i < m_in; i += 32 * ranks) token(i, c0 + i, ln, hv, fs, rr, ok);
      for (int64_t j = rank * 32 + lane; j < nd; j += 32 * ranks) fresh(j, hv, fs, rr);
      for (int64_t j = rank * 32 + lane; j < bk; j += 32 * ranks) give(j, b0, rr);
    }
    carry = carry + chunk;
    __syncthreads();  // warp_sums are rewritten in the next chunk
  }
  for (int64_t t = carry.tokens + rank * kPlanThreads + tid; t < a.n_slots; t += (int64_t)ranks * kPlanThreads)
    a.slots[t] = -1, a.pos[t] = -1;
  if (rank == 0 && tid == 0) {
    const int64_t taken = (int64_t)taken_max;
    a.state_out[0] = (int32_t)((head + taken) % size);
    a.state_out[1] = (int32_t)(count - taken + min(carry.back, size - count));
  }
  if (bad_page) set_device_error(a.err, kDevErrBadPage);
}

// --------------------------------------------------------------------- write
//
// One row (token, head) of K or V: D/8 lanes of 8 values each.  Bound by
// bytes: inputs read once, cache rows written once.

struct WriteArgs {
  const void *in[2];
  void *cache[2];
  float *scale[2];
  const int32_t *slots;
  int64_t tokens, ld_token, ld_head, page_stride, head_stride, token_stride, n_slots;
  int heads, page;
  unsigned *err;
};

template <int D, typename TI, bool E4M3>
__global__ void __launch_bounds__(256) kv_write_kernel(const WriteArgs a) {
  constexpr int LPR = D / 8;  // lanes per row
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int c = threadIdx.x % LPR;
  const int64_t t = row / a.heads;
  const int h = (int)(row - t * a.heads), kv = blockIdx.y;
  if (t >= a.tokens) return;  // whole warps or whole rows: the shuffles below stay within a row
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.n_slots) {
    if (slot != -1 && c == 0) set_device_error(a.err, kDevErrBadPage);
    return;
  }
  const int64_t page = slot / a.page, off = slot - page * a.page;
  float v[8];
  load8(static_cast<const TI *>(a.in[kv]) + t * a.ld_token + h * a.ld_head + c * 8, v);
  const int64_t to = page * a.page_stride + h * a.head_stride + off * a.token_stride + c * 8;
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
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.cache[kv]) + to) = to_e4m3x8(v, 448.f / amax);
    if (c == 0) a.scale[kv][(page * a.heads + h) * a.page + off] = amax / 448.f;
  }
}

template <int D>
void launch_write_d(const WriteArgs &a, bool bf16_in, bool e4m3, cudaStream_t s) {
  const int64_t rows = a.tokens * a.heads;
  constexpr int kRows = 256 / (D / 8);
  const dim3 grid((unsigned)((rows + kRows - 1) / kRows), 2);
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
                      n_slots, n, width, page, pool_size, device_error_word()};
  // One CTA writes about 4096 tokens in the time that a wider cluster's
  // barriers take.
  const int ranks = n_slots <= 4096 ? 1 : n_slots <= 16384 ? 4 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kPlanThreads);
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
  const WriteArgs a = {{k, v}, {k_cache, v_cache}, {k_scale, v_scale}, slots, tokens, ld_token,
                       ld_head, page_stride, head_stride, token_stride, n_pages * page, heads, page,
                       device_error_word()};
  const bool b = in_dtype == Q4K_DTYPE_BF16, e = cache_dtype == Q4K_DTYPE_E4M3;
  if (dim == 64) launch_write_d<64>(a, b, e, stream);
  else if (dim == 128) launch_write_d<128>(a, b, e, stream);
  else launch_write_d<256>(a, b, e, stream);
  return cudaGetLastError();
}

}  // namespace q4k
