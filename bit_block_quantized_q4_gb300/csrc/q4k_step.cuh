// q4k_step.cuh -- device helpers of the kernels around the projections (norm,
// cache writes, attention): 8-value vectors of fp32 or bf16, and the e4m3
// rounding with a scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "q4k_device.cuh"

namespace q4k {

// Device error word: a page, slot or length outside the cache or the table.
constexpr unsigned kDevErrBadPage = 4u;

// Tiled tensor copy global -> shared, completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(c4)
      : "memory");
}

// Division of 0 <= x < 2^31 by a fixed 1 <= d < 2^31 with one multiplication:
// with s = ceil(log2 d) and m = floor(2^(31+s) / d) + 1 (< 2^32 + 1; d = 1 and
// other powers of two are shifts), x m / 2^(31+s) exceeds x / d by less than
// 1 / d for x < 2^31, so its floor is the quotient.
struct FastDiv {
  uint32_t d, m, s;  // m = 0: shift by s
  explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
    while (s < 31 && (1u << s) < d) ++s;
    if ((1u << s) != d) {
      m = (uint32_t)(((uint64_t)1 << (31 + s)) / d + 1);
      --s;
    }
  }
  __host__ __device__ uint32_t div(uint32_t x) const {
    if (!m) return x >> s;
    return (uint32_t)(((uint64_t)x * m) >> 32) >> s;
  }
};

// The smallest block maximum a scale is derived from: keeps 448 / max finite
// and the scale a normal number, so a block of zeros has a scale of its own.
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100

// 8 values as they lie in memory (bf16: 4 registers until they are used).
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void to(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void to(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
};
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
  Raw8<T> r;
  r.load(p);
  r.to(v);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                             pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
// The scale of a block, max / 448, in the block's first lane and the factor of
// its values, 448 / max, in all others and returned to all: one division.  Lanes
// of a block are consecutive, `place` is the lane's in it; `mask` are the lanes
// that take part.
__device__ __forceinline__ float block_factor(float amax, int place, unsigned mask, float &scale) {
  const bool first = place == 0;
  const float q = (first ? amax : 448.f) / (first ? 448.f : amax);
  scale = q;
  return __shfl_sync(mask, q, (int)(threadIdx.x & 31) - place + 1);
}
// e4m3(v * inv), nearest even, finite overflow saturating to 448, NaN kept.
__device__ __forceinline__ uint2 to_e4m3x8(const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j] * inv, v[4 * j + 1] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * j + 2] * inv, v[4 * j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[j] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace q4k
