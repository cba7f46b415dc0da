// Device helpers of the 8-bit block-scaled cache: e4m3 conversions, the
// power-of-two scale rule, dense element types, and finding a row's sequence.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace mtkv {
namespace f8 {

// Two codes (the low 16 bits of w) as two f16, exactly: every e4m3 value is
// an f16 value. Lower byte to the lower half.
__device__ __forceinline__ uint32_t codes_to_h2(uint16_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
  return h;
}

// Four codes as two f16 pairs: bytes (0, 1) and bytes (2, 3).
__device__ __forceinline__ void code4_to_h2(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; "
      "cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Four floats to four codes (x0 in the lowest byte), round to nearest even;
// beyond +-448 saturates, NaN becomes 0x7f.
__device__ __forceinline__ uint32_t to_code4(float x0, float x1, float x2, float x3) {
  uint32_t w;
  asm("{ .reg .b16 a, b; cvt.rn.satfinite.e4m3x2.f32 a, %2, %1; "
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3; mov.b32 %0, {a, b}; }"
      : "=r"(w)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return w;
}

// The least 2^e, e >= -126, with amax <= 448 * 2^e; 0 for amax == 0. From the
// bits of amax = 1.m * 2^x: 448 = 1.75 * 2^8, so e = x - 8, one more when
// 1.m > 1.75. (amax finite and not negative.)
__device__ __forceinline__ float pow2_scale(float amax) {
  if (amax == 0.f) return 0.f;
  const uint32_t b = __float_as_uint(amax);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -126);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// 1 / s for a power of two 2^-126 <= s <= 2^120 (as pow2_scale gives): exact.
__device__ __forceinline__ float pow2_inv(float s) {
  return __uint_as_float(0x7f000000u - __float_as_uint(s));
}

// ---------------------------------------------------- dense element types

// 8 consecutive elements (16 or 32 bytes) as raw words, and as floats.
template <int DT>
struct Raw8 {
  uint4 w[DT == MT_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *p) {
    w[0] = __ldg(reinterpret_cast<const uint4 *>(p));
    if constexpr (DT == MT_F32) w[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
  }
  __device__ __forceinline__ void zero() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (DT == MT_F32) w[1] = w[0];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
    if constexpr (DT == MT_F32) {
      const uint32_t v[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = __uint_as_float(u[i]);
        x[4 + i] = __uint_as_float(v[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MT_F16) {
          const float2 f = h2_to_f2(u[i]);
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        } else {
          x[2 * i] = __uint_as_float(u[i] << 16);
          x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
      }
    }
  }
};

// Two floats rounded to a pair of 16-bit elements.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == MT_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

// Store 4 floats as elements [i, i + 4) of p (i a multiple of 4).
template <int DT>
__device__ __forceinline__ void store4(void *p, size_t i, float a, float b, float c, float d) {
  if constexpr (DT == MT_F32)
    reinterpret_cast<float4 *>(p)[i / 4] = make_float4(a, b, c, d);
  else
    reinterpret_cast<uint2 *>(p)[i / 4] = make_uint2(pack2<DT>(a, b), pack2<DT>(c, d));
}

// --------------------------------------------------------- sequence search

// The largest s in [0, n) with f(s) <= u, for a non-decreasing f with f(0) <=
// u: 32 probes a round, so one round trip to memory up to 32 sequences and
// two up to 1024. The whole warp takes part; every lane gets the answer.
template <typename F>
__device__ __forceinline__ int warp_search(int n, int u, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {  // the answer lies in [lo, lo + n)
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const bool le = at < n && f(lo + at) <= u;
    const uint32_t b = __ballot_sync(0xffffffffu, le) | 1u;
    const int k = 31 - __clz(b);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

}  // namespace f8
}  // namespace mtkv
