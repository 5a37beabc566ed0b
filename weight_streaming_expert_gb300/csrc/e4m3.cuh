// e4m3.cuh -- rows of the quantised cache (include/attention.h): E4M3 codes
// with one power of two for each row of a key/value head.
//
// e is the least integer with max |y| <= 448 * 2^e, so the largest value takes
// one of the two highest binades of the format and no bit of a code's precision
// is lost to the scale; code * 2^e is exact in bf16 and fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"

namespace wse {

constexpr int kScaleBias = 127, kLowestScale = -40, kHighestScale = 40;

// The exponent for a row whose largest finite |value| is `largest`: 448 = 1.75 *
// 2^8, and adding what is left of the mantissa above .75 carries where it is
// larger.
__device__ __forceinline__ int scale_for(float largest) {
  const int e = (int)((__float_as_uint(largest) + 0x1fffffu) >> 23) - 127 - 8;
  return min(max(e, kLowestScale), kHighestScale);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A scale byte as its exponent.  Bytes that no write leaves count as the
// nearest ones that it does (what lies in unused rows may be anything).
__device__ __forceinline__ int exponent_of(uint32_t byte) {
  return min(max((int)byte - kScaleBias, kLowestScale), kHighestScale);
}

// |y| where y is finite, else 0: what counts for the largest value.
__device__ __forceinline__ float finite_size(float y) {
  const float a = fabsf(y);
  return a < INFINITY ? a : 0.f;
}

// Four values to codes (the first in the lowest byte): rounded to the nearest,
// ties to even, finite ones saturated at 448; infinities become NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d, float inv) {
  auto scaled = [&](float y) { return fabsf(y) < INFINITY ? y * inv : __uint_as_float(0x7fffffffu); };
  uint32_t codes;
  asm("{ .reg .b16 p, q; cvt.rn.satfinite.e4m3x2.f32 p, %2, %1; cvt.rn.satfinite.e4m3x2.f32 q, %4, %3; "
      "mov.b32 %0, {p, q}; }"
      : "=r"(codes)
      : "f"(scaled(a)), "f"(scaled(b)), "f"(scaled(c)), "f"(scaled(d)));
  return codes;
}

// Sixteen codes times a power of two as 16-bit elements: exact in bf16; in fp16
// rounded below 2^-14 and cut to its largest number.
__device__ __forceinline__ void expand_e4m3(uint4 codes, float scale, bool bf16, uint32_t (&o)[8]) {
  const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t half[2];
    e4m3x4_to_f16x2(c[i], half[0], half[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float2 v = __half22float2(*reinterpret_cast<const __half2*>(&half[k]));
      v.x *= scale;
      v.y *= scale;
      if (bf16) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
        o[2 * i + k] = *reinterpret_cast<const uint32_t*>(&r);
      } else {
        auto cut = [](float x) { return fabsf(x) > 65504.f ? copysignf(65504.f, x) : x; };  // a NaN stays
        const __half2 r = __floats2half2_rn(cut(v.x), cut(v.y));
        o[2 * i + k] = *reinterpret_cast<const uint32_t*>(&r);
      }
    }
  }
}

}  // namespace wse
