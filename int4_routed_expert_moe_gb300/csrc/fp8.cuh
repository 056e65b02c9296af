// E4M3 block scaling shared by the FP8 kernels.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "device.cuh"

namespace moe {
namespace fp8 {

constexpr int kBlock = 128;       // elements of K per scale
constexpr float kMax = 448.0f;    // largest E4M3 value
constexpr float kMinAmax = 0x1p-126f * kMax;  // below, the scale is no normal number

// Running maximum of |x| over eight FP16 values, as two 16-bit patterns: the
// patterns of non-negative values order as the values do, infinities and NaN
// above every finite one.
__device__ __forceinline__ uint32_t amax_bits(const uint4& v, uint32_t m) {
  m = __vmaxu2(m, v.x & 0x7fff7fffu);
  m = __vmaxu2(m, v.y & 0x7fff7fffu);
  m = __vmaxu2(m, v.z & 0x7fff7fffu);
  return __vmaxu2(m, v.w & 0x7fff7fffu);
}

struct BlockScale {
  float scale;  // amax / 448: what a code is multiplied by
  float inv;    // 448 * (1 / amax): what a value is multiplied by
};
// A block of zeros has scale 0 and codes 0, and so has one whose scale would be
// below FP32's normal numbers (an intermediate h may come to that, FP16 values
// cannot): 448 / amax would overflow, and its zeros times infinity be NaN. A
// block that holds an infinity or NaN has scale and codes NaN, so that what is
// computed from it says so.
// inv is the reciprocal, rounded, times 448, rounded: what PyTorch computes for
// 448.0 / amax, so that the codes are those of x * (448.0 / amax) there, bit for
// bit. One rounded division gives other codes only where x * 448 / amax is at or
// within 2^-22 of a tie (7e-5 of FP16 normal values), and both codes are as near
// to x: distance 0.025715586 of |x| either way. In a product of one token such
// a code is 1 % of the result, so the two choices are not left to chance.
__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale b;
  if (!(amax < INFINITY)) {
    b.scale = b.inv = __int_as_float(0x7fffffff);
  } else {
    const bool some = amax >= kMinAmax;
    b.scale = some ? amax / kMax : 0.0f;
    b.inv = some ? __frcp_rn(amax) * kMax : 0.0f;
  }
  return b;
}
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_half_bits) {
  return block_scale(__half2float(__ushort_as_half((unsigned short)amax_half_bits)));
}

// silu(v) = v / (1 + 2^(-v log2 e)) of the FFN's kernels, with the
// special-function unit's own 2^x and 1/x (relative errors about 2^-22, and the
// exponent's rounding, 2^-24 |v|). Below v = -87.3 the reciprocal is 0, and so
// is the result; NaN and -infinity give NaN.
__device__ __forceinline__ float silu(float v) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return v * r;
}

// Two values to two E4M3 codes (a in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  return encode2(a, b) | (encode2(c, d) << 16);
}
// Sixteen FP16 values times inv to sixteen codes.
__device__ __forceinline__ uint4 encode16(const uint4 (&in)[2], float inv) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 a = __half22float2(u32_as_h2(w[2 * j])), b = __half22float2(u32_as_h2(w[2 * j + 1]));
      o[2 * i + j] = encode4(a.x * inv, a.y * inv, b.x * inv, b.y * inv);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace fp8
}  // namespace moe
