// What the kernels of moe_linear share.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device.cuh"
#include "moe.h"

namespace moe {

struct LinearArgs {
  int T, N, K;
  const __half* x;
  long long ldx;
  const __half* w;
  const float* bias;
  bool bias_vec;  // on 16 bytes
  int act;
  const void* residual;  // of y's type
  long long ldr;
  void* y;
  bool y32;
  long long ldy;
  bool vec;  // rows of y and of the residual start on 16 bytes
  int32_t* flags;
};

constexpr int kLinearStreamTokens = 16;  // up to here the weight stream, above the tensor-memory kernels
int linear_stream(const LinearArgs& a, cudaStream_t st);
int linear_gemm(const LinearArgs& a, cudaStream_t st);

// 1 / (1 + e^-v). FAST, for results that FP16 rounds: the special-function
// unit's 2^x and 1/x (relative errors about 2^-22, and the exponent's rounding,
// 2^-24 |v|); else expf and a division to 2 units in the last place. 0 where
// 1 + e^-v is beyond 2^126, v < -87.
template <bool FAST>
__device__ __forceinline__ float sigmoid_times(float v, float m) {
  if (!FAST) return __fdividef(m, 1.0f + expf(-v));
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return m * r;
}
// v Phi(v) = max(v, 0) - |v| e^(-v^2/2) t q(t), t = 1 / (1 + 0.34 |v|), where
// t q(t) stands for e^(v^2/2) erfc(|v| / sqrt 2) / 2: no difference of numbers
// near 1 (v / 2 (1 + erf) is 2^-24 |v| / 2 off however small the result: FP16
// results from v = -3.7 down were 4 half steps off). q was fitted for the smallest
// relative error (least squares, the points weighted by their errors: Lawson's
// method), 2.5e-8 up to |v| = 13.3, where e^(-v^2/2) ends; all in all within
// (12 + 1.5 v^2) 2^-24 of the result. -infinity gives NaN, as the product of its
// factors does. 8192 x 8192 FP32 results of K = 1024, us: 157, with erff 181, with
// erfcf 370.
__device__ __forceinline__ float gelu(float v) {
  float a, z, t;
  asm("min.NaN.f32 %0, %1, 0f41800000;" : "=f"(a) : "f"(v));  // 16: infinity times 0 is NaN
  a = fabsf(a);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(v * v * -0.72134752f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(a, 0.34f, 1.0f)));
  float q = -0.026471842f;
  q = fmaf(q, t, 0.14114988f);
  q = fmaf(q, t, -0.2764137f);
  q = fmaf(q, t, 0.20577717f);
  q = fmaf(q, t, -0.047084384f);
  q = fmaf(q, t, 0.11631409f);
  q = fmaf(q, t, 0.11496757f);
  q = fmaf(q, t, 0.13614237f);
  q = fmaf(q, t, 0.13561885f);
  return fmaf(-z, a * t * q, fmaxf(v, 0.0f));
}
// The activations in FP32, of N values at a time. NaN gives NaN.
template <bool FAST, int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(v[i]));
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = sigmoid_times<FAST>(v[i], v[i]);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = gelu(v[i]);
      break;
    case MOE_ACT_GELU_TANH:  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = 0.79788456f * (v[i] + 0.044715f * v[i] * v[i] * v[i]);
        v[i] = sigmoid_times<FAST>(2.0f * u, v[i]);
      }
      break;
    case MOE_ACT_SIGMOID:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = sigmoid_times<FAST>(v[i], 1.0f);
      break;
    default: break;
  }
}

// The bias of columns n .. n + N - 1; every lane of a warp reads the same ones,
// 16 bytes at a time: a load or a shuffle per column takes shared-memory
// bandwidth from the MMAs' operands.
template <int N>
__device__ __forceinline__ void add_bias(const LinearArgs& a, int n, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    if (a.bias_vec && n + i + 4 <= a.N) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(a.bias + n + i));
      v[i] += q.x; v[i + 1] += q.y; v[i + 2] += q.z; v[i + 3] += q.w;
    } else {
#pragma unroll
      for (int e = i; e < i + 4; ++e)
        if (n + e < a.N) v[e] += __ldg(a.bias + n + e);
    }
  }
}

// N values of row t from column n: bias, activation, residual, one rounding,
// stored. N a multiple of 8 (of 4 for FP32) starting at such a column.
template <int N>
__device__ __forceinline__ void finish(const LinearArgs& a, int t, int n, float (&v)[N]) {
  const int left = a.N - n;
  if (left <= 0) return;
  if (a.bias) add_bias(a, n, v);
  const size_t at = (size_t)t * (size_t)a.ldy + n, ra = (size_t)t * (size_t)a.ldr + n;
  if (a.y32) {
    const float* r = static_cast<const float*>(a.residual) + ra;
    float* y = static_cast<float*>(a.y) + at;
    activate<false>(a.act, v);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      if (a.vec && i + 4 <= left) {
        if (a.residual) {
          const float4 q = *reinterpret_cast<const float4*>(r + i);
          v[i] += q.x; v[i + 1] += q.y; v[i + 2] += q.z; v[i + 3] += q.w;
        }
        *reinterpret_cast<float4*>(y + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      } else {
#pragma unroll
        for (int e = i; e < i + 4; ++e)
          if (e < left) y[e] = a.residual ? v[e] + r[e] : v[e];
      }
    }
  } else {
    const __half* r = static_cast<const __half*>(a.residual) + ra;
    __half* y = static_cast<__half*>(a.y) + at;
    activate<true>(a.act, v);
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 8) {
        if (a.vec && i + 8 <= left) {
          if (a.residual) {
            const uint4 q = *reinterpret_cast<const uint4*>(r + i);
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 p = __half22float2(u32_as_h2(u[e]));
              v[i + 2 * e] += p.x;
              v[i + 2 * e + 1] += p.y;
            }
          }
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const half2 p = __floats2half2_rn(v[i + 2 * e], v[i + 2 * e + 1]);
            h[e] = *reinterpret_cast<const uint32_t*>(&p);
          }
          *reinterpret_cast<uint4*>(y + i) = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
#pragma unroll
          for (int e = i; e < i + 8; ++e)
            if (e < left) y[e] = __float2half_rn(a.residual ? v[e] + __half2float(r[e]) : v[e]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < left) y[e] = __float2half_rn(a.residual ? v[e] + __half2float(r[e]) : v[e]);
    }
  }
}

}  // namespace moe
