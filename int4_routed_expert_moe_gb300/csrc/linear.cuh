// What the kernels of moe_linear share.
#pragma once

#include <cuda_fp16.h>

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
  int act;
  const void* residual;  // of y's type
  long long ldr;
  void* y;
  bool y32;
  long long ldy;
  int32_t* flags;
};

// The activations in FP32. NaN gives NaN (relu: v > 0 ? v : 0 v).
__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {
    case MOE_ACT_RELU: return v > 0.0f ? v : 0.0f * v;
    case MOE_ACT_SILU: return v / (1.0f + expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678f));
    case MOE_ACT_GELU_TANH: return 0.5f * v * (1.0f + tanhf(0.79788456f * (v + 0.044715f * v * v * v)));
    case MOE_ACT_SIGMOID: return 1.0f / (1.0f + expf(-v));
    default: return v;
  }
}

}  // namespace moe
