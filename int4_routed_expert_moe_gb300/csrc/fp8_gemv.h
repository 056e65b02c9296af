// The FP8 weight stream for a few tokens (see fp8_gemv.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace moe {

constexpr int kGemvMaxTokens = 16;

// y [T][N] = x W^T from codes and scales, T <= kGemvMaxTokens.
int fp8_gemv(const uint8_t* xq, const float* xs, int T, const uint8_t* wq, const float* ws, int N, int K, __half* y,
             cudaStream_t st);
// The shared FFN, T <= kGemvMaxTokens; xq, xs, hq, hs: scratch for x and h as
// codes and scales; h: FP32 scratch [T][Is].
int fp8_gemv_ffn(const __half* x, int T, int H, int Is, const uint8_t* wg, const float* sg, const uint8_t* wu,
                 const float* su, const uint8_t* wd, const float* sd, uint8_t* xq, float* xs, uint8_t* hq, float* hs,
                 float* h, __half* y, cudaStream_t st);

}  // namespace moe
