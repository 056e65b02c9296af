// y = act(x W^T + bias) + residual, FP16 operands, FP32 sums.
//
// Plain form: a block of 16 x 16 threads per 16 tokens and 16 rows of W, both
// operands through shared memory, one sum per thread.
#include <algorithm>

#include "common.h"
#include "device.cuh"
#include "kernels.h"
#include "linear.cuh"

namespace moe {
namespace {

__global__ void __launch_bounds__(256) linear_plain_kernel(const LinearArgs a) {
  griddep_wait();
  __shared__ float xs[16][17], ws[16][17];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int n0 = blockIdx.x * 16;
  for (int m0 = blockIdx.y * 16; m0 < a.T; m0 += gridDim.y * 16) {
    float s = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += 16) {
      const bool in = k0 + tx < a.K;
      xs[ty][tx] = in && m0 + ty < a.T ? __half2float(a.x[(size_t)(m0 + ty) * a.ldx + k0 + tx]) : 0.0f;
      ws[ty][tx] = in && n0 + ty < a.N ? __half2float(a.w[(size_t)(n0 + ty) * a.K + k0 + tx]) : 0.0f;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 16; ++i) s = fmaf(xs[ty][i], ws[tx][i], s);
      __syncthreads();
    }
    const int t = m0 + ty, n = n0 + tx;
    if (t < a.T && n < a.N) {
      if (a.bias) s += a.bias[n];
      s = activate(a.act, s);
      if (a.residual) s += a.y32 ? static_cast<const float*>(a.residual)[(size_t)t * a.ldr + n]
                                 : __half2float(static_cast<const __half*>(a.residual)[(size_t)t * a.ldr + n]);
      if (a.y32) static_cast<float*>(a.y)[(size_t)t * a.ldy + n] = s;
      else static_cast<__half*>(a.y)[(size_t)t * a.ldy + n] = __float2half_rn(s);
    }
  }
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_linear_workspace_bytes(int T, int N, int K) {
  if (T < 0 || T > (1 << 20) || N < 1 || N > 65536 || K < 8 || K % 8 || K > 65536) return 0;
  return moe::kWorkspaceHeader;
}

int moe_linear(const void* x, long long ldx, int T, int K, const void* w, int N, const float* bias, int act,
               const void* residual, long long ldr, void* y, int y_type, long long ldy, void* workspace,
               size_t workspace_bytes, void* stream) {
  moe::NvtxRange nvtx_range("moe_linear");
  moe::clear_error();
  if (T < 0 || T > (1 << 20) || N < 1 || N > 65536 || K < 8 || K % 8 || K > 65536)
    return moe::fail(MOE_ERR_ARG, "moe_linear: need 0 <= T <= 2^20, 1 <= N <= 65536, K a multiple of 8 up to 65536 "
                     "(T=%d N=%d K=%d)", T, N, K);
  if (act < MOE_ACT_NONE || act > MOE_ACT_SIGMOID) return moe::fail(MOE_ERR_ARG, "moe_linear: unknown act %d", act);
  if (y_type != MOE_F32 && y_type != MOE_F16) return moe::fail(MOE_ERR_ARG, "moe_linear: unknown type %d", y_type);
  const long long most = 0x7fffffffLL;
  if (ldx < K || ldx % 8 || ldx > most || ldy < N || ldy > most || (residual && (ldr < N || ldr > most)))
    return moe::fail(MOE_ERR_ARG, "moe_linear: need ldx >= K, a multiple of 8, ldy and ldr >= N, all below 2^31 "
                     "(%lld, %lld, %lld)", ldx, ldy, ldr);
  if (T == 0) return MOE_OK;
  if (!x || !w || !y || !workspace) return moe::fail(MOE_ERR_ARG, "moe_linear: NULL pointer");
  const uintptr_t al = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(y) |
                       reinterpret_cast<uintptr_t>(residual);
  if (al % 16 || reinterpret_cast<uintptr_t>(bias) % 4 || reinterpret_cast<uintptr_t>(workspace) % 256)
    return moe::fail(MOE_ERR_ARG, "moe_linear: x, w, y and residual 16-byte, bias 4-byte, workspace 256-byte aligned");
  const size_t need = moe_linear_workspace_bytes(T, N, K);
  if (workspace_bytes < need)
    return moe::fail(MOE_ERR_CAPACITY, "moe_linear: workspace %zu < %zu bytes", workspace_bytes, need);
  moe::LinearArgs a = {};
  a.T = T; a.N = N; a.K = K;
  a.x = static_cast<const __half*>(x);
  a.ldx = ldx;
  a.w = static_cast<const __half*>(w);
  a.bias = bias;
  a.act = act;
  a.residual = residual;
  a.ldr = ldr;
  a.y = y;
  a.y32 = y_type == MOE_F32;
  a.ldy = ldy;
  a.flags = static_cast<int32_t*>(workspace);
  const dim3 grid((unsigned)((N + 15) / 16), (unsigned)std::min((T + 15) / 16, 65535));
  moe::linear_plain_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return moe::check_launch("linear");
}

}  // extern "C"
