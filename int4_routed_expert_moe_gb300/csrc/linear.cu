// moe_linear: argument checks and the choice between the weight stream
// (linear_stream.cu, up to 16 tokens) and the tensor-memory kernels
// (linear_gemm.cu).
#include "common.h"
#include "kernels.h"
#include "linear.cuh"

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
  a.bias_vec = reinterpret_cast<uintptr_t>(bias) % 16 == 0;
  a.act = act;
  a.residual = residual;
  a.ldr = ldr;
  a.y = y;
  a.y32 = y_type == MOE_F32;
  a.ldy = ldy;
  a.flags = static_cast<int32_t*>(workspace);
  const int esz = a.y32 ? 4 : 2;
  a.vec = ldy * esz % 16 == 0 && (!residual || ldr * esz % 16 == 0);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return T <= moe::kLinearStreamTokens ? moe::linear_stream(a, st) : moe::linear_gemm(a, st);
}

}  // extern "C"
