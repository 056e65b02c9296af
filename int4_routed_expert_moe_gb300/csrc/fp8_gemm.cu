// Block-scaled FP8 matrix product and the shared SwiGLU FFN built from it.
//   y[t][n] = sum_b xs[t][b] ws[n/128][b] sum_{c in block b} xq[t][c] wq[n][c]
// with E4M3 codes, one scale per 1 x 128 block of x and per 128 x 128 block of
// W, FP32 sums.
#include <cuda_fp8.h>

#include "common.h"
#include "device.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 32;

__device__ __forceinline__ float decode1(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return (float)v;
}

// 64 tokens x 64 rows of W per block of 256 threads, 4 x 4 sums per thread;
// the sums of a 128-element block are scaled as they join the total.
template <bool F32OUT>
__global__ void __launch_bounds__(256) fp8_matmul_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ xs,
                                                         int T, const uint8_t* __restrict__ wq,
                                                         const float* __restrict__ ws, int N, int K, void* y) {
  __shared__ float sx[kTile][kStep + 1], sw[kTile][kStep + 1];
  const int n0 = blockIdx.x * kTile, t0 = blockIdx.y * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int nb = (K + fp8::kBlock - 1) / fp8::kBlock;
  float total[4][4] = {};
  for (int b = 0; b < nb; ++b) {
    float acc[4][4] = {};
    for (int k0 = b * fp8::kBlock; k0 < min(K, (b + 1) * fp8::kBlock); k0 += kStep) {
      __syncthreads();
      for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
        const int r = i / kStep, c = i % kStep;
        const bool kc = k0 + c < K;
        sx[r][c] = kc && t0 + r < T ? decode1(xq[(size_t)(t0 + r) * K + k0 + c]) : 0.0f;
        sw[r][c] = kc && n0 + r < N ? decode1(wq[(size_t)(n0 + r) * K + k0 + c]) : 0.0f;
      }
      __syncthreads();
#pragma unroll 8
      for (int c = 0; c < kStep; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sx[ty * 4 + i][c], sw[tx * 4 + j][c], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (t < T && n < N)
          total[i][j] = fmaf(xs[(size_t)t * nb + b] * ws[(size_t)(n / fp8::kBlock) * nb + b], acc[i][j], total[i][j]);
      }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (t < T && n < N) {
        if (F32OUT) static_cast<float*>(y)[(size_t)t * N + n] = total[i][j];
        else static_cast<__half*>(y)[(size_t)t * N + n] = __float2half_rn(total[i][j]);
      }
    }
}

// h = silu(gate) * up, quantised in 1 x 128 blocks: a warp per block.
__global__ void __launch_bounds__(256) swiglu_quantize_kernel(const float* __restrict__ gate,
                                                              const float* __restrict__ up, unsigned units, int cols,
                                                              int cblocks, uint8_t* __restrict__ q,
                                                              float* __restrict__ scales) {
  const unsigned u = (blockIdx.x * 256u + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (u >= units) return;
  const unsigned r = u / (unsigned)cblocks;
  const int c0 = (int)(u - r * (unsigned)cblocks) * 128 + lane * 4;
  float h[4] = {};
  float m = 0.0f;
  bool bad = false;
  if (c0 < cols) {
    for (int j = 0; j < 4; ++j) {
      const size_t i = (size_t)r * cols + c0 + j;
      h[j] = silu_f(gate[i]) * up[i];
      bad |= !(fabsf(h[j]) < INFINITY);
      m = fmaxf(m, fabsf(h[j]));
    }
  }
  if (bad) m = INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const fp8::BlockScale b = fp8::block_scale(m);
  if (c0 < cols)
    *reinterpret_cast<uint32_t*>(q + (size_t)r * cols + c0) =
        fp8::encode4(h[0] * b.inv, h[1] * b.inv, h[2] * b.inv, h[3] * b.inv);
  if (lane == 0) scales[u] = b.scale;
}

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }
inline int blocks128(int n) { return (n + 127) / 128; }

int launch_matmul(const uint8_t* xq, const float* xs, int T, const uint8_t* wq, const float* ws, int N, int K, void* y,
                  bool f32, cudaStream_t st) {
  const dim3 grid((N + kTile - 1) / kTile, (T + kTile - 1) / kTile);
  if (f32) fp8_matmul_kernel<true><<<grid, 256, 0, st>>>(xq, xs, T, wq, ws, N, K, y);
  else fp8_matmul_kernel<false><<<grid, 256, 0, st>>>(xq, xs, T, wq, ws, N, K, y);
  return check_launch("fp8 matmul");
}

// Workspace of the FFN after the header: xq, xs, hq, hs, gate, up.
struct FfnWs {
  size_t xq, xs, hq, hs, gate, up, total;
};
FfnWs ffn_ws(int T, int H, int Is) {
  FfnWs w;
  size_t o = kWorkspaceHeader;
  w.xq = o; o += round256((size_t)T * H);
  w.xs = o; o += round256((size_t)T * blocks128(H) * 4);
  w.hq = o; o += round256((size_t)T * Is);
  w.hs = o; o += round256((size_t)T * blocks128(Is) * 4);
  w.gate = o; o += round256((size_t)T * Is * 4);
  w.up = o; o += round256((size_t)T * Is * 4);
  w.total = o;
  return w;
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_matmul_fp8_workspace_bytes(int T, int N, int K) {
  if (T < 0 || N < 1 || K < 16 || K % 16) return 0;
  return moe::kWorkspaceHeader;
}

int moe_matmul_fp8(const void* xq, const float* xs, int T, const void* wq, const float* ws, int N, int K, void* y,
                   void* workspace, size_t workspace_bytes, void* stream) {
  moe::NvtxRange nvtx_range("moe_matmul_fp8");
  moe::clear_error();
  if (T < 0 || T > (1 << 20) || N < 1 || N > 65536 || K < 16 || K % 16 || K > 65536)
    return moe::fail(MOE_ERR_ARG, "moe_matmul_fp8: need 0 <= T <= 2^20, 1 <= N <= 65536, K a multiple of 16 up to "
                     "65536 (T=%d N=%d K=%d)", T, N, K);
  if (T == 0) return MOE_OK;
  if (!xq || !xs || !wq || !ws || !y || !workspace) return moe::fail(MOE_ERR_ARG, "moe_matmul_fp8: NULL pointer");
  const uintptr_t al = reinterpret_cast<uintptr_t>(xq) | reinterpret_cast<uintptr_t>(wq) | reinterpret_cast<uintptr_t>(y);
  if (al % 16 || (reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(ws)) % 4 ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return moe::fail(MOE_ERR_ARG, "moe_matmul_fp8: codes and y 16-byte, scales 4-byte, workspace 256-byte aligned");
  const size_t need = moe_matmul_fp8_workspace_bytes(T, N, K);
  if (workspace_bytes < need)
    return moe::fail(MOE_ERR_CAPACITY, "moe_matmul_fp8: workspace %zu < %zu bytes", workspace_bytes, need);
  return moe::launch_matmul(static_cast<const uint8_t*>(xq), xs, T, static_cast<const uint8_t*>(wq), ws, N, K, y,
                            false, static_cast<cudaStream_t>(stream));
}

size_t moe_shared_fp8_workspace_bytes(int T, int H, int Is) {
  if (T < 0 || H <= 0 || Is <= 0 || H % 64 || Is % 64) return 0;
  return moe::ffn_ws(T, H, Is).total;
}

int moe_shared_forward_fp8(const void* x, int T, int H, int Is, const void* wg, const float* sg, const void* wu,
                           const float* su, const void* wd, const float* sd, void* y, void* workspace,
                           size_t workspace_bytes, void* stream) {
  moe::NvtxRange nvtx_range("moe_shared_forward_fp8");
  moe::clear_error();
  if (T < 0 || T > (1 << 20) || H <= 0 || Is <= 0 || H % 64 || Is % 64 || H > 65536 || Is > 65536)
    return moe::fail(MOE_ERR_ARG, "moe_shared_forward_fp8: need 0 <= T <= 2^20, H, Is positive multiples of 64 up to "
                     "65536 (H=%d Is=%d T=%d)", H, Is, T);
  if (T == 0) return MOE_OK;
  if (!x || !wg || !sg || !wu || !su || !wd || !sd || !y || !workspace)
    return moe::fail(MOE_ERR_ARG, "moe_shared_forward_fp8: NULL pointer");
  const uintptr_t al = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(wg) |
                       reinterpret_cast<uintptr_t>(wu) | reinterpret_cast<uintptr_t>(wd) |
                       reinterpret_cast<uintptr_t>(y);
  const uintptr_t sl = reinterpret_cast<uintptr_t>(sg) | reinterpret_cast<uintptr_t>(su) |
                       reinterpret_cast<uintptr_t>(sd);
  if (al % 16 || sl % 4 || reinterpret_cast<uintptr_t>(workspace) % 256)
    return moe::fail(MOE_ERR_ARG, "moe_shared_forward_fp8: x, weights, y 16-byte, scales 4-byte and workspace "
                     "256-byte aligned");
  const size_t need = moe_shared_fp8_workspace_bytes(T, H, Is);
  if (workspace_bytes < need)
    return moe::fail(MOE_ERR_CAPACITY, "moe_shared_forward_fp8: workspace %zu < %zu bytes", workspace_bytes, need);
  const moe::FfnWs o = moe::ffn_ws(T, H, Is);
  uint8_t* w8 = static_cast<uint8_t*>(workspace);
  uint8_t *xq = w8 + o.xq, *hq = w8 + o.hq;
  float *xs = reinterpret_cast<float*>(w8 + o.xs), *hs = reinterpret_cast<float*>(w8 + o.hs);
  float *gate = reinterpret_cast<float*>(w8 + o.gate), *up = reinterpret_cast<float*>(w8 + o.up);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc = moe::launch_quantize_fp8(static_cast<const __half*>(x), T, H, 1, xq, xs, st);
  if (rc != MOE_OK) return rc;
  if ((rc = moe::launch_matmul(xq, xs, T, static_cast<const uint8_t*>(wg), sg, Is, H, gate, true, st))) return rc;
  if ((rc = moe::launch_matmul(xq, xs, T, static_cast<const uint8_t*>(wu), su, Is, H, up, true, st))) return rc;
  const unsigned units = (unsigned)T * (unsigned)moe::blocks128(Is);
  moe::swiglu_quantize_kernel<<<(units + 7) / 8, 256, 0, st>>>(gate, up, units, Is, moe::blocks128(Is), hq, hs);
  if ((rc = moe::check_launch("swiglu quantize"))) return rc;
  return moe::launch_matmul(hq, hs, T, static_cast<const uint8_t*>(wd), sd, H, Is, y, false, st);
}

}  // extern "C"
