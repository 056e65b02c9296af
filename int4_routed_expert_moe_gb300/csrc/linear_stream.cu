// y = act(x W^T + bias) + residual for a few tokens: the weights are read once
// and that is the cost (2 N K bytes against 2 T N K operations), so the kernel
// is a weight stream. A block owns 16 rows of W, its warps take steps of 64
// columns in turn, and a warp's share of a step goes straight from global
// memory to registers in 16-byte pieces.
//
// The dot products run on m16n8k16 MMAs (16 rows by 8 tokens), whose order
// along K is free as long as both operands agree: lane (g, q) loads the pieces
// at columns 8 q and 32 + 8 q of rows g and g + 8 and of token g, and words 2 i
// and 2 i + 1 of a piece are the operands of MMA i. Each step's MMAs start from
// zero, and a warp adds its steps in FP32 (an MMA cuts the running sum off: in one
// accumulator for all of a warp's K, 8192 terms of K = 65536, terms of one sign
// were 875 2^-24 off, so 8 2^-24, and a router's logits over K = 2048 3.5e-7, so
// 1.3e-7); the loads hide the additions. The warps' sums are added in warp order.
//
// Measured, us: one token, 256 x 2048 2.4 (a launch's latency), 4096 x 4096 6.6,
// 8192 x 8192 22.3 (6.0 TB/s, 89 % of the measured copy rate); 16 tokens 2.9,
// 7.9 and 24.9.
#include "common.h"
#include "device.cuh"
#include "kernels.h"
#include "linear.cuh"

namespace moe {
namespace {

constexpr int kStep = 64;
constexpr int kSms = 152;  // of a GB300: where the variants below change over

__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// NB: tiles of 8 tokens. DEPTH: steps whose loads are on their way; with one, four
// blocks per SM (with 68 registers three fit: 16 tokens of 8192 x 8192 34.8 us).
template <int NB, int DEPTH, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, DEPTH == 1 ? 4 : 16 / kWarps) linear_stream_kernel(const LinearArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * 16, steps = (a.K + kStep - 1) / kStep;
  const __half* lo = n0 + g < a.N ? a.w + (size_t)(n0 + g) * a.K : nullptr;
  const __half* hi = n0 + g + 8 < a.N ? a.w + (size_t)(n0 + g + 8) * a.K : nullptr;
  uint4 wl[DEPTH][2], wh[DEPTH][2], x[DEPTH][NB][2];
  auto load = [&](int d, int s) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int k = s * kStep + 32 * p + 8 * q;
      const uint4 z = make_uint4(0, 0, 0, 0);
      wl[d][p] = lo && k < a.K ? ld_stream_v4(lo + k) : z;
      wh[d][p] = hi && k < a.K ? ld_stream_v4(hi + k) : z;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int t = 8 * i + g;
        x[d][i][p] = t < a.T && k < a.K ? *reinterpret_cast<const uint4*>(a.x + (size_t)t * (size_t)a.ldx + k) : z;
      }
    }
  };
  griddep_wait();
  griddep_launch_dependents();
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(d, warp + d * kWarps);
  float c[NB][4] = {};
  for (int s0 = warp; s0 < steps; s0 += DEPTH * kWarps) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int s = s0 + d * kWarps;
      if (s >= steps) break;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        float m[4] = {};
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            mma_m16n8k16(m, word(wl[d][p], 2 * j), word(wh[d][p], 2 * j), word(wl[d][p], 2 * j + 1),
                         word(wh[d][p], 2 * j + 1), word(x[d][i][p], 2 * j), word(x[d][i][p], 2 * j + 1));
#pragma unroll
        for (int e = 0; e < 4; ++e) c[i][e] += m[e];
      }
      load(d, s + DEPTH * kWarps);
    }
  }
  // Thread (t, n) of 16 tokens and 16 rows.
  __shared__ float red[kWarps][8 * NB][17];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][8 * i + 2 * q + (e & 1)][g + 8 * (e >> 1)] = c[i][e];
  __syncthreads();
  const int t = threadIdx.x >> 4, n = threadIdx.x & 15;
  if (t >= min(8 * NB, a.T)) return;
  float v[1] = {};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v[0] += red[w][t][n];
  if (n0 + n >= a.N) return;
  if (a.bias) v[0] += a.bias[n0 + n];
  activate<false>(a.act, v);
  const size_t at = (size_t)t * (size_t)a.ldy + n0 + n, ra = (size_t)t * (size_t)a.ldr + n0 + n;
  if (a.y32) {
    if (a.residual) v[0] += static_cast<const float*>(a.residual)[ra];
    static_cast<float*>(a.y)[at] = v[0];
  } else {
    if (a.residual) v[0] += __half2float(static_cast<const __half*>(a.residual)[ra]);
    static_cast<__half*>(a.y)[at] = __float2half_rn(v[0]);
  }
}

template <int NB, int DEPTH, int kWarps>
int launch_stream(const LinearArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + 15) / 16));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_stream_kernel<NB, DEPTH, kWarps>, a);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "moe_linear launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}

}  // namespace

int linear_stream(const LinearArgs& a, cudaStream_t st) {
  if (a.T <= 8) return launch_stream<1, 4, 8>(a, st);
  // Two tiles of tokens, us at 16 tokens: where the SMs have a block each at
  // most and K is long, 16 warps per block (2048 x 4096: 6.3 against 7.0); where
  // they have three and more, one step ahead is enough and leaves registers for
  // more blocks (8192 x 8192: 24.4 against 26.5; 4096 x 4096: 9.9 against 8.8).
  const int blocks = (a.N + 15) / 16;
  if (blocks <= kSms && a.K >= 4096) return launch_stream<2, 2, 16>(a, st);
  if (blocks >= 3 * kSms) return launch_stream<2, 1, 8>(a, st);
  return launch_stream<2, 2, 8>(a, st);
}

}  // namespace moe
