// FP16 to FP8 (E4M3) with one FP32 scale per block: 1 x 128 for activations,
// 128 x 128 for weights. Per block: amax = max |x|, s = amax / 448,
// q = E4M3(x * (448 * (1 / amax))) rounded to nearest even, so that x ~ q * s and
// the largest value takes the type's largest code.
//
// Memory-bound: 2 bytes read and 1 written per element; every value is read
// once, 32 bytes per thread, and stays in registers between the maximum and the
// rounding. 8192 x 4096 activations: 16.4 us, 6.2 TB/s, 92 % of the measured
// copy rate. 4040 x 2048 weights (in L2): 3.5 us.
#include <cuda_fp8.h>

#include "common.h"
#include "device.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Activations: eight lanes per 1 x 128 block, sixteen values per lane.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __half* __restrict__ x, unsigned units, int cols,
                                                            int cblocks, uint8_t* __restrict__ q,
                                                            float* __restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
  // The call admits 2^30 - 1 units: their threads would not fit 32 bits.
  const unsigned u = blockIdx.x * 32u + (threadIdx.x >> 3);
  const int sub = threadIdx.x & 7;
  const unsigned r = u / (unsigned)cblocks;
  const int cb = (int)(u - r * (unsigned)cblocks), c0 = cb * 128 + sub * 16;
  const bool on = u < units && c0 < cols;
  uint4 in[2] = {};
  if (on) {
    const uint4* p = reinterpret_cast<const uint4*>(x + (size_t)r * cols + c0);
    in[0] = p[0];
    in[1] = p[1];
  }
  uint32_t m = fp8::amax_bits(in[0], fp8::amax_bits(in[1], 0u));
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const fp8::BlockScale b = fp8::block_scale(m);
  if (on) *reinterpret_cast<uint4*>(q + (size_t)r * cols + c0) = fp8::encode16(in, b.inv);
  if (u < units && sub == 0) scales[u] = b.scale;
}

// Weights: one block of 256 threads per 128 x 128 block; its values stay in
// registers between the maximum and the rounding.
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const __half* __restrict__ x, int rows, int cols,
                                                             uint8_t* __restrict__ q, float* __restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 7, r0 = blockIdx.y * 128 + (threadIdx.x >> 3);
  const int c0 = blockIdx.x * 128 + sub * 16;
  uint4 in[4][2] = {};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (r0 + 32 * i < rows && c0 < cols) {
      const uint4* p = reinterpret_cast<const uint4*>(x + (size_t)(r0 + 32 * i) * cols + c0);
      in[i][0] = p[0];
      in[i][1] = p[1];
      m = fp8::amax_bits(in[i][0], fp8::amax_bits(in[i][1], m));
    }
  }
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  __shared__ uint32_t wm[8];
  if ((threadIdx.x & 31) == 0) wm[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, wm[w]);
  const fp8::BlockScale b = fp8::block_scale(m);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + 32 * i < rows && c0 < cols)
      *reinterpret_cast<uint4*>(q + (size_t)(r0 + 32 * i) * cols + c0) = fp8::encode16(in[i], b.inv);
  if (threadIdx.x == 0) scales[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = b.scale;
}

}  // namespace

int launch_quantize_fp8(const __half* x, int rows, int cols, int block_rows, uint8_t* q, float* scales,
                        cudaStream_t st) {
  const int cblocks = (cols + 127) / 128;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (block_rows == 1) {
    const unsigned units = (unsigned)rows * (unsigned)cblocks;
    cfg.gridDim = dim3((units + 31) / 32);
    e = cudaLaunchKernelEx(&cfg, quantize_rows_kernel, x, units, cols, cblocks, q, scales);
  } else {
    cfg.gridDim = dim3((unsigned)cblocks, (unsigned)((rows + 127) / 128));
    e = cudaLaunchKernelEx(&cfg, quantize_tiles_kernel, x, rows, cols, q, scales);
  }
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "quantize launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}

}  // namespace moe

extern "C" int moe_quantize_fp8(const void* x, int rows, int cols, int block_rows, void* q, float* scales,
                                void* stream) {
  moe::NvtxRange nvtx_range("moe_quantize_fp8");
  moe::clear_error();
  if (rows < 0 || cols < 16 || cols % 16 || cols > 65536 || (block_rows != 1 && block_rows != 128))
    return moe::fail(MOE_ERR_ARG, "moe_quantize_fp8: need cols a multiple of 16 up to 65536, block_rows 1 or 128 "
                     "(rows=%d cols=%d block_rows=%d)", rows, cols, block_rows);
  if ((long long)rows * ((cols + 127) / 128) > 0x3fffffffLL || (block_rows == 128 && rows > 65535 * 128))
    return moe::fail(MOE_ERR_ARG, "moe_quantize_fp8: too many blocks (rows=%d cols=%d)", rows, cols);
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scales) return moe::fail(MOE_ERR_ARG, "moe_quantize_fp8: NULL pointer");
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q)) % 16 ||
      reinterpret_cast<uintptr_t>(scales) % 4)
    return moe::fail(MOE_ERR_ARG, "moe_quantize_fp8: x and q must be 16-byte aligned, scales 4-byte");
  return moe::launch_quantize_fp8(static_cast<const __half*>(x), rows, cols, block_rows, static_cast<uint8_t*>(q),
                                  scales, static_cast<cudaStream_t>(stream));
}
