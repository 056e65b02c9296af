// Norms before and after a block, fused with its gate, scales and residual,
// and with the FP8 quantisation of what comes out:
//   a = branch or norm(branch);  h = rs * residual + s * gate * a;  y = norm(h)
// RMS: v / sqrt(mean v^2 + eps) * w; layer: the same of v - mean v, plus b.
//
// About a dozen operations per element, so bytes are the bound: every row is
// read once, stays in registers between the sums and the outputs, and each
// output is written once. A row is shared by whole warps, eight consecutive
// elements per lane and step; a 1 x 128 scale block is then sixteen lanes of a
// warp. Measured: 8192 x 4096, FP32 stream, channel gate, FP16 and codes out
// 66.8 us, 6.55 TB/s, 97 % of the measured copy rate; 8192 x 4096 FP16 x alone 23 us
// (partly in L2); one token of 2048 1.8 us.
#include <algorithm>

#include "common.h"
#include "device.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxVec = 4;  // eight elements each, per lane

struct NormArgs {
  int T, H;
  int warps;      // per row
  int rows;       // per block
  int gate_kind;
  float eps, off, inv_h, scale, rscale;
  const __half *branch, *pw, *pb, *w, *b;
  const void *res, *gate;
  void* h;
  __half* y;
  uint8_t* q;
  float* scales;
  int nb;
  int32_t *clear, *into, *from[2];  // error words of a whole block's workspace
};

__device__ __forceinline__ void widen(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(u32_as_h2(u[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void load8(const __half* p, float (&f)[8]) { widen(*reinterpret_cast<const uint4*>(p), f); }
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(__half* p, const float (&f)[8]) { *reinterpret_cast<uint4*>(p) = narrow(f); }
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The row's sum; red: the block's warps' sums. Every warp of the block calls it.
__device__ __forceinline__ float row_sum(float v, int warps, float* red) {
  v = warp_sum(v);
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5;
  __syncthreads();  // the sums before these have been read
  if ((threadIdx.x & 31) == 0) red[threadIdx.y * warps + warp] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < warps; ++i) v += red[threadIdx.y * warps + i];
  return v;
}

// v becomes its norm, elements [8 (lane + 32 warps i), + 8) of the row.
template <int V, bool LAYER>
__device__ __forceinline__ void norm_row(float (&v)[V][8], const NormArgs& a, const __half* w, const __half* b,
                                         float* red) {
  const int step = 256 * a.warps;
  if (LAYER) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) m += v[i][e];
    m = row_sum(m, a.warps, red) * a.inv_h;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((int)threadIdx.x * 8 + i * step < a.H)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] -= m;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[i][e], v[i][e], s);
  const float r = rsqrtf(row_sum(s, a.warps, red) * a.inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x * 8 + i * step;
    if (c < a.H) {
      float wv[8];
      load8(w + c, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * r * (wv[e] + a.off);
      if (LAYER && b) {
        load8(b + c, wv);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] += wv[e];
      }
    }
  }
}

// S: the residual stream's type; BRANCH: moe_norm_residual. With 32 elements
// per lane of branch and residual the compiler saves registers by loading them
// in turns unless one block per SM is asked for (8192 x 16384: 374 us, so 277);
// the other variants are faster as they come.
template <int V, typename S, bool LAYER, bool BRANCH>
__global__ void __launch_bounds__(kMaxThreads, BRANCH && V == 4 ? 1 : 0) norm_kernel(const NormArgs a) {
  __shared__ float red[kMaxThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  if (a.clear || a.into) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && threadIdx.y == 0) {
      if (a.clear) *a.clear = 0;
      for (int i = 0; a.into && i < 2; ++i)
        if (a.from[i] && *a.from[i]) {
          *a.into |= *a.from[i];
          *a.from[i] = 0;
        }
    }
  }
  const long long t = (long long)blockIdx.x * a.rows + threadIdx.y;
  const bool live = t < a.T;
  const size_t row = (size_t)(live ? t : 0) * a.H;
  const int step = 256 * a.warps;
  float v[V][8];
  const S* res = static_cast<const S*>(a.res);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x * 8 + i * step;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
    if (live && c < a.H && (!BRANCH || res)) load8(res + row + c, v[i]);
  }
  if (BRANCH) {
    float br[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x * 8 + i * step;
#pragma unroll
      for (int e = 0; e < 8; ++e) br[i][e] = 0.0f;
      if (live && c < a.H) load8(a.branch + row + c, br[i]);
    }
    if (a.pw) norm_row<V, LAYER>(br, a, a.pw, a.pb, red);
    float s = a.scale;
    if (a.gate_kind == MOE_GATE_TOKEN && live) s *= static_cast<const float*>(a.gate)[t];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x * 8 + i * step;
      if (live && c < a.H) {
        if (a.gate_kind >= MOE_GATE_CHANNEL) {
          float g[8];
          load8(static_cast<const __half*>(a.gate) + (a.gate_kind == MOE_GATE_ELEMENT ? row : 0) + c, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) br[i][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = res ? fmaf(br[i][e], s, v[i][e] * a.rscale) : br[i][e] * s;
        if (a.h) store8(static_cast<S*>(a.h) + row + c, v[i]);
      }
    }
    if (!a.w) return;
  }
  norm_row<V, LAYER>(v, a, a.w, a.b, red);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x * 8 + i * step;
    const bool on = live && c < a.H;
    if (a.y && on) store8(a.y + row + c, v[i]);
    if (a.q) {  // a scale block: sixteen lanes
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmax_nan(m, fabsf(v[i][e]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const fp8::BlockScale s = fp8::block_scale(m);
      if (on) {
        uint2 code;
        code.x = fp8::encode4(v[i][0] * s.inv, v[i][1] * s.inv, v[i][2] * s.inv, v[i][3] * s.inv);
        code.y = fp8::encode4(v[i][4] * s.inv, v[i][5] * s.inv, v[i][6] * s.inv, v[i][7] * s.inv);
        *reinterpret_cast<uint2*>(a.q + row + c) = code;
        if ((threadIdx.x & 15) == 0) a.scales[(size_t)t * a.nb + c / fp8::kBlock] = s.scale;
      }
    }
  }
}

template <int V, typename S>
cudaError_t launch(const cudaLaunchConfig_t& cfg, const NormArgs& a, bool layer) {
  if (a.branch)
    return layer ? cudaLaunchKernelEx(&cfg, norm_kernel<V, S, true, true>, a)
                 : cudaLaunchKernelEx(&cfg, norm_kernel<V, S, false, true>, a);
  return layer ? cudaLaunchKernelEx(&cfg, norm_kernel<V, S, true, false>, a)
               : cudaLaunchKernelEx(&cfg, norm_kernel<V, S, false, false>, a);
}
template <typename S>
cudaError_t launch(const cudaLaunchConfig_t& cfg, const NormArgs& a, bool layer, int vec) {
  return vec == 1 ? launch<1, S>(cfg, a, layer) : vec == 2 ? launch<2, S>(cfg, a, layer) : launch<4, S>(cfg, a, layer);
}

int run_norm(const char* who, NormArgs a, bool f32, bool layer, cudaStream_t st) {
  a.inv_h = 1.0f / (float)a.H;
  a.nb = (a.H + fp8::kBlock - 1) / fp8::kBlock;
  // A small batch is over soonest with eight elements per lane (one token of
  // 4096: 1.8 us, with sixteen 2.0, with 32 2.4). From 4 M elements on, where
  // bytes count, fewer warps with more loads each: x alone takes 32 elements
  // per lane (8192 x 4096: 23.1 us, with eight 32.6), with a branch and its norm
  // or long rows sixteen (8192 x 4096: 61 and 59 us, with eight 72 and 60, with
  // 32 65 and 60).
  const int units = (a.H / 8 + 31) / 32;  // warps, with eight elements per lane
  int vec = 1;
  if ((long long)a.T * a.H >= (1 << 22)) {
    if (!a.branch) vec = units >= 4 ? 4 : units;
    else if (units >= (a.pw ? 8 : 16)) vec = 2;
    if (vec == 3) vec = 2;
  }
  while (vec * (kMaxThreads / 32) < units) vec *= 2;
  a.warps = (units + vec - 1) / vec;
  a.rows = a.warps == 1 ? 8 : a.warps == 2 ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.T + a.rows - 1) / a.rows));
  cfg.blockDim = dim3(32u * (unsigned)a.warps, (unsigned)a.rows);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = f32 ? launch<float>(cfg, a, layer, vec) : launch<__half>(cfg, a, layer, vec);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return MOE_OK;
}

bool finite(float v) { return v > -INFINITY && v < INFINITY; }

// The checks that both calls share.
int check_norm(const char* who, const moe_norm_cfg* cfg, int type, int T, int H, const void* b, bool q) {
  if (!cfg) return fail(MOE_ERR_ARG, "%s: NULL settings", who);
  if (cfg->kind != MOE_NORM_RMS && cfg->kind != MOE_NORM_LAYER)
    return fail(MOE_ERR_ARG, "%s: unknown norm %d", who, cfg->kind);
  if (!finite(cfg->eps) || cfg->eps < 0.0f || !finite(cfg->weight_offset))
    return fail(MOE_ERR_ARG, "%s: need eps >= 0, and both settings finite", who);
  if (type != MOE_F32 && type != MOE_F16) return fail(MOE_ERR_ARG, "%s: unknown type %d", who, type);
  if (T < 0 || H < 8 || H % 8 || H > 8 * 32 * kMaxVec * (kMaxThreads / 32))
    return fail(MOE_ERR_ARG, "%s: need T >= 0, H a multiple of 8 up to 16384 (T=%d H=%d)", who, T, H);
  if (q && H % 16) return fail(MOE_ERR_ARG, "%s: codes need H a multiple of 16 (H=%d)", who, H);
  if (b && cfg->kind != MOE_NORM_LAYER) return fail(MOE_ERR_ARG, "%s: only a layer norm has a bias", who);
  return MOE_OK;
}

}  // namespace

int block_norm_in(const moe_norm_cfg* cfg, const void* x, int type, int T, int H, const void* w, const void* b,
                  void* y, int32_t* clear, cudaStream_t st) {
  NormArgs a = {};
  a.T = T; a.H = H;
  a.eps = cfg->eps; a.off = cfg->weight_offset;
  a.res = x;
  a.w = static_cast<const __half*>(w);
  a.b = static_cast<const __half*>(b);
  a.y = static_cast<__half*>(y);
  a.clear = clear;
  return run_norm("moe_block_forward", a, type == MOE_F32, cfg->kind == MOE_NORM_LAYER, st);
}

int block_norm_out(const moe_norm_cfg* cfg, const void* branch, void* h, int type, int T, int H, const void* post_w,
                   const void* post_b, float scale, float residual_scale, int32_t* into, int32_t* from0,
                   int32_t* from1, cudaStream_t st) {
  NormArgs a = {};
  a.T = T; a.H = H;
  a.eps = cfg->eps; a.off = cfg->weight_offset;
  a.scale = scale; a.rscale = residual_scale;
  a.branch = static_cast<const __half*>(branch);
  a.res = h;
  a.h = h;
  a.pw = static_cast<const __half*>(post_w);
  a.pb = static_cast<const __half*>(post_b);
  a.into = into;
  a.from[0] = from0;
  a.from[1] = from1;
  return run_norm("moe_block_forward", a, type == MOE_F32, cfg->kind == MOE_NORM_LAYER, st);
}

}  // namespace moe

extern "C" {

int moe_norm(const moe_norm_cfg* cfg, const void* x, int x_type, int T, int H, const void* w, const void* b, void* y,
             void* q, float* scales, void* stream) {
  moe::NvtxRange nvtx_range("moe_norm");
  moe::clear_error();
  const int rc = moe::check_norm("moe_norm", cfg, x_type, T, H, b, q != nullptr);
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  if (!x || !w || (!y && !q) || (!q != !scales)) return moe::fail(MOE_ERR_ARG, "moe_norm: NULL pointer");
  const uintptr_t al = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(b) |
                       reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(q);
  if (al % 16 || reinterpret_cast<uintptr_t>(scales) % 4)
    return moe::fail(MOE_ERR_ARG, "moe_norm: buffers must be 16-byte aligned, scales 4-byte");
  moe::NormArgs a = {};
  a.T = T; a.H = H;
  a.eps = cfg->eps; a.off = cfg->weight_offset;
  a.res = x;
  a.w = static_cast<const __half*>(w);
  a.b = static_cast<const __half*>(b);
  a.y = static_cast<__half*>(y);
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  return moe::run_norm("moe_norm", a, x_type == MOE_F32, cfg->kind == MOE_NORM_LAYER, static_cast<cudaStream_t>(stream));
}

int moe_norm_residual(const moe_norm_cfg* cfg, const void* branch, const void* residual, int stream_type, int T, int H,
                      const void* post_w, const void* post_b, const void* gate, int gate_kind, float scale,
                      float residual_scale, void* h, const void* w, const void* b, void* y, void* q, float* scales,
                      void* stream) {
  const char* who = "moe_norm_residual";
  moe::NvtxRange nvtx_range(who);
  moe::clear_error();
  const int rc = moe::check_norm(who, cfg, stream_type, T, H, post_b ? post_b : b, q != nullptr);
  if (rc != MOE_OK) return rc;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_ELEMENT)
    return moe::fail(MOE_ERR_ARG, "%s: unknown gate %d", who, gate_kind);
  if (!moe::finite(scale) || !moe::finite(residual_scale))
    return moe::fail(MOE_ERR_ARG, "%s: scales must be finite", who);
  if (T == 0) return MOE_OK;
  const bool next = y || q;
  if (!branch || (!h && !next) || (next && !w) || (!q != !scales) || (gate_kind != MOE_GATE_NONE && !gate) ||
      (post_b && !post_w))
    return moe::fail(MOE_ERR_ARG, "%s: NULL pointer", who);
  const uintptr_t al = reinterpret_cast<uintptr_t>(branch) | reinterpret_cast<uintptr_t>(residual) |
                       reinterpret_cast<uintptr_t>(post_w) | reinterpret_cast<uintptr_t>(post_b) |
                       reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(b) |
                       reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(q) |
                       (gate_kind >= MOE_GATE_CHANNEL ? reinterpret_cast<uintptr_t>(gate) : 0);
  if (al % 16 || reinterpret_cast<uintptr_t>(scales) % 4 ||
      (gate_kind == MOE_GATE_TOKEN && reinterpret_cast<uintptr_t>(gate) % 4))
    return moe::fail(MOE_ERR_ARG, "%s: buffers must be 16-byte aligned, token gates and scales 4-byte", who);
  moe::NormArgs a = {};
  a.T = T; a.H = H;
  a.gate_kind = gate_kind;
  a.eps = cfg->eps; a.off = cfg->weight_offset;
  a.scale = scale; a.rscale = residual_scale;
  a.branch = static_cast<const __half*>(branch);
  a.res = residual;
  a.pw = static_cast<const __half*>(post_w);
  a.pb = static_cast<const __half*>(post_b);
  a.gate = gate;
  a.h = h;
  if (next) {
    a.w = static_cast<const __half*>(w);
    a.b = static_cast<const __half*>(b);
  }
  a.y = static_cast<__half*>(y);
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  return moe::run_norm(who, a, stream_type == MOE_F32, cfg->kind == MOE_NORM_LAYER, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
