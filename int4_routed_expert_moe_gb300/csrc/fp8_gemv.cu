// Block-scaled FP8 product for a few tokens: the weights are read once and
// that is the cost (N K bytes against 2 T N K operations), so the kernel is a
// weight stream. A block owns 16 rows of W, its warps take the 128-column
// scale blocks in turn, and a warp's share of a block goes straight from
// global memory to registers in 16-byte pieces.
//
// The dot products run on m16n8k32 MMAs (16 rows by 8 tokens): the order of
// the reduction index inside a scale block is free as long as both operands
// agree, so lane (g, q) loads 16-byte pieces q and q + 4 of rows g and g + 8
// and of token g, and word i of each piece is an operand of MMA i. Staging W
// through shared memory for tcgen05 costs about 2000 cycles before the first
// MMA and some 600 per scale block here (barriers, copies and MMAs issued one
// by one); this form starts with the loads. Measured, us, here against the
// tensor-memory kernel: 4096 x 2048, 1 token 2.8 / 6.5, 16 tokens 3.7 / 6.5;
// 8192 x 8192, 1 token 10.3 (6.5 TB/s) / 22, 16 tokens 16.5 / 22; at 32 tokens
// the two were even, so this takes up to 16.
//
// FFN form. Where x and h are small (up to 32 scale blocks each: one pass of
// a block's threads), every block quantises them for itself into shared
// memory, FP16 x in the gate/up launch and FP32 h in the down launch. Beyond
// that x is quantised by a launch of its own, and the gate/up launch runs
// clusters of eight blocks, which together own the 128 columns of one scale
// block of h: they exchange their tokens' largest magnitudes through
// distributed shared memory and store h as codes. Measured, us per call: one
// token, 2048 x 1024: 5.5 against 6.3 with clusters; two tokens, 2048 x 4096
// (64 blocks): 10.0 against 9.4.
#include <algorithm>

#include "common.h"
#include "device.cuh"
#include "fp8.cuh"
#include "fp8_gemv.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void mma_m16n8k32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

struct GemvArgs {
  int T, N, K, nb;
  const uint8_t* xq;  // codes [T][K] and scales [T][nb], or
  const float* xs;
  const void* xf;     // FP16 or FP32 activations [T][K]
  const uint8_t *w, *w2;
  const float *ws, *ws2;
  __half* y;          // [T][N]
  float* h;           // gate/up: h in FP32 [T][N], or
  uint8_t* hq;        // codes [T][N] and scales [T][nbh]
  float* hs;
  int nbh;
};

// A scale block's weights of one matrix: pieces q and q + 4 of rows g, g + 8.
struct WFrag {
  uint4 lo[2], hi[2];  // [piece] of row g / row g + 8
};
__device__ __forceinline__ void load_w(WFrag& f, const uint8_t* lo, const uint8_t* hi, int k, int K) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const bool on = k + 64 * p < K;
    f.lo[p] = on && lo ? ld_stream_v4(lo + k + 64 * p) : make_uint4(0, 0, 0, 0);
    f.hi[p] = on && hi ? ld_stream_v4(hi + k + 64 * p) : make_uint4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// How a kernel gets its activations.
enum X { kCodes, kHalf, kFloat };

// Sixteen values of an activation row, their largest magnitude and codes.
template <X XT>
struct X16;
template <>
struct X16<kHalf> {
  uint4 v[2];
  __device__ __forceinline__ void load(const void* x, size_t i, bool on) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __half*>(x) + i);
    v[0] = on ? p[0] : make_uint4(0, 0, 0, 0);
    v[1] = on ? p[1] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float amax() const {
    const uint32_t m = fp8::amax_bits(v[0], fp8::amax_bits(v[1], 0u));
    return __half2float(__ushort_as_half((unsigned short)max(m & 0xffffu, m >> 16)));
  }
  __device__ __forceinline__ uint4 encode(float inv) const { return fp8::encode16(v, inv); }
};
template <>
struct X16<kFloat> {
  float4 v[4];
  __device__ __forceinline__ void load(const void* x, size_t i, bool on) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = on ? p[j] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  __device__ __forceinline__ float amax() const {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = fmax_nan(m, fmax_nan(fmax_nan(fabsf(v[j].x), fabsf(v[j].y)), fmax_nan(fabsf(v[j].z), fabsf(v[j].w))));
    return m;
  }
  __device__ __forceinline__ uint4 encode(float inv) const {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = fp8::encode4(v[j].x * inv, v[j].y * inv, v[j].z * inv, v[j].w * inv);
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};
template <>
struct X16<kCodes> {};

// x [T][K] quantised into shared memory: unit u = t * nb + kb holds the codes
// of one scale block, eight lanes of sixteen values.
template <X XT>
__device__ __forceinline__ void load_unit(const GemvArgs& a, X16<XT>& v) {
  const int u = (int)(threadIdx.x >> 3), t = u / a.nb, c = (u - t * a.nb) * fp8::kBlock + 16 * (threadIdx.x & 7);
  v.load(a.xf, (size_t)t * a.K + c, u < a.T * a.nb && c < a.K);
}
template <X XT>
__device__ __forceinline__ void quantize_unit(const GemvArgs& a, const X16<XT>& v, uint8_t (*codes)[fp8::kBlock],
                                              float* scales) {
  const int u = (int)(threadIdx.x >> 3), sub = threadIdx.x & 7;
  float m = v.amax();
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const fp8::BlockScale b = fp8::block_scale(m);
  if (u < a.T * a.nb) {
    *reinterpret_cast<uint4*>(&codes[u][16 * sub]) = v.encode(b.inv);
    if (sub == 0) scales[u] = b.scale;
  }
}

constexpr int kUnits = 4 * kWarps;  // scale blocks of x a block quantises for itself, eight lanes each
constexpr int kCluster = 8;  // blocks of 16 columns per scale block of h

__device__ __forceinline__ void st_cluster(float* p, uint32_t rank, float v) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ra), "f"(v) : "memory");
}

// NB: tiles of 8 tokens. GATEUP: gate and up rows, h out (as codes, by
// clusters, or in FP32: HF); else one matrix, y out. EARLY: the launch before
// this one is of the same call and starts it only after everything before the
// call has finished, so the weights may be read before that launch's results
// are waited for.
template <int NB, bool GATEUP, X XT, bool HF, bool EARLY>
__global__ void __launch_bounds__(32 * kWarps, 2) fp8_gemv_kernel(const GemvArgs a) {
  constexpr int NP = GATEUP ? 2 : 1;  // projections
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  constexpr bool XF = XT != kCodes;
  if (GATEUP && !HF) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int n0 = blockIdx.x * 16;
  const bool on_lo = n0 + g < a.N, on_hi = n0 + g + 8 < a.N;
  const int wb = min(n0, a.N - 1) / fp8::kBlock;
  const uint8_t *lo[NP], *hi[NP];
  const float* ws[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const uint8_t* w = p ? a.w2 : a.w;
    lo[p] = on_lo ? w + (size_t)(n0 + g) * a.K : nullptr;
    hi[p] = on_hi ? w + (size_t)(n0 + g + 8) * a.K : nullptr;
    ws[p] = (p ? a.ws2 : a.ws) + (size_t)wb * a.nb;
  }
  __shared__ __align__(16) uint8_t xcodes[XF ? kUnits : 1][fp8::kBlock];
  __shared__ float xscales[XF ? kUnits : 1];
  // A step is one scale block; a warp takes steps warp, warp + 8, ... with the
  // loads of the next DEPTH on their way.
  constexpr int DEPTH = NB == 1 ? 2 : 1;
  WFrag wf[DEPTH][NP];
  uint4 x[DEPTH][NB][2];
  float s0[DEPTH][NB], s1[DEPTH][NB], sw[DEPTH][NP];  // scales of tokens 2q and 2q + 1 of each tile, of the rows
  auto load_weights = [&](int d, int kb) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      load_w(wf[d][p], lo[p], hi[p], kb * fp8::kBlock + 16 * q, a.K);  // past K: nothing
      sw[d][p] = kb < a.nb ? ws[p][kb] : 0.0f;
    }
  };
  auto load_tokens = [&](int d, int kb) {
    const int k = kb * fp8::kBlock + 16 * q;
    const bool in = kb < a.nb;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int t = 8 * i + g, ta = 8 * i + 2 * q;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        x[d][i][p] = make_uint4(0, 0, 0, 0);
        if (XF) {
          if (in && t < a.T) x[d][i][p] = *reinterpret_cast<const uint4*>(&xcodes[t * a.nb + kb][16 * q + 64 * p]);
        } else if (t < a.T && k + 64 * p < a.K) {
          x[d][i][p] = *reinterpret_cast<const uint4*>(a.xq + (size_t)t * a.K + k + 64 * p);
        }
      }
      s0[d][i] = in && ta < a.T ? (XF ? xscales[ta * a.nb + kb] : a.xs[(size_t)ta * a.nb + kb]) : 0.0f;
      s1[d][i] = in && ta + 1 < a.T ? (XF ? xscales[(ta + 1) * a.nb + kb] : a.xs[(size_t)(ta + 1) * a.nb + kb]) : 0.0f;
    }
  };
  X16<XT> xv;
  if (!EARLY) {
    griddep_wait();
    if constexpr (XF) load_unit<XT>(a, xv);  // ahead of the weights: its way is the longer one
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load_weights(d, warp + d * kWarps);
  if (EARLY) {
    griddep_wait();
    if constexpr (XF) load_unit<XT>(a, xv);
  }
  griddep_launch_dependents();
  if constexpr (XF) {
    quantize_unit<XT>(a, xv, xcodes, xscales);
    __syncthreads();
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load_tokens(d, warp + d * kWarps);

  float tot[NP][NB][4] = {};
  for (int kb0 = warp; kb0 < a.nb; kb0 += DEPTH * kWarps) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int kb = kb0 + d * kWarps;
      if (kb >= a.nb) break;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const WFrag& w = wf[d][p];
          float c[4] = {};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_m16n8k32(c, word(w.lo[0], j), word(w.hi[0], j), word(w.lo[1], j), word(w.hi[1], j),
                         word(x[d][i][0], j), word(x[d][i][1], j));
          const float u0 = s0[d][i] * sw[d][p], u1 = s1[d][i] * sw[d][p];
          tot[p][i][0] = fmaf(c[0], u0, tot[p][i][0]);
          tot[p][i][1] = fmaf(c[1], u1, tot[p][i][1]);
          tot[p][i][2] = fmaf(c[2], u0, tot[p][i][2]);
          tot[p][i][3] = fmaf(c[3], u1, tot[p][i][3]);
        }
      load_weights(d, kb + DEPTH * kWarps);
      load_tokens(d, kb + DEPTH * kWarps);
    }
  }
  // The warps' sums, added in warp order: thread (t, n) of 16 tokens.
  __shared__ float red[kWarps][NP][8 * NB][17];
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[warp][p][8 * i + 2 * q + (e & 1)][g + 8 * (e >> 1)] = tot[p][i][e];
  __syncthreads();
  static_assert(16 * 8 * NB <= 32 * kWarps, "a thread per (token, row)");
  const int t = threadIdx.x >> 4, n = threadIdx.x & 15;
  const bool on = t < min(8 * NB, a.T);
  float v[NP] = {};
  if (on) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v[p] += red[w][p][t][n];
  }
  if (!GATEUP) {
    if (on && n0 + n < a.N) a.y[(size_t)t * a.N + n0 + n] = __float2half_rn(v[0]);
    return;
  }
  const float h = fp8::silu(v[0]) * v[NP - 1];
  if (HF) {
    if (on && n0 + n < a.N) a.h[(size_t)t * a.N + n0 + n] = h;
    return;
  }
  // h's block's largest magnitude: 16 columns here, the cluster's 128.
  float m = fabsf(h);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  __shared__ float amax[kCluster][8 * NB];
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every block of the cluster has started
  if (on && n < kCluster) st_cluster(&amax[rank][t], (uint32_t)n, m);
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (!on) return;
#pragma unroll
  for (int r = 0; r < kCluster; ++r) m = fmax_nan(m, amax[r][t]);
  const fp8::BlockScale b = fp8::block_scale(m);
  if (n0 + n < a.N) a.hq[(size_t)t * a.N + n0 + n] = (uint8_t)fp8::encode2(h * b.inv, 0.0f);
  if (rank == 0 && n == 0) a.hs[(size_t)t * a.nbh + n0 / fp8::kBlock] = b.scale;
}

template <int NB, bool GATEUP, X XT, bool HF, bool EARLY>
int launch(const GemvArgs& a, cudaStream_t st) {
  constexpr bool kClusters = GATEUP && !HF;
  cudaLaunchConfig_t cfg = {};
  const int tiles = (a.N + 15) / 16;
  cfg.gridDim = dim3((unsigned)(kClusters ? (tiles + kCluster - 1) / kCluster * kCluster : tiles));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kClusters ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_gemv_kernel<NB, GATEUP, XT, HF, EARLY>, a);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "fp8 gemv launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}
template <bool GATEUP, X XT, bool HF, bool EARLY>
int launch(const GemvArgs& a, cudaStream_t st) {
  return a.T <= 8 ? launch<1, GATEUP, XT, HF, EARLY>(a, st) : launch<2, GATEUP, XT, HF, EARLY>(a, st);
}

}  // namespace

int fp8_gemv(const uint8_t* xq, const float* xs, int T, const uint8_t* wq, const float* ws, int N, int K, __half* y,
             cudaStream_t st) {
  GemvArgs a = {};
  a.T = T; a.N = N; a.K = K;
  a.nb = (K + fp8::kBlock - 1) / fp8::kBlock;
  a.xq = xq; a.xs = xs;
  a.w = wq; a.ws = ws;
  a.y = y;
  return launch<false, kCodes, false, false>(a, st);
}

int fp8_gemv_ffn(const __half* x, int T, int H, int Is, const uint8_t* wg, const float* sg, const uint8_t* wu,
                 const float* su, const uint8_t* wd, const float* sd, uint8_t* xq, float* xs, uint8_t* hq, float* hs,
                 float* h, __half* y, cudaStream_t st) {
  GemvArgs a = {};
  a.T = T; a.N = Is; a.K = H;
  a.nb = (H + fp8::kBlock - 1) / fp8::kBlock;
  a.w = wg; a.ws = sg;
  a.w2 = wu; a.ws2 = su;
  a.nbh = (Is + fp8::kBlock - 1) / fp8::kBlock;
  const bool small = T * std::max(a.nb, a.nbh) <= kUnits;
  int rc;
  if (small) {
    a.xf = x;
    a.h = h;
    rc = launch<true, kHalf, true, false>(a, st);
  } else {
    if ((rc = launch_quantize_fp8(x, T, H, 1, xq, xs, st)) != MOE_OK) return rc;
    a.xq = xq; a.xs = xs;
    a.hq = hq; a.hs = hs;
    rc = launch<true, kCodes, false, true>(a, st);
  }
  if (rc != MOE_OK) return rc;
  a.N = H; a.K = Is;
  a.nb = a.nbh;
  a.w = wd; a.ws = sd;
  a.y = y;
  if (small) {
    a.xf = h;
    return launch<false, kFloat, false, true>(a, st);
  }
  a.xq = hq; a.xs = hs;
  return launch<false, kCodes, false, true>(a, st);
}

}  // namespace moe
