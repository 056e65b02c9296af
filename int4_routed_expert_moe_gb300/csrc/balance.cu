// Balance loss of a router by sequence, per-expert counts, and the gradient.
//   f_se = E c_se / (k n_s),  P_se = mean of p_te over the n_s good tokens,
//   loss = coef / S' sum_s sum_e f_se P_se,
//   dl_te = g coef / (S' n_s) p_te (f_se - sum_j f_sj p_tj) [* (1 - sigmoid(l_te))]
//
// A token's logits stay in the registers of a group of lanes: 8, 16 or 32
// lanes with 8 values each for up to 256 experts, then 32 lanes with 16 or 32.
// Forward, launch 1: chunks of consecutive tokens, one per block; each lane
// adds its experts' probabilities over the group's tokens, the block adds its
// groups in order and writes a partial row per sequence that the chunk meets,
// row chunk + sequence: (chunk, sequence) pairs along the tokens never share
// that sum, since each next pair raises one of the two. Launch 2: a block per
// sequence and 32 experts adds the partial rows in order; the last block to
// finish adds the losses in order. No floating-point atomics, so the same
// inputs give the same bits. Backward: one pass, the probabilities recomputed.
#include <algorithm>

#include "common.h"
#include "device.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kMaxChunks = 152;  // one block per SM
constexpr int kMinChunk = 32;    // tokens

struct BalanceArgs {
  const void* logits;
  long long ld;
  int T, E, k, S, chunk, chunks;
  bool sigmoid;
  float coef;
  const int32_t *ids, *offsets;
  float* psum;      // partial rows [chunks + S][E]: probabilities,
  int32_t* csum;    // counts,
  int32_t* nsum;    // [chunks + S]: good tokens
  float* lsum;      // [S][ceil(E / 32)]
  uint32_t* ticket;
  int32_t *counts, *tokens;
  float *mean, *loss;
  // backward
  const int32_t *bcounts, *btokens;
  const float* grad;
  float* dl;
  long long ldd;
  bool accumulate, vec_out;
};

__device__ __forceinline__ int offset_at(const BalanceArgs& a, int i) {
  if (!a.offsets) return i ? a.T : 0;
  return min(max(a.offsets[i], 0), a.T);
}

// Lane l of a group of L holds NV experts: VEC = 4: 4 (l + L j) + i, VEC = 1: l + L j.
template <int L, int NV, int VEC>
__device__ __forceinline__ int expert_of(int l, int v) {
  return VEC == 4 ? 4 * (l + L * (v >> 2)) + (v & 3) : l + L * v;
}
template <int L, int NV, int VEC, bool F16>
__device__ __forceinline__ void load_row(const BalanceArgs& a, int t, int l, float (&x)[NV]) {
  const size_t at = (size_t)t * (size_t)a.ld;
  if (VEC == 4) {
#pragma unroll
    for (int j = 0; j < NV / 4; ++j) {
      const int e = 4 * (l + L * j);
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < a.E) {
        if (F16) {
          const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __half*>(a.logits) + at + e);
          const float2 p = __half22float2(u32_as_h2(u.x)), q = __half22float2(u32_as_h2(u.y));
          f = make_float4(p.x, p.y, q.x, q.y);
        } else {
          f = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at + e);
        }
      }
      x[4 * j] = f.x; x[4 * j + 1] = f.y; x[4 * j + 2] = f.z; x[4 * j + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = l + L * v;
      x[v] = -INFINITY;
      if (e < a.E)
        x[v] = F16 ? __half2float(static_cast<const __half*>(a.logits)[at + e])
                   : static_cast<const float*>(a.logits)[at + e];
    }
  }
}

// x: logits in, probabilities out (0 for every expert of a bad token); rest:
// 1 - sigmoid(l). False for a bad token: NaN or +inf, or nothing above -inf.
template <int L, int NV, bool REST>
__device__ __forceinline__ bool probabilities(float (&x)[NV], float (&rest)[NV], bool sigmoid, unsigned mask) {
  float m = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    bad |= !(x[v] < INFINITY);
    m = fmaxf(m, x[v]);
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
  bad = __ballot_sync(mask, bad) & mask ? true : m == -INFINITY;
  float s = 0.0f;
  if (!sigmoid) {
#pragma unroll
    for (int v = 0; v < NV; ++v) s += x[v] = expf(x[v] - m);
  } else {
    // With u = e^-|l|, sigmoid(l) = (l < 0 ? u : 1) / (1 + u). Where every logit
    // is negative, numerators e^(l - max l) keep the sum away from 0.
    const bool low = m < 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const float l = x[v], u = expf(-fabsf(l)), r = 1.0f / (1.0f + u);
      if (REST) rest[v] = l < 0.0f ? r : u * r;
      s += x[v] = (l < 0.0f ? (low ? expf(l - m) : u) : 1.0f) * r;
    }
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) s += __shfl_xor_sync(mask, s, o);
  const float inv = 1.0f / s;
#pragma unroll
  for (int v = 0; v < NV; ++v) x[v] = bad ? 0.0f : x[v] * inv;
  return !bad;
}

// The first sequence with tokens from t0 on that can hold t0: offsets at or
// below t0, less one. Whole block.
__device__ __forceinline__ int first_sequence(const BalanceArgs& a, int t0) {
  int n = 0;
  for (int i = 0; i <= a.S; i += blockDim.x) {
    const int j = i + (int)threadIdx.x;
    n += __syncthreads_count(j <= a.S && offset_at(a, j) <= t0);
  }
  return max(n - 1, 0);
}

template <int L, int NV, int VEC, bool F16>
__global__ void __launch_bounds__(256) balance_partial_kernel(const BalanceArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int G = 32 / L, kGroups = 8 * G;  // groups per warp, per block
  __shared__ float sums[kGroups][L * NV];
  __shared__ int32_t cnt[1024];
  __shared__ int32_t good[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & (L - 1), grp = warp * G + lane / L;
  const unsigned mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~(L - 1));
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  for (int s = first_sequence(a, t0); s < a.S; ++s) {
    const int b0 = offset_at(a, s), lo = max(b0, t0), hi = min(offset_at(a, s + 1), t1);
    if (b0 >= t1) break;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < a.E; e += 256) cnt[e] = 0;
    __syncthreads();
    for (long long i = (long long)lo * a.k + threadIdx.x; i < (long long)hi * a.k; i += 256) {
      const int e = a.ids[i];
      if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
    }
    float p[NV] = {};
    int n = 0;
    for (int t = lo + grp; t < hi; t += kGroups) {
      float x[NV], rest[NV];
      load_row<L, NV, VEC, F16>(a, t, l, x);
      n += probabilities<L, NV, false>(x, rest, a.sigmoid, mask);
#pragma unroll
      for (int v = 0; v < NV; ++v) p[v] += x[v];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) sums[grp][expert_of<L, NV, VEC>(l, v)] = p[v];
    n = __reduce_add_sync(0xffffffffu, l == 0 ? n : 0);
    if (lane == 0) good[warp] = n;
    __syncthreads();
    const size_t row = (size_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < a.E; e += 256) {
      float v = 0.0f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) v += sums[g][e];
      a.psum[row * a.E + e] = v;
      a.csum[row * a.E + e] = cnt[e];
    }
    if (threadIdx.x == 0) {
      int v = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += good[w];
      a.nsum[row] = v;
    }
    __syncthreads();
  }
}

// Block (x, s): experts 32 x .. + 31 of sequence s; 8 warps share the partial rows.
__global__ void __launch_bounds__(256) balance_join_kernel(const BalanceArgs a) {
  griddep_wait();
  const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
  const int lo = offset_at(a, s), hi = offset_at(a, s + 1);
  const int c0 = hi > lo ? lo / a.chunk : 0, c1 = hi > lo ? (hi - 1) / a.chunk + 1 : 0;
  float p = 0.0f;
  int c = 0, n = 0;
  for (int r = c0 + warp; r < c1; r += 8) {
    const size_t row = (size_t)r + s;
    n += a.nsum[row];
    if (e < a.E) {
      p += a.psum[row * a.E + e];
      c += a.csum[row * a.E + e];
    }
  }
  __shared__ float ps[8][32];
  __shared__ int32_t cs[8][32], ns[8];
  ps[warp][lane] = p;
  cs[warp][lane] = c;
  if (lane == 0) ns[warp] = n;
  __syncthreads();
  __shared__ bool last;
  if (warp == 0) {
    p = 0.0f;
    c = n = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      p += ps[w][lane];
      c += cs[w][lane];
      n += ns[w];
    }
    const float mean = n ? p / (float)n : 0.0f;
    if (e < a.E) {
      a.counts[(size_t)s * a.E + e] = c;
      if (a.mean) a.mean[(size_t)s * a.E + e] = mean;
    }
    if (blockIdx.x == 0 && lane == 0) a.tokens[s] = n;
    if (!a.loss) return;
    const float f = e < a.E && n ? (float)c * ((float)a.E / ((float)a.k * (float)n)) * mean : 0.0f;
    const float part = warp_sum(f);
    if (lane == 0) {
      a.lsum[(size_t)s * gridDim.x + blockIdx.x] = part;
      __threadfence();
      const uint32_t total = gridDim.x * gridDim.y;
      last = atomicInc(a.ticket, total - 1) == total - 1;  // back to 0 with the last
    }
  }
  if (!a.loss) return;
  __syncthreads();
  if (!last) return;
  __threadfence();
  double v = 0.0;
  int live = 0;
  for (int i = threadIdx.x; i < (int)(gridDim.x * a.S); i += 256) v += (double)__ldcg(a.lsum + i);
  for (int i = threadIdx.x; i < a.S; i += 256) live += __ldcg(a.tokens + i) > 0;
  __shared__ double vs[256];
  vs[threadIdx.x] = v;
  live = __syncthreads_count(0) + live;
  __shared__ int lives;
  if (threadIdx.x == 0) lives = 0;
  __syncthreads();
  if (live) atomicAdd(&lives, live);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 256; ++i) v += vs[i];
    a.loss[0] = lives ? (float)(v * (double)a.coef / (double)lives) : 0.0f;
  }
}

template <int L, int NV, int VEC, bool F16>
__global__ void __launch_bounds__(256) balance_back_kernel(const BalanceArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int G = 32 / L, kGroups = 8 * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & (L - 1), grp = warp * G + lane / L;
  const unsigned mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~(L - 1));
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  int live = 0;
  for (int i = 0; i < a.S; i += 256) {
    const int j = i + (int)threadIdx.x;
    live += __syncthreads_count(j < a.S && a.btokens[j] > 0);
  }
  const float g = a.coef * (a.grad ? *a.grad : 1.0f);
  for (int s = first_sequence(a, t0); s < a.S; ++s) {
    const int b0 = offset_at(a, s), lo = max(b0, t0), hi = min(offset_at(a, s + 1), t1);
    if (b0 >= t1) break;
    if (lo >= hi) continue;
    const float n = (float)a.btokens[s];
    const float unit = n > 0.0f ? (float)a.E / ((float)a.k * n) : 0.0f;
    const float outer = n > 0.0f ? g / ((float)live * n) : 0.0f;
    float f[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = expert_of<L, NV, VEC>(l, v);
      f[v] = e < a.E ? (float)a.bcounts[(size_t)s * a.E + e] * unit : 0.0f;
    }
    for (int t = lo + grp; t < hi; t += kGroups) {
      float x[NV], rest[NV];
      load_row<L, NV, VEC, F16>(a, t, l, x);
      const bool ok = probabilities<L, NV, true>(x, rest, a.sigmoid, mask);
      float dot = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) dot = fmaf(x[v], f[v], dot);
#pragma unroll
      for (int o = 1; o < L; o <<= 1) dot += __shfl_xor_sync(mask, dot, o);
      float* out = a.dl + (size_t)t * (size_t)a.ldd;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = expert_of<L, NV, VEC>(l, v);
        float d = outer * x[v] * (f[v] - dot);
        if (a.sigmoid) d *= rest[v];
        if (!ok) d = 0.0f;
        if (e < a.E) out[e] = a.accumulate ? out[e] + d : d;
      }
    }
  }
}

struct Ws {
  size_t psum, csum, nsum, lsum, total;
};
Ws ws_of(int T, int E, int S) {
  const size_t rows = (size_t)std::min((T + kMinChunk - 1) / kMinChunk, kMaxChunks) + S;
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  Ws w;
  size_t o = kWorkspaceHeader;
  w.psum = o; o += up(rows * E * 4);
  w.csum = o; o += up(rows * E * 4);
  w.nsum = o; o += up(rows * 4);
  w.lsum = o; o += up((size_t)S * ((E + 31) / 32) * 4);
  w.total = o;
  return w;
}

template <bool BACK, int L, int NV, int VEC, bool F16>
cudaError_t launch_tokens(const cudaLaunchConfig_t& cfg, const BalanceArgs& a) {
  if (BACK) return cudaLaunchKernelEx(&cfg, balance_back_kernel<L, NV, VEC, F16>, a);
  return cudaLaunchKernelEx(&cfg, balance_partial_kernel<L, NV, VEC, F16>, a);
}
template <bool BACK, int VEC, bool F16>
cudaError_t launch_tokens(const cudaLaunchConfig_t& cfg, const BalanceArgs& a) {
  if (a.E <= 64) return launch_tokens<BACK, 8, 8, VEC, F16>(cfg, a);
  if (a.E <= 128) return launch_tokens<BACK, 16, 8, VEC, F16>(cfg, a);
  if (a.E <= 256) return launch_tokens<BACK, 32, 8, VEC, F16>(cfg, a);
  if (a.E <= 512) return launch_tokens<BACK, 32, 16, VEC, F16>(cfg, a);
  return launch_tokens<BACK, 32, 32, VEC, F16>(cfg, a);
}
// Four experts per load where every row allows it.
template <bool BACK>
cudaError_t launch_tokens(const cudaLaunchConfig_t& cfg, const BalanceArgs& a, int logit_type) {
  const int esz = logit_type == MOE_F16 ? 2 : 4;
  const bool vec = reinterpret_cast<uintptr_t>(a.logits) % (4 * esz) == 0 && a.ld % 4 == 0 && a.E % 4 == 0;
  if (logit_type == MOE_F16)
    return vec ? launch_tokens<BACK, 4, true>(cfg, a) : launch_tokens<BACK, 1, true>(cfg, a);
  return vec ? launch_tokens<BACK, 4, false>(cfg, a) : launch_tokens<BACK, 1, false>(cfg, a);
}

int check_balance(const char* who, const moe_balance_cfg* c, const void* logits, int logit_type, long long ld, int T,
                  int E, int k, const int32_t* offsets, int S) {
  if (!c) return fail(MOE_ERR_ARG, "%s: NULL settings", who);
  if (T < 0 || T > (1 << 27) || E < 1 || E > 1024 || k < 1 || k > 32 || k > E || (long long)T * k > 0x7fffffffLL)
    return fail(MOE_ERR_ARG, "%s: need 0 <= T <= 2^27, 1 <= k <= E <= 1024, k <= 32, T k < 2^31 (T=%d E=%d k=%d)", who,
                T, E, k);
  if (S < 1 || S > 65535 || (!offsets && S != 1))
    return fail(MOE_ERR_ARG, "%s: need 1 <= S <= 65535, one sequence without offsets (S=%d)", who, S);
  if (logit_type != MOE_F32 && logit_type != MOE_F16)
    return fail(MOE_ERR_ARG, "%s: unknown logit type %d", who, logit_type);
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_ARG, "%s: unknown score %d", who, c->score);
  if (!(c->coef > -INFINITY && c->coef < INFINITY)) return fail(MOE_ERR_ARG, "%s: coef must be finite", who);
  if (ld < E) return fail(MOE_ERR_ARG, "%s: row stride %lld below E=%d", who, ld, E);
  if (T > 0 && !logits) return fail(MOE_ERR_ARG, "%s: NULL pointer", who);
  if (reinterpret_cast<uintptr_t>(logits) % (logit_type == MOE_F16 ? 2 : 4) || reinterpret_cast<uintptr_t>(offsets) % 4)
    return fail(MOE_ERR_ARG, "%s: misaligned logits or offsets", who);
  return MOE_OK;
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(dim3 grid, cudaStream_t st) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_balance_workspace_bytes(int T, int E, int S) {
  if (T < 0 || E < 1 || E > 1024 || S < 1 || S > 65535) return 0;
  return moe::ws_of(T, E, S).total;
}

int moe_balance_loss(const moe_balance_cfg* cfg, const void* logits, int logit_type, long long ld, int T, int E,
                     const int32_t* ids, int k, const int32_t* offsets, int S, int32_t* counts, int32_t* tokens,
                     float* mean, float* loss, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "moe_balance_loss";
  moe::NvtxRange nvtx_range(who);
  moe::clear_error();
  const int rc = moe::check_balance(who, cfg, logits, logit_type, ld, T, E, k, offsets, S);
  if (rc != MOE_OK) return rc;
  if ((T > 0 && !ids) || !counts || !tokens || !workspace) return moe::fail(MOE_ERR_ARG, "%s: NULL pointer", who);
  if ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(tokens) |
       reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(loss)) % 4 ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return moe::fail(MOE_ERR_ARG, "%s: buffers must be 4-byte aligned, the workspace 256-byte", who);
  const moe::Ws w = moe::ws_of(T, E, S);
  if (workspace_bytes < w.total)
    return moe::fail(MOE_ERR_CAPACITY, "%s: workspace %zu < %zu bytes", who, workspace_bytes, w.total);
  uint8_t* w8 = static_cast<uint8_t*>(workspace);
  moe::BalanceArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.T = T; a.E = E; a.k = k; a.S = S;
  a.chunk = std::max(moe::kMinChunk, (T + moe::kMaxChunks - 1) / moe::kMaxChunks);
  a.chunks = (T + a.chunk - 1) / a.chunk;
  a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  a.coef = cfg->coef;
  a.ids = ids;
  a.offsets = offsets;
  a.psum = reinterpret_cast<float*>(w8 + w.psum);
  a.csum = reinterpret_cast<int32_t*>(w8 + w.csum);
  a.nsum = reinterpret_cast<int32_t*>(w8 + w.nsum);
  a.lsum = reinterpret_cast<float*>(w8 + w.lsum);
  a.ticket = reinterpret_cast<uint32_t*>(w8) + 1;
  a.counts = counts;
  a.tokens = tokens;
  a.mean = mean;
  a.loss = loss;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (T > 0) {
    const moe::Launch l(dim3((unsigned)a.chunks), st);
    e = moe::launch_tokens<false>(l.cfg, a, logit_type);
  }
  if (e == cudaSuccess) {
    const moe::Launch l(dim3((unsigned)((E + 31) / 32), (unsigned)S), st);
    e = cudaLaunchKernelEx(&l.cfg, moe::balance_join_kernel, a);
  }
  if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return MOE_OK;
}

int moe_balance_loss_backward(const moe_balance_cfg* cfg, const void* logits, int logit_type, long long ld, int T,
                              int E, int k, const int32_t* offsets, int S, const int32_t* counts,
                              const int32_t* tokens, const float* grad_loss, float* dlogits, long long ldd,
                              int accumulate, void* stream) {
  const char* who = "moe_balance_loss_backward";
  moe::NvtxRange nvtx_range(who);
  moe::clear_error();
  const int rc = moe::check_balance(who, cfg, logits, logit_type, ld, T, E, k, offsets, S);
  if (rc != MOE_OK) return rc;
  if (ldd < E) return moe::fail(MOE_ERR_ARG, "%s: row stride %lld below E=%d", who, ldd, E);
  if (T == 0) return MOE_OK;
  if (!counts || !tokens || !dlogits) return moe::fail(MOE_ERR_ARG, "%s: NULL pointer", who);
  if ((reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(tokens) |
       reinterpret_cast<uintptr_t>(grad_loss) | reinterpret_cast<uintptr_t>(dlogits)) % 4)
    return moe::fail(MOE_ERR_ARG, "%s: buffers must be 4-byte aligned", who);
  moe::BalanceArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.T = T; a.E = E; a.k = k; a.S = S;
  a.chunk = moe::kMinChunk;
  a.chunks = (T + a.chunk - 1) / a.chunk;
  a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  a.coef = cfg->coef;
  a.offsets = offsets;
  a.bcounts = counts;
  a.btokens = tokens;
  a.grad = grad_loss;
  a.dl = dlogits;
  a.ldd = ldd;
  a.accumulate = accumulate != 0;
  const moe::Launch l(dim3((unsigned)a.chunks), static_cast<cudaStream_t>(stream));
  const cudaError_t e = moe::launch_tokens<true>(l.cfg, a, logit_type);
  if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return MOE_OK;
}

}  // extern "C"
