// Scored router: softmax or sigmoid scores, a balance bias that only orders
// the experts, expert groups, top-k, renormalised and scaled weights.
// "Horizon RunMap -- Prévia Técnica", "02 / A solução": the router picks the
// experts of each token; it stays outside the INT4 compression.
//
//   s_e = sigmoid(l_e) or softmax(l)_e;  v_e = s_e + b_e  (v_e = l_e without a
//   bias: both scores grow with the logit, so the order needs no exponential);
//   groups of E/G experts ranked by max v or by the sum of their two largest
//   scores, the best top_groups kept; top-k of the kept experts by
//   (v desc, index asc); w_j = s_{id_j} [/ (sum_j s_{id_j} + 1e-20)] * scale.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "common.h"
#include "device.cuh"
#include "kernels.h"

namespace moe {
namespace {

struct ScoredArgs {
  const void* logits;
  long long ld;
  int T, E, k;
  int G, per;       // groups, experts per group
  int lg_shift;     // log2 of the lanes that hold one group
  int chunk;        // experts per lane
  int vec;          // rows can be read 16 bytes at a time
  int top_g, rank_top2, sigmoid, renorm;
  float scale;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t* bad;
};

// The value of an order_key (of a finite value).
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <bool HALF>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  if (HALF) return __half2float(static_cast<const __half*>(row)[e]);
  return static_cast<const float*>(row)[e];
}

// The special-function unit's own 2^x and 1/x (relative errors about 2^-22);
// with the rounding of v log2(e) a score is off by less than 1e-6 of itself
// for |v| <= 10.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_f(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * kLog2e));
  return r;
}
__device__ __forceinline__ float sigmoid_f(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp_f(-v)));
  return r;
}
// The larger of the two, NaN if one is.
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// N consecutive values at p, 16 bytes at a time (p 16-byte aligned).
template <int N, bool HALF>
__device__ __forceinline__ void load_vec(const void* p, float (&v)[N]) {
  if (HALF) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      const uint4 w = static_cast<const uint4*>(p)[i / 8];
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < N) v[i + j] = __half2float(__ushort_as_half((unsigned short)(u[j / 2] >> (16 * (j & 1)))));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 w = static_cast<const float4*>(p)[i / 4];
      const float u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < N) v[i + j] = u[j];
    }
  }
}

constexpr int kWarpsPerBlock = 4;

// One warp per token (looping over tokens when there are many). The lanes are
// split evenly over the groups (rounded up to a power of two), and a lane
// holds `chunk` consecutive experts of its group, so a group's two best are a
// butterfly over its own lanes.
//
// Top-k: the k-th largest of the lanes' maxima (k rounds of one warp
// reduction) is a bound that at least k candidates reach; the candidates that
// reach it are usually few more than k. They are compacted to shared memory as
// 64-bit keys (value, then lower index first), and each lane ranks one of them
// against the others. Where more than 32 reach the bound, k rounds of argmax
// instead. Bound by instruction issue: about 400 per token of 256 experts.
template <int PER, bool HALF>
__global__ void __launch_bounds__(32 * kWarpsPerBlock) route_scored_kernel(const ScoredArgs a) {
  constexpr bool kBiasRegs = PER <= 16;  // a lane's biases stay in registers over its tokens
  __shared__ unsigned long long cand_all[kWarpsPerBlock][32];
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long* cand = cand_all[warp];
  const int lanes = 1 << a.lg_shift;  // of a group
  const int grp = lane >> a.lg_shift, sub = lane & (lanes - 1);
  const int first = grp * a.per + sub * a.chunk;
  const int n = grp < a.G ? max(0, min(a.chunk, a.per - sub * a.chunk)) : 0;
  griddep_wait();
  griddep_launch_dependents();
  float bias[kBiasRegs ? PER : 1];
  bool bad_bias = false;
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float b = j < n ? a.bias[first + j] : 0.0f;
      bad_bias |= !(b < INFINITY);  // NaN or +inf
      if (kBiasRegs) bias[j] = b;
    }
  }
  for (int t = blockIdx.x * kWarpsPerBlock + warp; t < a.T; t += gridDim.x * kWarpsPerBlock) {
    const uint8_t* row = static_cast<const uint8_t*>(a.logits) + (size_t)t * a.ld * (HALF ? 2 : 4);
    float v[PER];  // logits, then what orders the experts (-inf: not to be chosen)
    if (a.vec && n == PER) {
      load_vec<PER, HALF>(row + (size_t)first * (HALF ? 2 : 4), v);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) v[j] = j < n ? load_logit<HALF>(row, first + j) : -INFINITY;
    }
    float mx = v[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) mx = fmax_nan(mx, v[j]);
    const bool bad = bad_bias || !(mx < INFINITY);  // NaN or +inf
    float m = 0.0f, inv = 1.0f;
    if (!a.sigmoid) {
      m = warp_max(mx);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < PER; ++j) s += v[j] > -INFINITY ? exp_f(v[j] - m) : 0.0f;
      inv = 1.0f / warp_sum(s);
    }
    auto sigmoid = [](float l) { return sigmoid_f(l); };
    auto softmax = [&](float l) { return exp_f(l - m) * inv; };
    float g1 = mx, g2 = -INFINITY;  // the lane's two best for the group's value
    float top = mx;                 // the lane's best in the order
    auto add_bias = [&](auto score) {
      g1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const float b = kBiasRegs ? bias[kBiasRegs ? j : 0] : (j < n ? a.bias[first + j] : 0.0f);
        v[j] = v[j] > -INFINITY ? score(v[j]) + b : -INFINITY;
        g2 = fmaxf(g2, fminf(g1, v[j]));
        g1 = fmaxf(g1, v[j]);
      }
      top = g1;
    };
    auto best_two = [&](auto score) {
      g1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const float r = v[j] > -INFINITY ? score(v[j]) : -INFINITY;
        g2 = fmaxf(g2, fminf(g1, r));
        g1 = fmaxf(g1, r);
      }
    };
    if (a.bias) {
      if (a.sigmoid) add_bias(sigmoid);
      else add_bias(softmax);
    } else if (a.rank_top2) {
      if (a.sigmoid) best_two(sigmoid);
      else best_two(softmax);
    }
    if (__any_sync(full, bad) || !__any_sync(full, top > -INFINITY)) {
      if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = -1;
        a.weights[(size_t)t * a.k + lane] = 0.0f;
      }
      if (lane == 0 && a.bad) atomicAdd(a.bad, 1);
      continue;
    }
    bool kept = grp < a.G;
    if (a.top_g < a.G) {
      for (int o = 1; o < lanes; o <<= 1) {
        const float h1 = __shfl_xor_sync(full, g1, o), h2 = __shfl_xor_sync(full, g2, o);
        g2 = fmaxf(fminf(g1, h1), fmaxf(g2, h2));
        g1 = fmaxf(g1, h1);
      }
      const float gv = a.rank_top2 && g2 > -INFINITY ? g1 + g2 : g1;
      // How many groups come before this one: its lanes share the comparisons.
      int before = 0;
      for (int h0 = 0; h0 < a.G; h0 += lanes) {
        const int h = h0 + sub;
        const float o = __shfl_sync(full, gv, (h << a.lg_shift) & 31);
        before += h < a.G && (o > gv || (o == gv && h < grp));
      }
      for (int o = 1; o < lanes; o <<= 1) before += __shfl_xor_sync(full, before, o);
      kept = kept && before < a.top_g;
    }

    uint32_t key = kept && top > -INFINITY ? order_key(top) : 0u, bound = 0u;  // a real key is above 0
#pragma unroll 4
    for (int r = 0; r < a.k; ++r) {
      bound = __reduce_max_sync(full, key);
      if (key == bound) key = 0u;
    }
    // Candidates: what reaches the bound, or (fewer than k lanes hold one) all.
    const float lim = !kept ? INFINITY : bound != 0u ? key_value(bound) : -FLT_MAX;
    int mine = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) mine += v[j] >= lim;
    int upto = mine;  // inclusive scan over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(full, upto, o);
      if (lane >= o) upto += x;
    }
    const int count = __shfl_sync(full, upto, 31);
    int my_i = -1, my_r = 32;  // this lane's pick and its rank
    if (count <= 32) {
      if (mine) {
        int pos = upto - mine;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (v[j] >= lim)
            cand[pos++] = ((unsigned long long)__float_as_uint(v[j]) << 32) | (uint32_t)(first + j);
      }
      __syncwarp();
      unsigned long long me = 0;
      if (lane < count) {
        me = cand[lane];
        my_i = (int)(uint32_t)me;
        me = ((unsigned long long)order_key(__uint_as_float((uint32_t)(me >> 32))) << 32) | (0xffffffffu - (uint32_t)me);
        cand[lane] = me;
        my_r = 0;
      }
      __syncwarp();
#pragma unroll 4
      for (int c = 0; c < count; ++c) my_r += cand[c] > me;
      if (lane >= count) my_r = lane < a.k ? lane : 32;  // no expert left for this pick
      __syncwarp();
    } else {
      float bv = -INFINITY;
      int bi = INT_MAX;
      auto best_after = [&](float lv, int li) {  // the lane's best that ranks after (lv, li)
        bv = -INFINITY;
        bi = INT_MAX;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (v[j] > -INFINITY && ranks_before(lv, li, v[j], first + j) && ranks_before(v[j], first + j, bv, bi)) {
            bv = v[j];
            bi = first + j;
          }
      };
      if (kept) best_after(INFINITY, -1);
      for (int r = 0; r < a.k; ++r) {  // more than 32 candidates, k <= 32: every round finds one
        const uint32_t bk = bi != INT_MAX ? order_key(bv) : 0u;
        const uint32_t kmax = __reduce_max_sync(full, bk);
        const int win = (int)__reduce_min_sync(full, bk == kmax ? (uint32_t)bi : 0xffffffffu);
        if (lane == r) my_i = win;
        if (bi == win) best_after(bv, win);
      }
      my_r = lane;
    }
    const bool picked = my_r < a.k && my_i >= 0;
    float s = 0.0f;
    if (picked) {
      const float l = load_logit<HALF>(row, my_i);
      s = a.sigmoid ? sigmoid(l) : softmax(l);
    }
    if (a.renorm) s = s / (warp_sum(s) + 1e-20f);
    if (my_r < a.k) {
      a.ids[(size_t)t * a.k + my_r] = my_i;
      a.weights[(size_t)t * a.k + my_r] = s * a.scale;
    }
  }
}

template <int PER, bool HALF>
cudaError_t launch_scored(const ScoredArgs& a, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min((a.T + kWarpsPerBlock - 1) / kWarpsPerBlock, sms * 18));
  cfg.blockDim = dim3(32 * kWarpsPerBlock);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_scored_kernel<PER, HALF>, a);
}

template <bool HALF>
cudaError_t launch_scored(const ScoredArgs& a, int sms, cudaStream_t st) {
  if (a.chunk <= 2) return launch_scored<2, HALF>(a, sms, st);
  if (a.chunk <= 4) return launch_scored<4, HALF>(a, sms, st);
  if (a.chunk <= 8) return launch_scored<8, HALF>(a, sms, st);
  if (a.chunk <= 16) return launch_scored<16, HALF>(a, sms, st);
  if (a.chunk <= 32) return launch_scored<32, HALF>(a, sms, st);
  return launch_scored<64, HALF>(a, sms, st);
}

}  // namespace

int check_route_cfg(const char* who, const moe_route_cfg* c, const void* logits, int logit_type, long long ld,
                    int T, int E, int k) {
  if (!c) return fail(MOE_ERR_ARG, "%s: NULL cfg", who);
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E)
    return fail(MOE_ERR_ARG, "%s: need T >= 0, 1 <= k <= min(E, 32), E <= 1024 (T=%d E=%d k=%d)", who, T, E, k);
  if (logit_type != MOE_F32 && logit_type != MOE_F16)
    return fail(MOE_ERR_ARG, "%s: unknown logit type %d", who, logit_type);
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_ARG, "%s: unknown score %d", who, c->score);
  if (c->group_rank != MOE_GROUP_MAX && c->group_rank != MOE_GROUP_TOP2)
    return fail(MOE_ERR_ARG, "%s: unknown group rank %d", who, c->group_rank);
  if (c->n_groups < 1 || c->n_groups > 32 || E % c->n_groups || c->top_groups < 1 || c->top_groups > c->n_groups)
    return fail(MOE_ERR_ARG, "%s: need 1 <= top_groups <= n_groups <= 32, n_groups dividing E (E=%d, %d of %d)", who, E,
                c->top_groups, c->n_groups);
  if (k > c->top_groups * (E / c->n_groups))
    return fail(MOE_ERR_ARG, "%s: k=%d exceeds the %d experts of %d groups", who, k,
                c->top_groups * (E / c->n_groups), c->top_groups);
  if (!(c->scale > -INFINITY && c->scale < INFINITY)) return fail(MOE_ERR_ARG, "%s: scale must be finite", who);
  if (ld < E) return fail(MOE_ERR_ARG, "%s: row stride %lld below E=%d", who, ld, E);
  if (T > 0 && reinterpret_cast<uintptr_t>(logits) % (logit_type == MOE_F16 ? 2 : 4))
    return fail(MOE_ERR_ARG, "%s: misaligned logits", who);
  return MOE_OK;
}

}  // namespace moe

extern "C" int moe_route_scored(const moe_route_cfg* cfg, const void* logits, int logit_type, long long ld, int T,
                                int E, int k, const float* bias, int32_t* ids, float* weights, int32_t* bad_tokens,
                                void* stream) {
  moe::NvtxRange nvtx_range("moe_route_scored");
  moe::clear_error();
  int rc = moe::check_route_cfg("moe_route_scored", cfg, logits, logit_type, ld, T, E, k);
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !weights) return moe::fail(MOE_ERR_ARG, "moe_route_scored: NULL pointer");
  moe::ScoredArgs a;
  a.logits = logits;
  a.ld = ld;
  a.T = T; a.E = E; a.k = k;
  a.G = cfg->n_groups;
  a.per = E / cfg->n_groups;
  int shift = 5;  // lanes per group: 32 over the groups rounded up to a power of two
  while ((32 >> shift) < a.G) --shift;
  a.lg_shift = shift;
  a.chunk = (a.per + (1 << shift) - 1) >> shift;
  // 16-byte loads where every lane's run of experts starts on 16 bytes.
  const int esz = logit_type == MOE_F16 ? 2 : 4;
  a.vec = reinterpret_cast<uintptr_t>(logits) % 16 == 0 && ld * esz % 16 == 0 && a.chunk * esz % 16 == 0 &&
          a.per * esz % 16 == 0;
  a.top_g = cfg->top_groups;
  a.rank_top2 = cfg->group_rank == MOE_GROUP_TOP2 && a.per > 1;
  a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  a.renorm = cfg->renorm != 0;
  a.scale = cfg->scale;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.bad = bad_tokens;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  if ((rc = moe::current_device_sms(&dev, &sms)) != MOE_OK) return rc;
  const cudaError_t e = logit_type == MOE_F16 ? moe::launch_scored<true>(a, sms, st)
                                             : moe::launch_scored<false>(a, sms, st);
  if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "moe_route_scored launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}
