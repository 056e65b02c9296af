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
  int top_g, rank_top2, sigmoid, renorm;
  float scale;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t* bad;
};

template <bool HALF>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  if (HALF) return __half2float(static_cast<const __half*>(row)[e]);
  return static_cast<const float*>(row)[e];
}

__device__ __forceinline__ float sigmoid_f(float v) { return 1.0f / (1.0f + expf(-v)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// One warp per token. The lanes are split evenly over the groups (rounded up
// to a power of two), and a lane holds `chunk` consecutive experts of its
// group, so a group's two best are a butterfly over its own lanes.
template <int PER, bool HALF>
__global__ void __launch_bounds__(128) route_scored_kernel(const ScoredArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (t >= a.T) return;
  const size_t esz = HALF ? 2 : 4;
  const uint8_t* row = static_cast<const uint8_t*>(a.logits) + (size_t)t * a.ld * esz;
  const int grp = lane >> a.lg_shift, sub = lane & ((1 << a.lg_shift) - 1);
  const int first = grp * a.per + sub * a.chunk;
  const int n = grp < a.G ? max(0, min(a.chunk, a.per - sub * a.chunk)) : 0;

  float v[PER];  // logits, then what orders the experts (-inf: not to be chosen)
  bool bad = false;
  float mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    v[j] = j < n ? load_logit<HALF>(row, first + j) : -INFINITY;
    bad |= isnan(v[j]) || v[j] == INFINITY;
    mx = fmaxf(mx, v[j]);
  }
  float m = 0.0f, sum = 1.0f;
  if (!a.sigmoid) {
    m = warp_max(mx);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) s += v[j] > -INFINITY ? expf(v[j] - m) : 0.0f;
    sum = warp_sum(s);
  }
  auto score = [&](float l) { return a.sigmoid ? sigmoid_f(l) : expf(l - m) / sum; };
  float g1 = -INFINITY, g2 = -INFINITY;  // the lane's two best for the group's value
  bool live = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (j < n) {
      float o = v[j], r = o;
      if (a.bias) {
        const float b = a.bias[first + j];
        bad |= isnan(b) || b == INFINITY;
        o = o > -INFINITY && b > -INFINITY ? score(o) + b : -INFINITY;
        r = o;
      } else if (a.rank_top2) {
        r = o > -INFINITY ? score(o) : -INFINITY;
      }
      v[j] = o;
      live |= o > -INFINITY;
      g2 = fmaxf(g2, fminf(g1, r));
      g1 = fmaxf(g1, r);
    }
  }
  if (__any_sync(full, bad) || !__any_sync(full, live)) {
    if (lane < a.k) {
      a.ids[(size_t)t * a.k + lane] = -1;
      a.weights[(size_t)t * a.k + lane] = 0.0f;
    }
    if (lane == 0 && a.bad) atomicAdd(a.bad, 1);
    return;
  }
  bool kept = grp < a.G;
  if (a.top_g < a.G) {
    for (int o = 1; o < (1 << a.lg_shift); o <<= 1) {
      const float h1 = __shfl_xor_sync(full, g1, o), h2 = __shfl_xor_sync(full, g2, o);
      g2 = fmaxf(fminf(g1, h1), fmaxf(g2, h2));
      g1 = fmaxf(g1, h1);
    }
    const float gv = a.rank_top2 && g2 > -INFINITY ? g1 + g2 : g1;
    int before = 0;
    for (int h = 0; h < a.G; ++h) before += ranks_before(__shfl_sync(full, gv, h << a.lg_shift), h, gv, grp);
    kept = kept && before < a.top_g;
  }

  // Top-k: each lane offers its best expert not yet picked; a round takes the
  // largest order key of the warp and the lowest index that has it.
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
  int my_i = -1;
  for (int r = 0; r < a.k; ++r) {
    const uint32_t key = bi != INT_MAX ? order_key(bv) : 0u;
    const uint32_t kmax = __reduce_max_sync(full, key);
    if (kmax == 0u) break;  // no expert left: the other picks stay -1
    const int win = (int)__reduce_min_sync(full, key == kmax ? (uint32_t)bi : 0xffffffffu);
    if (lane == r) my_i = win;
    if (bi == win) best_after(bv, win);
  }
  const float s = my_i >= 0 ? score(load_logit<HALF>(row, my_i)) : 0.0f;
  const float total = warp_sum(s);
  if (lane < a.k) {
    a.ids[(size_t)t * a.k + lane] = my_i;
    a.weights[(size_t)t * a.k + lane] = (a.renorm ? s / (total + 1e-20f) : s) * a.scale;
  }
}

template <int PER, bool HALF>
cudaError_t launch_scored(const ScoredArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_scored_kernel<PER, HALF>, a);
}

template <bool HALF>
cudaError_t launch_scored(const ScoredArgs& a, cudaStream_t st) {
  if (a.chunk <= 2) return launch_scored<2, HALF>(a, st);
  if (a.chunk <= 4) return launch_scored<4, HALF>(a, st);
  if (a.chunk <= 8) return launch_scored<8, HALF>(a, st);
  if (a.chunk <= 16) return launch_scored<16, HALF>(a, st);
  if (a.chunk <= 32) return launch_scored<32, HALF>(a, st);
  return launch_scored<64, HALF>(a, st);
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
  const int rc = moe::check_route_cfg("moe_route_scored", cfg, logits, logit_type, ld, T, E, k);
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
  const cudaError_t e = logit_type == MOE_F16 ? moe::launch_scored<true>(a, st) : moe::launch_scored<false>(a, st);
  if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "moe_route_scored launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}
