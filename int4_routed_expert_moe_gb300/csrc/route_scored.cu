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

// What orders the experts takes the special-function unit's own 2^x (relative
// error 2^-22) of v log2(e), whose rounding adds 1.2 |v| 2^-24, and the sum and
// reciprocal 3 units: a score is off by at most (7 + 1.2 |v|) 2^-24 of itself,
// in all less than 3e-7. The weights
// of the picks take expf: its range reduction keeps them within a few units of
// 2^-24 at any logit (at |v| = 78 the other form is 61 units off). Measured, us
// for 32768 tokens of 256 experts with a softmax and a bias: this 22.6, expf
// for the order too 27.5, the two-FMA correction of the exponent 24.9.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_order(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * kLog2e));
  return r;
}
__device__ __forceinline__ float rcp_f(float v) {  // one ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The larger of the two, NaN if one is.
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Reductions over the L lanes of a token.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if (L == 32) return __reduce_max_sync(0xffffffffu, v);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  return ~lanes_max<L>(~v);
}
template <int L>
__device__ __forceinline__ bool lanes_any(bool p) {
  const unsigned b = __ballot_sync(0xffffffffu, p);
  return L == 32 ? b != 0 : ((b >> (threadIdx.x & 31 & ~(L - 1))) & ((1u << (L & 31)) - 1u)) != 0;
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
constexpr int kHalfWarpTokens = 4096, kHalfWarpChunk = 4;  // see route_scored_kernel

// L lanes per token, 32 / L tokens per warp (looping over tokens when there
// are many). The lanes are split evenly over the groups (rounded up to a power
// of two), and a lane holds `chunk` consecutive experts of its group, so a
// group's two best are a butterfly over its own lanes.
//
// Top-k: the k-th largest of the lanes' two best (k rounds of one reduction)
// is a bound that at least k candidates reach (or all, where there are fewer);
// the candidates that reach it are usually few more than k. Their indexes are
// compacted to shared memory with their values, and each lane ranks one of
// them by (v desc, index asc), a 64-bit key, against the others. Where more
// than L reach the bound, k rounds of argmax instead.
//
// Bound by instruction issue (some 660 per token of 256 experts: 22.9 us for
// 32768 tokens, whose logits alone would take 5 us). Half a warp per token pays
// the reductions, the scan and the ranking once for two tokens, but holds twice
// the experts per lane. Measured with sigmoid scores and a bias, us for 32768
// tokens, warp against half: 20 experts 13.4 / 8.6, 64 experts 17.7 / 11.5, 256
// experts 23.0 / 21.8 (16 experts per lane), 512 experts 37 / 74 (32); 64
// experts, 2048 tokens 3.1 / 3.3, 4096 tokens 5.1 / 3.6. So half a warp where
// that leaves a lane at most 4 experts and there are 4096 tokens.
template <int PER, bool HALF, int L>
__global__ void __launch_bounds__(32 * kWarpsPerBlock) route_scored_kernel(const ScoredArgs a) {
  constexpr bool kBiasRegs = PER <= 16;  // a lane's biases stay in registers over its tokens
  constexpr int kTok = 32 / L;           // tokens per warp
  __shared__ unsigned long long cand_all[kWarpsPerBlock * kTok][L];
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & (L - 1), slot = threadIdx.x / L;
  unsigned long long* cand = cand_all[slot];
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
  // Unsigned: the step after the last tokens may pass 2^31, not 2^32.
  const unsigned T = (unsigned)a.T, step = gridDim.x * kWarpsPerBlock * kTok;
  for (unsigned t0 = blockIdx.x * kWarpsPerBlock * kTok; t0 < T; t0 += step) {
    const unsigned t = t0 + slot;
    const bool in = t < T;  // the last tokens' warps may be half empty
    const uint8_t* row = static_cast<const uint8_t*>(a.logits) + (size_t)(in ? t : 0) * a.ld * (HALF ? 2 : 4);
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
      m = lanes_max<L>(mx);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < PER; ++j) s += v[j] > -INFINITY ? exp_order(v[j] - m) : 0.0f;
      inv = 1.0f / lanes_sum<L>(s);
    }
    auto sigmoid = [](float l) { return rcp_f(1.0f + exp_order(-l)); };
    // Rounded before the bias is added: one FMA would order by other values than the score.
    auto softmax = [&](float l) { return __fmul_rn(exp_order(l - m), inv); };
    // The lane's two best: in the order (p1, p2), and for the group's value.
    float p1 = -INFINITY, p2 = -INFINITY, g1, g2;
    auto two = [](float& x1, float& x2, float x) {
      x2 = fmaxf(x2, fminf(x1, x));
      x1 = fmaxf(x1, x);
    };
    auto add_bias = [&](auto score) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const float b = kBiasRegs ? bias[kBiasRegs ? j : 0] : (j < n ? a.bias[first + j] : 0.0f);
        v[j] = v[j] > -INFINITY ? __fadd_rn(score(v[j]), b) : -INFINITY;
        two(p1, p2, v[j]);
      }
    };
    if (a.bias) {
      if (a.sigmoid) add_bias(sigmoid);
      else add_bias(softmax);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) two(p1, p2, v[j]);
    }
    g1 = p1;
    g2 = p2;
    if (!a.bias && a.rank_top2) {  // the scores grow with the logits: the same two experts
      if (g1 > -INFINITY) g1 = a.sigmoid ? sigmoid(g1) : softmax(g1);
      if (g2 > -INFINITY) g2 = a.sigmoid ? sigmoid(g2) : softmax(g2);
    }
    // Both votes by all the lanes: the halves of a warp may see different tokens.
    const bool any_bad = lanes_any<L>(bad), any_live = lanes_any<L>(p1 > -INFINITY);
    const bool dead = any_bad || !any_live;
    bool kept = grp < a.G && !dead;
    if (a.top_g < a.G) {
      for (int o = 1; o < lanes; o <<= 1) {
        const float h1 = __shfl_xor_sync(full, g1, o), h2 = __shfl_xor_sync(full, g2, o);
        g2 = fmaxf(fminf(g1, h1), fmaxf(g2, h2));
        g1 = fmaxf(g1, h1);
      }
      // Two biases of FP32's lowest value do not add up to what a group without experts is worth.
      const float gv = a.rank_top2 && g2 > -INFINITY ? fmaxf(g1 + g2, -FLT_MAX) : g1;
      // How many groups come before this one: its lanes share the comparisons.
      int before = 0;
      for (int h0 = 0; h0 < a.G; h0 += lanes) {
        const int h = h0 + sub;
        const float o = __shfl_sync(full, gv, (h << a.lg_shift) & (L - 1), L);
        before += h < a.G && (o > gv || (o == gv && h < grp));
      }
      for (int o = 1; o < lanes; o <<= 1) before += __shfl_xor_sync(full, before, o);
      kept = kept && before < a.top_g;
    }

    // A real key is above 0.
    uint32_t key = kept && p1 > -INFINITY ? order_key(p1) : 0u, key2 = kept && p2 > -INFINITY ? order_key(p2) : 0u;
    uint32_t bound = 0u;
#pragma unroll 4
    for (int r = 0; r < a.k; ++r) {
      bound = lanes_max<L>(key);
      if (key == bound) {
        key = key2;
        key2 = 0u;
      }
    }
    // Candidates: what reaches the bound, or (fewer than k in the lanes' two best) all.
    // (No logit compares with a NaN, not even the +inf of a bad token.)
    const float lim = !kept ? __int_as_float(0x7fffffff) : bound != 0u ? key_value(bound) : -FLT_MAX;
    int mine = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) mine += v[j] >= lim;
    int upto = mine;  // inclusive scan over the token's lanes
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      const int x = __shfl_up_sync(full, upto, o, L);
      if (lane >= o) upto += x;
    }
    const int count = __shfl_sync(full, upto, L - 1, L);
    const bool few = count <= L;
    if (few && mine) {
      int pos = upto - mine;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (v[j] >= lim)
          cand[pos++] = ((unsigned long long)__float_as_uint(v[j]) << 32) | (unsigned)(first + j);
    }
    __syncwarp();
    int my_i = -1, my_r = L;  // this lane's pick and its rank
    unsigned long long me = 0;
    if (few && lane < count) {
      const unsigned long long c = cand[lane];
      my_i = (int)(uint32_t)c;
      me = ((unsigned long long)order_key(__uint_as_float((uint32_t)(c >> 32))) << 32) | (0xffffffffu - (uint32_t)c);
    }
    if (__any_sync(full, !few)) {
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
      for (int r = 0; r < a.k; ++r) {
        const uint32_t bk = bi != INT_MAX ? order_key(bv) : 0u;
        const uint32_t kmax = lanes_max<L>(bk);
        const uint32_t win = lanes_min<L>(bk == kmax && kmax != 0u ? (uint32_t)bi : 0xffffffffu);
        if (!few && lane == r) my_i = (int)win;  // more candidates than k: every round finds one
        if ((uint32_t)bi == win) best_after(bv, (int)win);
      }
      if (!few) my_r = lane;
    }
    float s = 0.0f;  // the pick's score, from its logit again
    if (my_i >= 0) {
      const float l = load_logit<HALF>(row, my_i);
      const float e = expf(a.sigmoid ? -l : l - m);
      s = a.sigmoid ? rcp_f(1.0f + e) : e * inv;
    }
    __syncwarp();
    if (few) cand[lane] = me;
    __syncwarp();
    if (few) {
      if (my_i >= 0) {
        my_r = 0;
#pragma unroll 4
        for (int c = 0; c < count; ++c) my_r += cand[c] > me;
      } else {
        my_r = lane;  // no expert left for this pick
      }
    }
    __syncwarp();
    const bool out = my_r < a.k;
    if (!out) s = 0.0f;
    if (a.renorm) s = s / (lanes_sum<L>(s) + 1e-20f);
    if (in && out) {
      a.ids[(size_t)t * a.k + my_r] = my_i;
      a.weights[(size_t)t * a.k + my_r] = s * a.scale;
    }
    if (in && dead && lane == 0 && a.bad) atomicAdd(a.bad, 1);
  }
}

template <int PER, bool HALF, int L>
cudaError_t launch_scored(const ScoredArgs& a, int sms, cudaStream_t st) {
  constexpr int kTokens = kWarpsPerBlock * (32 / L);  // per block and round
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(((unsigned)a.T + kTokens - 1) / kTokens, (unsigned)sms * 18));
  cfg.blockDim = dim3(32 * kWarpsPerBlock);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_scored_kernel<PER, HALF, L>, a);
}

template <bool HALF>
cudaError_t launch_scored(const ScoredArgs& a, int L, int sms, cudaStream_t st) {
  if (L == 16) return launch_scored<kHalfWarpChunk, HALF, 16>(a, sms, st);
  if (a.chunk <= 2) return launch_scored<2, HALF, 32>(a, sms, st);
  if (a.chunk <= 4) return launch_scored<4, HALF, 32>(a, sms, st);
  if (a.chunk <= 8) return launch_scored<8, HALF, 32>(a, sms, st);
  if (a.chunk <= 16) return launch_scored<16, HALF, 32>(a, sms, st);
  if (a.chunk <= 32) return launch_scored<32, HALF, 32>(a, sms, st);
  return launch_scored<64, HALF, 32>(a, sms, st);
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
  auto split = [&](int L) {  // lanes per group: L over the groups rounded up to a power of two
    a.lg_shift = L == 32 ? 5 : 4;
    while ((L >> a.lg_shift) < a.G) --a.lg_shift;
    a.chunk = (a.per + (1 << a.lg_shift) - 1) >> a.lg_shift;
  };
  int L = 32;
  if (T >= moe::kHalfWarpTokens && k <= 16 && a.G <= 16) {
    split(16);
    if (a.chunk <= moe::kHalfWarpChunk) L = 16;
  }
  if (L == 32) split(32);
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
  const cudaError_t e = logit_type == MOE_F16 ? moe::launch_scored<true>(a, L, sms, st)
                                             : moe::launch_scored<false>(a, L, sms, st);
  if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "moe_route_scored launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}
