// Balance loss of a router by sequence, per-expert counts, and the gradient.
//   f_se = E c_se / (k n_s),  P_se = mean of p_te over the n_s good tokens,
//   loss = coef / S' sum_s sum_e f_se P_se,
//   dl_te = g coef / (S' n_s) p_te (f_se - sum_j f_sj p_tj) [* (1 - sigmoid(l_te))]
//
// A token's logits stay in the registers of a group of lanes: 8, 16 or 32
// lanes with 8 values each for up to 256 experts, then 32 lanes with 16 or 32.
// Forward: chunks of consecutive tokens, one per block; each lane adds its
// experts' probabilities over the group's tokens, the block adds its groups in
// order. A sequence inside one chunk is finished there; of one that several
// chunks share, each writes a partial row, and the last of them to arrive (a
// ticket per sequence) adds the rows in order. The last block of all adds the
// sequences' losses in order. Rows are numbered chunk + sequence: (chunk,
// sequence) pairs along the tokens never share that sum, since each next pair
// raises one of the two. Many experts' rows are too much for one block, so
// above 2^15 + 2^13 of them (chunks times experts) a second launch joins all.
// No floating-point atomics: the same inputs give the same bits. Backward: one
// pass, the probabilities recomputed.
//
// Measured, us: forward, 32768 x 256 in 16 sequences, 17.3: the tokens' loop ends
// after 8.5 (4.7 TB/s), then come steps that run once, each a round trip through
// L2 or more (adding the groups 1, ticket 1.6, joining rows 2 to 4, ticket 1.3,
// losses 1.3); 32768 x 64 12, 256 x 64 6.4. Backward, 32768 x 256: 14.6 (4.6 TB/s),
// instruction issue 63 %.
#include <algorithm>

#include "balance_plan.h"
#include "common.h"
#include "device.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Tokens that a lane adds one after the other: equal probabilities (an untrained
// router) make the rounding errors of a long chain add up, by n / 2 2^-25.
constexpr int kRun = 256;

struct BalanceArgs {
  const void* logits;
  long long ld;
  int T, E, k, S, chunk, chunks;
  int pitch;  // of the partial rows: E rounded up to 4
  float e_per_k;  // E / k
  bool sigmoid;
  float coef;
  const int32_t *ids, *offsets;
  float* psum;      // partial rows [chunks + S][pitch]: probabilities,
  int32_t* csum;    // counts,
  int32_t* nsum;    // [chunks + S]: good tokens
  float* lsum;      // [S][ceil(E / 32)]
  uint32_t* ticket;  // of all blocks
  uint32_t* tickets; // of the sequence that goes on past a chunk, by its first chunk
  int32_t *counts, *tokens;
  float *mean, *loss;
  bool fused;
  // backward
  const int32_t *bcounts, *btokens;
  const float* grad;
  float* dl;
  long long ldd;
  bool accumulate, vec_out;  // vec_out: four experts per store
};

__device__ __forceinline__ int offset_at(const BalanceArgs& a, int i) {
  if (!a.offsets) return i ? a.T : 0;
  return min(max(a.offsets[i], 0), a.T);
}
// The offsets, in shared memory where they fit: they are looked at some five
// times, and a load from memory takes 0.6 us each time. Whole block, before the
// first look.
constexpr int kLocalOffsets = 1024;
struct Offsets {
  const BalanceArgs& a;
  const int32_t* local;
  __device__ __forceinline__ Offsets(const BalanceArgs& a, int32_t* sm)
      : a(a), local(a.S < kLocalOffsets ? sm : nullptr) {
    if (local) {
      for (int i = threadIdx.x; i <= a.S; i += blockDim.x) sm[i] = offset_at(a, i);
      __syncthreads();
    }
  }
  __device__ __forceinline__ int operator()(int i) const { return local ? local[i] : offset_at(a, i); }
};

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

template <int L>
__device__ __forceinline__ float group_max(float v, unsigned mask) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v, unsigned mask) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

// e^v and 1/v of the special-function unit: relative errors about 2^-22, and
// for e^v the exponent's rounding, 2^-24 |v|.
__device__ __forceinline__ float exp_unit(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float rcp_unit(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// x: logits in, probabilities times their sum out; rest: 1 - sigmoid(l). The
// sum's reciprocal, 0 for a bad token: NaN or +inf, or nothing above -inf (its
// x may be anything). Those are where the sum is NaN: exponents +-inf - +-inf,
// or any - NaN; a sigmoid's +inf is looked for.
template <int L, int NV, bool REST>
__device__ __forceinline__ float probabilities(float (&x)[NV], float (&rest)[NV], bool sigmoid, unsigned mask) {
  float m = x[0];
#pragma unroll
  for (int v = 1; v < NV; ++v) m = fmaxf(m, x[v]);
  float s = 0.0f;
  if (!sigmoid) {
    m = group_max<L>(m, mask);
#pragma unroll
    for (int v = 0; v < NV; ++v) s += x[v] = exp_unit(x[v] - m);
  } else if (__ballot_sync(mask, m >= 0.0f) & mask) {
    if (__ballot_sync(mask, m == INFINITY) & mask) s = NAN;
    // u = e^-l is infinite below l = -88, and sigmoid(l) 0.
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const float l = x[v], u = exp_unit(-l);
      s += x[v] = rcp_unit(1.0f + u);
      if (REST) rest[v] = l < 0.0f ? 1.0f - x[v] : u * x[v];
    }
  } else {
    // Every logit is negative: e^(l - max l) / (1 + e^l), so that the sum stays
    // away from 0.
    m = group_max<L>(m, mask);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const float r = rcp_unit(1.0f + exp_unit(x[v]));
      if (REST) rest[v] = r;
      s += x[v] = exp_unit(x[v] - m) * r;
    }
  }
  s = group_sum<L>(s, mask);
  return s > 0.0f ? 1.0f / s : 0.0f;
}

// The first sequence with tokens from t0 on that can hold t0: offsets at or
// below t0, less one. Whole block.
__device__ __forceinline__ int first_sequence(const BalanceArgs& a, const Offsets& off, int t0) {
  int n = 0;
  for (int i = 0; i <= a.S; i += blockDim.x) {
    const int j = i + (int)threadIdx.x;
    n += __syncthreads_count(j <= a.S && off(j) <= t0);
  }
  return max(n - 1, 0);
}

// A warp's 32 experts of sequence s from the sums over its chunks: the outputs,
// and, returned, what they add to the loss.
__device__ __forceinline__ float finish_experts(const BalanceArgs& a, int s, int e, float p, int c, int n) {
  const float each = n ? __frcp_rn((float)n) : 0.0f, mean = p * each;
  if (e < a.E) {
    a.counts[(size_t)s * a.E + e] = c;
    if (a.mean) a.mean[(size_t)s * a.E + e] = mean;
  }
  if (e == 0) a.tokens[s] = n;
  return warp_sum(e < a.E ? (float)c * (a.e_per_k * each) * mean : 0.0f);
}

// The mean of n sequences' losses from their parts; whole block, in a fixed
// order. FP32: all terms are positive, and one FP64 division alone takes longer
// than the sum (3 us with FP64 sums).
__device__ __forceinline__ void write_loss(const BalanceArgs& a, int n, float* sums, int* live) {
  float v = 0.0f;
  int c = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) v += __ldcg(a.lsum + i);
  for (int i = threadIdx.x; i < a.S; i += blockDim.x) c += __ldcg(a.tokens + i) > 0;
  v = warp_sum(v);
  c = __reduce_add_sync(0xffffffffu, c);
  const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
  if (lane == 0) {
    sums[threadIdx.x >> 5] = v;
    live[threadIdx.x >> 5] = c;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    v = warp_sum(lane < warps ? sums[lane] : 0.0f);
    c = __reduce_add_sync(0xffffffffu, lane < warps ? live[lane] : 0);
    if (lane == 0) a.loss[0] = c ? v * a.coef / (float)c : 0.0f;
  }
}
// Whole block: true in the last one of `total` to call; the others' writes are
// then visible.
__device__ __forceinline__ bool last_block(uint32_t* ticket, uint32_t total, int* flag) {
  __syncthreads();
  if (threadIdx.x == 0) {  // its fences stand for the block's: the barriers order the others' accesses with them
    __threadfence();
    *flag = atomicInc(ticket, total - 1) == total - 1;  // back to 0 with the last
    __threadfence();
  }
  __syncthreads();
  return *flag;
}

// The sequence to go on with after the empty sequence s at token t: past all
// empty ones there. Whole block.
__device__ __forceinline__ int next_sequence(const BalanceArgs& a, const Offsets& off, int s, int t) {
  return max(s + 1, first_sequence(a, off, t));
}

// The partial rows of sequence s, all of them written, added in order and
// finished. A thread takes four experts of every slices-th row, four rows' loads
// in flight (one after the other they took 1 us each); up to 32 slices, whose
// sums are then added one by one. Whole block; sums (of 8 * kThreads values at
// least), good: scratch.
template <int kThreads, int kGroups>
__device__ __forceinline__ void join_rows(const BalanceArgs& a, const Offsets& off, int s, int blocks, float* sums,
                                          int32_t* good) {
  const int c0 = off(s) / a.chunk, c1 = (off(s + 1) - 1) / a.chunk + 1;
  const int quads = a.pitch / 4, slices = max(1, min(min(kThreads / quads, min(kGroups, 32)), c1 - c0));
  const int slice = (int)threadIdx.x / quads, e0 = 4 * ((int)threadIdx.x - slice * quads);
  int32_t* counts = reinterpret_cast<int32_t*>(sums + 4 * kThreads);
  if (slice < slices) {
    float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int4 c = make_int4(0, 0, 0, 0);
    int n = 0;
    for (int r = c0 + slice; r < c1; r += 4 * slices) {
      float4 q[4];
      int4 d[4];
      int k[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const size_t row = (size_t)(r + u * slices) + s;
        q[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        d[u] = make_int4(0, 0, 0, 0);
        k[u] = 0;
        if (r + u * slices < c1) {
          q[u] = __ldcg(reinterpret_cast<const float4*>(a.psum + row * a.pitch + e0));
          d[u] = __ldcg(reinterpret_cast<const int4*>(a.csum + row * a.pitch + e0));
          if (e0 == 0) k[u] = __ldcg(a.nsum + row);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        p.x += q[u].x; p.y += q[u].y; p.z += q[u].z; p.w += q[u].w;
        c.x += d[u].x; c.y += d[u].y; c.z += d[u].z; c.w += d[u].w;
        n += k[u];
      }
    }
    *reinterpret_cast<float4*>(sums + slice * a.pitch + e0) = p;
    *reinterpret_cast<int4*>(counts + slice * a.pitch + e0) = c;
    if (e0 == 0) good[slice] = n;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int w = lane; w < slices; w += 32) n += good[w];
  n = __reduce_add_sync(0xffffffffu, n);
  for (int i = warp; i < blocks; i += kThreads / 32) {
    const int e = i * 32 + lane;
    float v = 0.0f;
    int c = 0;
    if (e < a.E)
#pragma unroll 4
      for (int w = 0; w < slices; ++w) {
        v += sums[w * a.pitch + e];
        c += counts[w * a.pitch + e];
      }
    const float part = finish_experts(a, s, e, v, c, n);
    if (lane == 0) a.lsum[(size_t)s * blocks + i] = part;
  }
  __syncthreads();
}

// A pass of a block: up to M sequences that follow one another in its chunk.
template <int M>
struct Pass {
  int seq[M], lo[M], hi[M];  // and their tokens within the chunk
  int m;                     // how many
  int next;                  // sequence to go on with, S at the chunk's end
};
// From sequence s on, those with tokens below t1. Warp 0. Offsets that decrease
// are taken as their running maximum, so that the sequences of a pass always
// follow one another.
template <int M>
__device__ __forceinline__ void find_pass(const BalanceArgs& a, const Offsets& off, int s, int t0, int t1, Pass<M>& pass) {
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  int m = 0, next = a.S, start = max(off(s), t0);
  for (; s < a.S; s += 32) {
    int hi = off(min(s + lane + 1, a.S));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(full, hi, o);
      if (lane >= o) hi = max(hi, v);
    }
    hi = max(hi, start);
    const int before = __shfl_up_sync(full, hi, 1), lo = lane ? before : start;
    const bool in = s + lane < a.S && lo < min(hi, t1);
    const unsigned some = __ballot_sync(full, in);
    const int at = m + __popc(some & ((1u << lane) - 1u));
    if (in && at < M) {
      pass.seq[at] = s + lane;
      pass.lo[at] = lo;
      pass.hi[at] = min(hi, t1);
    }
    const unsigned over = __ballot_sync(full, in && at == M);  // the first that does not fit
    if (over) {
      m = M;
      next = s + __ffs(over) - 1;
      break;
    }
    m += __popc(some);
    start = __shfl_sync(full, hi, 31);
    if (start >= t1) break;
    if (m && !some) {  // a run of empty sequences: the next pass jumps over it
      next = s + 32;
      break;
    }
  }
  if (lane == 0) {
    pass.m = m;
    pass.next = min(next, a.S);
  }
}

template <int L, int NV, int VEC, bool F16>
__global__ void __launch_bounds__(threads_of(NV)) balance_partial_kernel(const BalanceArgs a) {
  constexpr int kThreads = threads_of(NV), kWarps = kThreads / 32;
  constexpr int kGroups = kWarps * (32 / L);  // in a block
  constexpr int kE = L * NV, M = sequences_of(L, NV);  // experts at most, sequences of a pass
  // Rows group + sequence, as the partial rows in memory.
  __shared__ __align__(16) float sums[(kGroups + M) * kE];
  static_assert((kGroups + M) * kE >= 8 * kThreads, "scratch of the joining");
  __shared__ int32_t good[kGroups + M], cnt[M * kE];
  __shared__ float parts[32];
  __shared__ int32_t count[M], flags[2];
  __shared__ Pass<M> pass;
  __shared__ int32_t offs[kLocalOffsets];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & (L - 1), grp = (int)threadIdx.x / L;
  const unsigned mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~(L - 1));
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk), blocks = (a.E + 31) / 32;
  const bool alone = gridDim.x == 1;
  const Offsets off(a, offs);
  float loss = 0.0f;
  int live = 0;
  for (int s0 = t0 < t1 ? first_sequence(a, off, t0) : a.S; s0 < a.S;) {
    if (warp == 0) find_pass<M>(a, off, s0, t0, t1, pass);
    for (int e = threadIdx.x; e < M * kE; e += kThreads) cnt[e] = 0;
    __syncthreads();
    const int m = pass.m;
    if (m == 0) break;
    const int p0 = pass.lo[0], p1 = pass.hi[m - 1];
    // Group g takes tokens from p0 + g per on; the next token's logits and
    // first picks are on their way while one is worked on (not with 32 values
    // per lane: the registers are wanted for the values).
    const int per = (p1 - p0 + kGroups - 1) / kGroups;
    int t = p0 + grp * per;
    const int end = min(p1, t + per);
    constexpr bool kAhead = NV <= 16;
    float x[NV], p[NV] = {};
    int id = -1, n = 0, j = 0, run = 0;
    bool begun = false;  // the row holds the sums of whole runs
    if (t < end) {
      if (kAhead) {
        load_row<L, NV, VEC, F16>(a, t, l, x);
        if (l < a.k) id = a.ids[(size_t)t * a.k + l];
      }
      while (t >= pass.hi[j]) ++j;
      for (;;) {
        float next[NV], rest[NV];
        int next_id = -1;
        if (!kAhead) {
          load_row<L, NV, VEC, F16>(a, t, l, x);
          if (l < a.k) id = a.ids[(size_t)t * a.k + l];
        } else if (t + 1 < end) {
          load_row<L, NV, VEC, F16>(a, t + 1, l, next);
          if (l < a.k) next_id = a.ids[(size_t)(t + 1) * a.k + l];
        }
        const float inv = probabilities<L, NV, false>(x, rest, a.sigmoid, mask);
        if (inv > 0.0f) {
          ++n;
#pragma unroll
          for (int v = 0; v < NV; ++v) p[v] = fmaf(x[v], inv, p[v]);
        }
        if (id >= 0 && id < a.E) atomicAdd(&cnt[j * kE + id], 1);
        for (int q = l + L; q < a.k; q += L) {
          id = a.ids[(size_t)t * a.k + q];
          if (id >= 0 && id < a.E) atomicAdd(&cnt[j * kE + id], 1);
        }
        ++t;
        const bool done = t == end || t == pass.hi[j];
        if (done || ++run == kRun) {
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            float& sum = sums[(grp + j) * kE + expert_of<L, NV, VEC>(l, v)];
            sum = begun ? sum + p[v] : p[v];
            p[v] = 0.0f;
          }
          run = 0;
          begun = !done;
          if (done) {
            if (l == 0) good[grp + j] = n;
            n = 0;
            ++j;
            if (t == end) break;
          }
        }
        if (kAhead) {
#pragma unroll
          for (int v = 0; v < NV; ++v) x[v] = next[v];
          id = next_id;
        }
      }
    }
    __syncthreads();
    // A warp per sequence and 32 experts.
    for (int i = warp; i < m * blocks; i += kWarps) {
      const int q = i / blocks, e = (i - q * blocks) * 32 + lane, s = pass.seq[q], lo = pass.lo[q], hi = pass.hi[q];
      const int g0 = (lo - p0) / per, g1 = (hi - 1 - p0) / per;
      int c = 0;
      for (int g = g0 + lane; g <= g1; g += 32) c += good[g + q];
      c = __reduce_add_sync(0xffffffffu, c);
      float v = 0.0f;
      if (e < a.E)
#pragma unroll 8
        for (int g = g0; g <= g1; ++g) v += sums[(g + q) * kE + e];
      const size_t row = (size_t)blockIdx.x + s;
      if (a.fused && lo == off(s) && hi == off(s + 1)) {
        const float part = finish_experts(a, s, e, v, e < a.E ? cnt[q * kE + e] : 0, c);
        if (lane == 0) {
          parts[i] = part;
          if (!alone) a.lsum[(size_t)s * blocks + (i - q * blocks)] = part;
        }
      } else if (e < a.E) {
        a.psum[row * a.pitch + e] = v;
        a.csum[row * a.pitch + e] = cnt[q * kE + e];
        if (e == 0) a.nsum[row] = c;
      }
      if (e == 0) count[q] = c;
    }
    if (alone) {
      __syncthreads();
      if (warp == 0) {
        loss += warp_sum(lane < m * blocks ? parts[lane] : 0.0f);
        live += __reduce_add_sync(0xffffffffu, lane < m && count[lane < m ? lane : 0] > 0 ? 1 : 0);
      }
    } else if (a.fused) {
      // Sequences that other chunks share are the pass's first or last. The
      // last chunk of a sequence to arrive adds its rows.
      int c0 = 0, c1 = 0;
      bool shared = false;
      if (threadIdx.x < 2 && (threadIdx.x == 0 || m > 1)) {
        const int q = threadIdx.x == 0 ? 0 : m - 1, s = pass.seq[q], b0 = off(s), b1 = off(s + 1);
        shared = pass.lo[q] != b0 || pass.hi[q] != b1;
        c0 = b0 / a.chunk;
        c1 = (b1 - 1) / a.chunk + 1;
      }
      if (__syncthreads_or(shared)) {
        if (threadIdx.x < 2) {
          const uint32_t total = (uint32_t)(c1 - c0);
          __threadfence();
          flags[threadIdx.x] = shared && atomicInc(a.tickets + c0, total - 1) == total - 1;  // back to 0 with the last
          __threadfence();
        }
        __syncthreads();
        for (int w = 0; w < 2; ++w)
          if (flags[w]) join_rows<kThreads, kGroups>(a, off, pass.seq[w ? m - 1 : 0], blocks, sums, good);
      }
    }
    const int from = pass.next;
    s0 = m == M || from == a.S ? from : max(from, first_sequence(a, off, p1));
    __syncthreads();
  }
  if (!a.fused) return;
  // The sequences without tokens, a warp for each.
  for (int s = (int)blockIdx.x * kWarps + warp; s < a.S; s += (int)gridDim.x * kWarps) {
    if (off(s) < off(s + 1)) continue;
    for (int i = 0; i < blocks; ++i) {
      finish_experts(a, s, i * 32 + lane, 0.0f, 0, 0);
      if (lane == 0 && !alone) a.lsum[(size_t)s * blocks + i] = 0.0f;
    }
  }
  if (alone) {
    if (threadIdx.x == 0 && a.loss) a.loss[0] = live ? loss * a.coef / (float)live : 0.0f;
    return;
  }
  if (!last_block(a.ticket, gridDim.x, &flags[0])) return;
  // Tickets are back at 0 by themselves, unless offsets decreased.
  for (int c = threadIdx.x; c < a.chunks; c += kThreads) a.tickets[c] = 0;
  if (a.loss) write_loss(a, blocks * a.S, parts, good);
}

// Block (x, s): experts 32 x .. + 31 of sequence s; its warps share the partial rows.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps) balance_join_kernel(const BalanceArgs a) {
  __shared__ float ps[kJoinWarps][32];
  __shared__ int32_t cs[kJoinWarps][32], ns[kJoinWarps];
  __shared__ float dsum[kJoinWarps];
  __shared__ int flag;
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
  const int lo = offset_at(a, s), hi = offset_at(a, s + 1);
  const int c0 = hi > lo ? lo / a.chunk : 0, c1 = hi > lo ? (hi - 1) / a.chunk + 1 : 0;
  float p = 0.0f;
  int c = 0, n = 0;
  for (int r = c0 + warp; r < c1; r += 8 * kJoinWarps) {
    float q[8];
    int d[8], k[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const size_t row = (size_t)(r + u * kJoinWarps) + s;
      const bool in = r + u * kJoinWarps < c1;
      q[u] = in && e < a.E ? a.psum[row * a.pitch + e] : 0.0f;
      d[u] = in && e < a.E ? a.csum[row * a.pitch + e] : 0;
      k[u] = in ? a.nsum[row] : 0;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      p += q[u];
      c += d[u];
      n += k[u];
    }
  }
  ps[warp][lane] = p;
  cs[warp][lane] = c;
  if (lane == 0) ns[warp] = n;
  __syncthreads();
  if (warp == 0) {
    p = 0.0f;
    c = n = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      p += ps[w][lane];
      c += cs[w][lane];
      n += ns[w];
    }
    const float part = finish_experts(a, s, e, p, c, n);
    if (lane == 0 && a.loss) a.lsum[s * (int)gridDim.x + (int)blockIdx.x] = part;
  }
  if (!a.loss || !last_block(a.ticket, gridDim.x * gridDim.y, &flag)) return;
  write_loss(a, (int)(gridDim.x * gridDim.y), dsum, ns);
}

template <int L, int NV, int VEC, bool F16>
__global__ void __launch_bounds__(back_threads_of(NV)) balance_back_kernel(const BalanceArgs a) {
  constexpr int kThreads = back_threads_of(NV);
  constexpr int G = 32 / L, kGroups = kThreads / 32 * G;
  __shared__ int32_t offs[kLocalOffsets];
  griddep_wait();
  griddep_launch_dependents();
  const Offsets off(a, offs);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & (L - 1), grp = warp * G + lane / L;
  const unsigned mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~(L - 1));
  const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
  int live = 0;
  for (int i = 0; i < a.S; i += kThreads) {
    const int j = i + (int)threadIdx.x;
    live += __syncthreads_count(j < a.S && a.btokens[j] > 0);
  }
  const float g = a.coef * (a.grad ? *a.grad : 1.0f);
  for (int s = first_sequence(a, off, t0); s < a.S;) {
    const int b0 = off(s), lo = max(b0, t0), hi = min(off(s + 1), t1);
    if (b0 >= t1) break;
    if (lo >= hi) {
      s = next_sequence(a, off, s, lo);
      continue;
    }
    constexpr bool kAhead = NV <= 16;
    float x[NV], f[NV];
    int t = lo + grp;
    if (kAhead && t < hi) load_row<L, NV, VEC, F16>(a, t, l, x);
    const float n = (float)a.btokens[s];
    const float unit = n > 0.0f ? (float)a.E / ((float)a.k * n) : 0.0f;
    const float outer = n > 0.0f ? g / ((float)live * n) : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = expert_of<L, NV, VEC>(l, v);
      f[v] = e < a.E ? (float)a.bcounts[(size_t)s * a.E + e] * unit : 0.0f;
    }
    for (; t < hi; t += kGroups) {
      float next[NV], rest[NV];
      if (!kAhead) load_row<L, NV, VEC, F16>(a, t, l, x);
      if (kAhead && t + kGroups < hi) load_row<L, NV, VEC, F16>(a, t + kGroups, l, next);
      const float inv = probabilities<L, NV, true>(x, rest, a.sigmoid, mask);
      float dot = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) dot = fmaf(x[v], f[v], dot);
      dot = group_sum<L>(dot, mask) * inv;
      const float c = outer * inv;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        x[v] = inv > 0.0f ? c * x[v] * (f[v] - dot) : 0.0f;
        if (a.sigmoid && inv > 0.0f) x[v] *= rest[v];
      }
      float* out = a.dl + (size_t)t * (size_t)a.ldd;
      if (VEC == 4 && a.vec_out) {
#pragma unroll
        for (int j = 0; j < NV / 4; ++j) {
          const int e = 4 * (l + L * j);
          if (e < a.E) {
            float4* o = reinterpret_cast<float4*>(out + e);
            float4 d = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            if (a.accumulate) {
              const float4 q = *o;
              d.x += q.x; d.y += q.y; d.z += q.z; d.w += q.w;
            }
            *o = d;
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = expert_of<L, NV, VEC>(l, v);
          if (e < a.E) out[e] = a.accumulate ? out[e] + x[v] : x[v];
        }
      }
      if (kAhead)
#pragma unroll
        for (int v = 0; v < NV; ++v) x[v] = next[v];
    }
    ++s;
  }
}

struct Ws {
  size_t psum, csum, nsum, lsum, tickets, total;
};
Ws ws_of(int T, int E, int S) {
  const size_t rows = (size_t)std::min((T + kMinChunk - 1) / kMinChunk, max_chunks(E)) + S;
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  Ws w;
  size_t o = kWorkspaceHeader;
  // In the same place for every T, E and S: they have to stay zero between calls.
  w.tickets = o; o += up(max_chunks(1024) * 4);
  const size_t pitch = (size_t)(E + 3) / 4 * 4;
  w.psum = o; o += up(rows * pitch * 4);
  w.csum = o; o += up(rows * pitch * 4);
  w.nsum = o; o += up(rows * 4);
  w.lsum = o; o += up((size_t)S * ((E + 31) / 32) * 4);
  w.total = o;
  return w;
}

template <bool BACK, int L, int NV, int VEC, bool F16>
cudaError_t launch_tokens(cudaLaunchConfig_t cfg, const BalanceArgs& a) {
  cfg.blockDim = dim3(BACK ? back_threads_of(NV) : threads_of(NV));
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

void set_chunks(BalanceArgs& a, bool back) {
  const BalancePlan p = balance_plan(a.T, a.E, a.S, back);
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  a.fused = p.fused;
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(dim3 grid, int threads, cudaStream_t st) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
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
  if (T < 0 || T > (1 << 27) || E < 1 || E > 1024 || S < 1 || S > 65535) return 0;
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
  a.pitch = (E + 3) / 4 * 4;
  a.e_per_k = (float)E / (float)k;
  moe::set_chunks(a, false);
  a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  a.coef = cfg->coef;
  a.ids = ids;
  a.offsets = offsets;
  a.psum = reinterpret_cast<float*>(w8 + w.psum);
  a.csum = reinterpret_cast<int32_t*>(w8 + w.csum);
  a.nsum = reinterpret_cast<int32_t*>(w8 + w.nsum);
  a.lsum = reinterpret_cast<float*>(w8 + w.lsum);
  a.ticket = reinterpret_cast<uint32_t*>(w8) + 1;
  a.tickets = reinterpret_cast<uint32_t*>(w8 + w.tickets);
  a.counts = counts;
  a.tokens = tokens;
  a.mean = mean;
  a.loss = loss;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  {
    const moe::Launch l(dim3((unsigned)a.chunks), 0, st);
    e = moe::launch_tokens<false>(l.cfg, a, logit_type);
  }
  if (e == cudaSuccess && !a.fused) {
    const moe::Launch l(dim3((unsigned)((E + 31) / 32), (unsigned)S), 32 * moe::kJoinWarps, st);
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
  moe::set_chunks(a, true);
  a.vec_out = reinterpret_cast<uintptr_t>(dlogits) % 16 == 0 && ldd % 4 == 0;
  a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  a.coef = cfg->coef;
  a.offsets = offsets;
  a.bcounts = counts;
  a.btokens = tokens;
  a.grad = grad_loss;
  a.dl = dlogits;
  a.ldd = ldd;
  a.accumulate = accumulate != 0;
  const moe::Launch l(dim3((unsigned)a.chunks), 0, static_cast<cudaStream_t>(stream));
  const cudaError_t e = moe::launch_tokens<true>(l.cfg, a, logit_type);
  if (e != cudaSuccess) return moe::fail(MOE_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return MOE_OK;
}

}  // extern "C"
