// Block-scaled FP8 matrix product and the shared SwiGLU FFN built from it.
//   y[t][n] = sum_b xs[t][b] ws[n/128][b] sum_{c in block b} xq[t][c] wq[n][c]
// with E4M3 codes, one scale per 1 x 128 block of x and per 128 x 128 block of
// W, FP32 sums.
//
// Tensor-core kernels: tokens are the MMA's M, rows of W its N; both operands
// come by TMA in the 128-byte-swizzled K-major layout, one scale block (128
// codes, 128 bytes) per pipeline step. The scales change every step, so a
// step's four MMAs (K = 32 each) start a fresh FP32 accumulator in tensor
// memory, and promotion warps read it back and add it, times its scale, to
// sums in registers. A token is a lane of tensor memory, hence one thread; the
// weight scale is the same for 128 columns: the scale of a step is one number
// per thread, and promotion one packed FMA per two sums.
//
// fp8_gemm_kernel: a block and 128 tokens by NT columns, the K steps of a tile
// split over a cluster where the tiles are few. fp8_pair_kernel: two blocks and
// 256 x 256. plan_of picks; up to 16 tokens take fp8_gemv.cu instead (64 tokens
// against 4096 x 2048: 6.2 us here; one token there 2.8 us, here 6.5).
#include <algorithm>
#include <mutex>

#include "common.h"
#include "device.cuh"
#include "fp8.cuh"
#include "fp8_gemv.h"
#include "fp8_plan.h"
#include "kernels.h"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int BM = kPlanTokens;   // tokens per tile
constexpr int BK = fp8::kBlock;   // codes per step: one scale block, one swizzle row
constexpr uint32_t kABytes = BM * BK;
// Scales of up to 32 steps in shared memory: the tokens' [step][token] (odd
// pitch: written by step, read by token), the two weight blocks' [2][step].
constexpr int kChunk = 32, kScalePitch = BM + 1;
constexpr uint32_t kScaleBytes = (kChunk * kScalePitch + 2 * kChunk) * 4;

// Geometry by tile width. Warp 0 issues TMA, warp 1 owns tensor memory and
// issues the MMAs, the others promote, at most 64 columns each.
template <int NT>
struct Geo {
  static constexpr int cols = NT < 64 ? NT : 64;  // columns per promotion warp
  static constexpr int promo = 4 * (NT / cols);
  static constexpr int threads = 64 + 32 * promo;
  static constexpr uint32_t stage = kABytes + (uint32_t)NT * BK;
  static constexpr int stages = NT == 256 ? 4 : NT == 128 ? 6 : 8;
  static constexpr int bufs = NT == 256 ? 2 : NT == 128 ? 4 : 8;  // accumulators in tensor memory
  static constexpr uint32_t tmem_cols = (uint32_t)bufs * NT;
  static constexpr uint32_t off_scale = (uint32_t)stages * stage;
  static constexpr uint32_t off_ctrl = off_scale + kScaleBytes;
  static constexpr size_t smem = (size_t)off_ctrl + 4096 + 1024;  // control block, alignment
  static constexpr int red_pitch = NT + 4;                        // floats per row of a partial tile
  static_assert((size_t)BM * red_pitch * 4 <= off_scale, "partial tile fits the stage area");
  static_assert(tmem_cols <= 512 && (tmem_cols & (tmem_cols - 1)) == 0, "tensor memory budget");
};

struct GemmArgs {
  int T, N, K;        // N: rows of W (output columns; Is for gate/up)
  int nb;             // scale blocks along K
  int mt, tiles;      // token tiles, tiles in all
  int splits;         // blocks of a cluster share one tile's K steps
  uint32_t a_bytes;   // bytes of the token tile's box
  const float *xs, *ws, *ws2;
  __half* y;          // product
  uint8_t* hq;        // gate/up: h codes [T][N] and scales [T][nbh]
  float* hs;
  int nbh;
  int32_t* flags;
};

struct Bars {
  uint64_t *full, *empty, *acc_full, *acc_empty;
  uint32_t* tmem_slot;
  int* abort;
  float* amax;  // [4][BM], gate/up
};
template <int NT>
__device__ __forceinline__ Bars bars_at(uint8_t* p) {
  using G = Geo<NT>;
  Bars b;
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  b.full = q; q += G::stages;
  b.empty = q; q += G::stages;
  b.acc_full = q; q += G::bufs;
  b.acc_empty = q; q += G::bufs;
  b.tmem_slot = reinterpret_cast<uint32_t*>(q);
  b.abort = reinterpret_cast<int*>(b.tmem_slot + 1);
  b.amax = reinterpret_cast<float*>(p + 1024);
  return b;
}
__device__ __forceinline__ void abort_block(const Bars& b, int32_t* flags) {
  atomicOr(flags, 4);
  *reinterpret_cast<volatile int*>(b.abort) = 1;
}
__device__ __forceinline__ bool is_aborted(const Bars& b) { return *reinterpret_cast<volatile int*>(b.abort) != 0; }

// sum (two FP32 lanes) += d * s (both lanes).
__device__ __forceinline__ void fma2(uint64_t& sum, uint32_t d0, uint32_t d1, uint64_t s2) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(d), "l"(s2));
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes of another block's shared memory, at this block's address `a`.
__device__ __forceinline__ float4 ld_cluster(uint32_t a, uint32_t rank) {
  uint32_t ra;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(ra)
               : "memory");
  return v;
}
// Named barrier over the promotion warps; true for all if q is true for any.
template <int THREADS>
__device__ __forceinline__ bool promo_any(bool q) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.or.pred p, 1, %2, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r) : "r"((uint32_t)q), "n"(THREADS) : "memory");
  return r != 0;
}

// The larger of the two, NaN if one is.
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// h = silu(gate) * up of N values in place of gate, and their largest
// magnitude (NaN or infinite if one of them is). A reciprocal shared by two
// SiLUs, 1/a = b / (ab), saves a quarter of the special-function results, but
// ab overflows at strongly negative gates: with the exponent capped for that
// silu(-60) came out 9e7 times too large, and a test for such gates costs more
// than the reciprocals (2048 tokens of 2048 x 4096, us: capped 53.3, one
// reciprocal each 53.6, shared behind a test 54.1).
template <int N>
__device__ __forceinline__ float swiglu(float (&gt)[N], const float (&up)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    gt[i] = fp8::silu(gt[i]) * up[i];
    m = fmax_nan(m, fabsf(gt[i]));
  }
  return m;
}

// GATEUP: the tile is 128 rows of W_g and the same 128 of W_u; the epilogue
// forms h = silu(gate) * up of one 128-column block and quantises it.
template <int NT, bool GATEUP>
__global__ void __launch_bounds__(Geo<NT>::threads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_w2, const GemmArgs a) {
  using G = Geo<NT>;
  static_assert(!GATEUP || NT == 256, "gate/up tile");
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = tc::align1024(smraw);
  const Bars b = bars_at<NT>(sm + G::off_ctrl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_w);
    if (GATEUP) tc::tma_prefetch_desc(&map_w2);
    for (int s = 0; s < G::stages; ++s) {
      tc::bar_init(&b.full[s], 1);
      tc::bar_init(&b.empty[s], 1);
    }
    for (int s = 0; s < G::bufs; ++s) {
      tc::bar_init(&b.acc_full[s], 1);
      tc::bar_init(&b.acc_empty[s], G::promo);
    }
    *b.abort = 0;
    tc::bar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc(b.tmem_slot, G::tmem_cols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *b.tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const int S = a.splits;
  const int rank = S > 1 ? (int)cluster_rank() : 0;
  const int kb0 = a.nb * rank / S, kb1 = a.nb * (rank + 1) / S;
  const int first = (int)blockIdx.x / S, stride = (int)gridDim.x / S;
  constexpr int kN = GATEUP ? 128 : NT;  // output columns per tile

  if (warp == 0) {
    int g = 0;
    bool ok = true;
    for (int tile = first; tile < a.tiles && ok; tile += stride) {
      const int m0 = (tile % a.mt) * BM, n0 = (tile / a.mt) * kN;
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        const int s = g % G::stages;
        if (g >= G::stages && !tc::bar_wait_warp(&b.empty[s], ((g / G::stages) - 1) & 1)) {
          if (lane == 0) abort_block(b, a.flags);
          ok = false;
          break;
        }
        if (__any_sync(0xffffffffu, is_aborted(b))) {
          ok = false;
          break;
        }
        if (tc::elect_one()) {
          uint8_t* st = sm + (size_t)s * G::stage;
          tc::bar_expect_tx(&b.full[s], a.a_bytes + NT * BK);
          tc::tma_load_2d(st, &map_x, kb * BK, m0, &b.full[s]);
          tc::tma_load_2d(st + kABytes, &map_w, kb * BK, n0, &b.full[s]);
          if (GATEUP) tc::tma_load_2d(st + kABytes + 128 * BK, &map_w2, kb * BK, n0, &b.full[s]);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0)  // loads still in flight land before the block leaves (bounded)
      for (int i = g > G::stages ? g - G::stages : 0; i < g; ++i)
        tc::bar_wait(&b.full[i % G::stages], (i / G::stages) & 1);
  } else if (warp == 1) {
    constexpr uint32_t idesc = tc::idesc_f16(BM, NT);
    int g = 0;
    bool ok = true;
    for (int tile = first; tile < a.tiles && ok; tile += stride) {
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        const int s = g % G::stages, u = g % G::bufs;
        if ((g >= G::bufs && !tc::bar_wait_warp(&b.acc_empty[u], ((g / G::bufs) - 1) & 1)) ||
            !tc::bar_wait_warp(&b.full[s], (g / G::stages) & 1)) {
          if (lane == 0) abort_block(b, a.flags);
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t base = tc::smem_addr(sm + (size_t)s * G::stage);
        const uint64_t ad = tc::sw128_desc(base), bd = tc::sw128_desc(base + kABytes);
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            tc::mma_f8(tmem + (uint32_t)(u * NT), ad + 2 * kk, bd + 2 * kk, idesc, kk > 0);
          tc::mma_commit(&b.empty[s]);
          tc::mma_commit(&b.acc_full[u]);
        }
        __syncwarp();
      }
    }
  } else {
    // Promotion warp: lane quarter q4, columns [c0, c0 + cols) (gate/up: 32
    // gate columns and the same 32 of up).
    const int q4 = warp & 3, j4 = (warp - 2) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(32 * q4) << 16);
    const uint32_t ca = GATEUP ? 32 * j4 : G::cols * j4, cb = GATEUP ? 128 + 32 * j4 : ca + 32;
    constexpr int kPairs = G::cols / 2;
    float* sx = reinterpret_cast<float*>(sm + G::off_scale);
    float* sw = sx + kChunk * kScalePitch;
    const int blk = GATEUP ? 0 : (int)ca / 128;
    int g = 0;
    bool ok = true;
    for (int tile = first; tile < a.tiles; tile += stride) {
      const int m0 = (tile % a.mt) * BM, n0 = (tile / a.mt) * kN;
      const int r = 32 * q4 + lane, row = m0 + r;
      const bool live = row < a.T;
      uint64_t sum[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) sum[i] = 0;
      bool stop = false;
      for (int kc = kb0; kc < kb1; kc += kChunk) {
        // The chunk's scales, all loads in flight at once. One verdict for all
        // the warps, and the last chunk's scales have been read.
        const int steps = min(kChunk, kb1 - kc);
        if ((stop = promo_any<32 * G::promo>(!ok))) break;
        const int tid = (int)threadIdx.x - 64, e = tid & 31, rows = min(BM, a.T - m0);
        if (e < steps) {
#pragma unroll 8
          for (int i = tid >> 5; i < rows; i += G::promo)
            sx[e * kScalePitch + i] = a.xs[(size_t)(m0 + i) * a.nb + kc + e];
          if (tid < 64) {  // warp i: weight block i of the tile
            const int wb = n0 / 128 + (GATEUP ? 0 : tid >> 5);
            const float* pw = GATEUP && tid >= 32 ? a.ws2 : a.ws;
            sw[tid] = wb * 128 < a.N ? pw[(size_t)wb * a.nb + kc + e] : 0.0f;
          }
        }
        asm volatile("barrier.sync 1, %0;" ::"n"(32 * G::promo) : "memory");
        for (int st = 0; st < steps; ++st, ++g) {
          const int u = g % G::bufs;
          const float x = sx[st * kScalePitch + r];
          const float sa = x * sw[blk * kChunk + st], sb = GATEUP ? x * sw[kChunk + st] : sa;
          if (!tc::bar_wait_warp(&b.acc_full[u], (g / G::bufs) & 1)) {
            if (lane == 0) abort_block(b, a.flags);
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t buf = tl + (uint32_t)(u * NT);
          const uint64_t sa2 = pack2(sa, sa), sb2 = GATEUP ? pack2(sb, sb) : sa2;
          uint32_t d[16];
#pragma unroll
          for (int c = 0; c < G::cols / 16; ++c) {
            tc::tmem_ld16u(buf + (c < 2 ? ca + 16 * c : cb + 16 * (c - 2)), d);
            if (c == G::cols / 16 - 1) {
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::bar_arrive(&b.acc_empty[u]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) fma2(sum[8 * c + i], d[2 * i], d[2 * i + 1], c < 2 ? sa2 : sb2);
          }
        }
      }
      if (stop) break;
      if (S > 1) {  // partial tile to shared memory (every stage has been consumed)
        if (live && ok) {
          float* red = reinterpret_cast<float*>(sm) + (size_t)r * G::red_pitch;
#pragma unroll
          for (int i = 0; i < kPairs; i += 2) {
            const float2 p = unpack2(sum[i]), q = unpack2(sum[i + 1]);
            *reinterpret_cast<float4*>(red + (i < 16 ? ca + 2 * i : cb + 2 * (i - 16))) =
                make_float4(p.x, p.y, q.x, q.y);
          }
        }
        break;
      }
      if (!GATEUP) {
        if (live && ok) {
          __half* out = a.y + (size_t)row * a.N + n0 + ca;
          const int left = a.N - (n0 + (int)ca);
          if (a.N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < kPairs; i += 4) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 p = unpack2(sum[i + e]);
                h[e] = half2_bits(p.x, p.y);
              }
              if (2 * i < left) *reinterpret_cast<uint4*>(out + 2 * i) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
              const float2 p = unpack2(sum[i]);
              if (2 * i < left) out[2 * i] = __float2half_rn(p.x);
              if (2 * i + 1 < left) out[2 * i + 1] = __float2half_rn(p.y);
            }
          }
        }
      } else {
        // h of 32 columns per thread; the block's amax over its four warps.
        float h[32], up[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 p = unpack2(sum[i]), q = unpack2(sum[(16 + i) % kPairs]);
          h[2 * i] = p.x; h[2 * i + 1] = p.y;
          up[2 * i] = q.x; up[2 * i + 1] = q.y;
        }
        float m = swiglu(h, up);
        b.amax[j4 * BM + r] = m;
        asm volatile("barrier.sync 1, %0;" ::"n"(32 * G::promo) : "memory");
#pragma unroll
        for (int w = 0; w < 4; ++w) m = fmax_nan(m, b.amax[w * BM + r]);
        // Maxima read before the next tile's; one verdict for all the warps.
        if (promo_any<32 * G::promo>(!ok || is_aborted(b))) break;
        const fp8::BlockScale bs = fp8::block_scale(m);
        if (live) {
          uint8_t* out = a.hq + (size_t)row * a.N + n0 + ca;
#pragma unroll
          for (int i = 0; i < 32; i += 16) {
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              c[e] = fp8::encode4(h[i + 4 * e] * bs.inv, h[i + 4 * e + 1] * bs.inv, h[i + 4 * e + 2] * bs.inv,
                                  h[i + 4 * e + 3] * bs.inv);
            if (n0 + (int)ca + i < a.N) *reinterpret_cast<uint4*>(out + i) = make_uint4(c[0], c[1], c[2], c[3]);
          }
          if (j4 == 0) a.hs[(size_t)row * a.nbh + n0 / 128] = bs.scale;
        }
      }
    }
  }
  if (S > 1) {
    // The cluster's partial tiles, added in rank order (the same order every
    // time), each block finishing its share of the tile.
    __syncwarp();
    cluster_sync();
    const int m0 = (first % a.mt) * BM, n0 = (first / a.mt) * kN;
    const int rows = min(BM, a.T - m0);
    const uint32_t red = tc::smem_addr(sm);
    if (!GATEUP) {
      constexpr int kQ = NT / 4;  // 4-column pieces per row
      for (int i = rank * G::threads + (int)threadIdx.x; i < rows * kQ; i += S * G::threads) {
        const int r = i / kQ, c = (i % kQ) * 4;
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int p = 0; p < S; ++p) {
          const float4 v = ld_cluster(red + (uint32_t)(r * G::red_pitch + c) * 4, (uint32_t)p);
          t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
        }
        __half* out = a.y + (size_t)(m0 + r) * a.N + n0 + c;
        const int left = a.N - (n0 + c);
        if (a.N % 4 == 0) {
          if (left > 0) *reinterpret_cast<uint2*>(out) = make_uint2(half2_bits(t.x, t.y), half2_bits(t.z, t.w));
        } else {
          const float v[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < left) out[e] = __float2half_rn(v[e]);
        }
      }
    } else {
      constexpr int kWarps = G::threads / 32;
      for (int r = rank * kWarps + warp; r < rows; r += S * kWarps) {
        float h[4] = {}, up[4] = {};
        for (int p = 0; p < S; ++p) {
          const float4 v = ld_cluster(red + (uint32_t)(r * G::red_pitch + 4 * lane) * 4, (uint32_t)p);
          const float4 w = ld_cluster(red + (uint32_t)(r * G::red_pitch + 128 + 4 * lane) * 4, (uint32_t)p);
          h[0] += v.x; h[1] += v.y; h[2] += v.z; h[3] += v.w;
          up[0] += w.x; up[1] += w.y; up[2] += w.z; up[3] += w.w;
        }
        float m = swiglu(h, up);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const fp8::BlockScale bs = fp8::block_scale(m);
        if (n0 + 4 * lane < a.N)
          *reinterpret_cast<uint32_t*>(a.hq + (size_t)(m0 + r) * a.N + n0 + 4 * lane) =
              fp8::encode4(h[0] * bs.inv, h[1] * bs.inv, h[2] * bs.inv, h[3] * bs.inv);
        if (lane == 0) a.hs[(size_t)(m0 + r) * a.nbh + n0 / 128] = bs.scale;
      }
    }
    __syncwarp();
    cluster_sync();  // nobody leaves while its partial tile is read
  }
  tc::gemm_teardown(tmem, G::tmem_cols);
}

// ---- SM pairs: 256 tokens by 256 rows of W ----------------------------------
// Two blocks of a cluster run one tile with cta_group::2 MMAs: each holds its
// 128 tokens (A) and half of the weight rows (B), and each accumulates its
// tokens against all 256 rows. Against a block on its own with a 128 x 256
// tile (2.25 PFLOP/s with the promotion left out), a step's TMA writes fall
// from 48 KB to 32 KB per SM, and so do the operand bytes its MMAs read from it.
//
// Measured: a step's MMAs end every 710 cycles, back to back and whatever the
// promotion does, against 512 at the tensor pipe's nominal rate (the pipe is
// active 64 % of the time): 32 KB written and what the two tensor cores read of
// both blocks' operands keep the shared memory busy. The promotion needs 8 % on
// top (its FMAs issue every other cycle: 260 of a step's cycles per scheduler).
// 8192 x 8192 x 4096: 190 us, 2.9 PFLOP/s, 75 % of twice the measured BF16
// rate; under sustained load the power limit takes it to 215 us.
// 2048 x 4096 x 2048: 18.4 us; its 128 tiles are 1.7 waves of 76 pairs, a tile
// is 16 steps, and starting, switching tiles and ending take 5 us.
// Warps: 0 TMA, 1 tensor memory and (in the leading block) MMA issue, 2-3
// scales, 4-11 promotion (a lane quarter, 128 columns each).
struct Pair {
  static constexpr int promo = 8, threads = 384;
  static constexpr int stages = 4, bufs = 2, groups = 2, slots = 4 * groups;  // scales: groups of four steps
  static constexpr uint32_t stage = kABytes + 128 * BK;  // per block: 128 tokens, 128 rows of W
  static constexpr uint32_t off_out = stages * stage;    // [promo][2][32 rows][64 columns] FP16
  static constexpr uint32_t off_scale = off_out + promo * 8192;
  static constexpr uint32_t off_ctrl = off_scale + slots * 2 * BM * 4;
  static constexpr size_t smem = (size_t)off_ctrl + 4096 + 1024;
};
struct PairBars {
  uint64_t *full, *empty, *acc_full, *acc_empty, *sc_full, *sc_empty;
  uint32_t* tmem_slot;
  int* abort;
  float* amax;
};
__device__ __forceinline__ PairBars pair_bars(uint8_t* p) {
  PairBars b;
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  b.full = q; q += Pair::stages;
  b.empty = q; q += Pair::stages;
  b.acc_full = q; q += Pair::bufs;
  b.acc_empty = q; q += Pair::bufs;
  b.sc_full = q; q += Pair::groups;
  b.sc_empty = q; q += Pair::groups;
  b.tmem_slot = reinterpret_cast<uint32_t*>(q);
  b.abort = reinterpret_cast<int*>(b.tmem_slot + 1);
  b.amax = reinterpret_cast<float*>(p + 1024);
  return b;
}
__device__ __forceinline__ void pair_abort(const PairBars& b, int32_t* flags) {
  atomicOr(flags, 4);
  *reinterpret_cast<volatile int*>(b.abort) = 1;
}

// A promotion warp's wait: no verdict to agree on. After a wait that ran out
// (here or in another role of the block) the rest return at once, the warp
// walks through its tiles without results, and every barrier is met.
// (Shared-memory addresses, not pointers: the promotion loop is short of
// registers.)
__device__ __forceinline__ void pair_wait(uint32_t bar, uint32_t parity, uint32_t abort, int32_t* flags) {
  if (!tc::bar_try_wait_at(bar, parity)) {
    const uint64_t t0 = tc::global_ns();
    for (;;) {
      if (tc::bar_try_wait_at(bar, parity)) break;
      uint32_t gone;
      asm volatile("ld.volatile.shared::cta.u32 %0, [%1];" : "=r"(gone) : "r"(abort) : "memory");
      if (gone) break;
      if (tc::global_ns() - t0 > tc::kWaitNs) {
        atomicOr(flags, 4);
        asm volatile("st.volatile.shared::cta.u32 [%0], %1;" ::"r"(abort), "r"(1) : "memory");
        break;
      }
    }
  }
  __syncwarp();
}

template <bool GATEUP>
__global__ void __launch_bounds__(Pair::threads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_w2, const __grid_constant__ CUtensorMap map_y,
                    const GemmArgs a) {
  using G = Pair;
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = tc::align1024(smraw);
  const PairBars b = pair_bars(sm + G::off_ctrl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(rank && GATEUP ? &map_w2 : &map_w);
    tc::tma_prefetch_desc(&map_y);
    for (int s = 0; s < G::stages; ++s) {
      tc::bar_init(&b.full[s], 1);
      tc::bar_init(&b.empty[s], 1);
    }
    for (int s = 0; s < G::bufs; ++s) {
      tc::bar_init(&b.acc_full[s], 1);
      tc::bar_init(&b.acc_empty[s], 2 * G::promo);
    }
    for (int s = 0; s < G::groups; ++s) {
      tc::bar_init(&b.sc_full[s], 2);
      tc::bar_init(&b.sc_empty[s], G::promo);
    }
    *reinterpret_cast<volatile int*>(b.abort) = 0;
    tc::bar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc2(b.tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = *b.tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const int nb = a.nb;
  const int first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
  constexpr int kN = GATEUP ? 128 : 256;  // output columns per tile

  // 384 x 168 registers at launch = 128 x 72 + 256 x 216.
  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // Lane quarter q4; 128 columns from 128 j2 (gate/up: 64 of each from
    // 64 j2), taken from tensor memory 32 at a time (a load returns in some 35
    // cycles; the other warp of the scheduler has FMAs to issue meanwhile).
    const int q4 = warp & 3, j2 = (warp - 4) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(32 * q4) << 16);
    const uint32_t c0 = GATEUP ? 64 * j2 : 128 * j2;
    auto col = [&](int c) { return GATEUP && c >= 2 ? 128 + c0 + 32 * (c - 2) : c0 + 32 * c; };
    const float* sca = reinterpret_cast<const float*>(sm + G::off_scale) + (GATEUP ? 0 : j2 * BM) + 32 * q4 + lane;
    const uint32_t acc_full = tc::smem_addr(b.acc_full), sc_full = tc::smem_addr(b.sc_full);
    const uint32_t abort = tc::smem_addr(b.abort);
    const uint32_t acc_empty0 = tc::map_rank(tc::smem_addr(&b.acc_empty[0]), 0);
    uint8_t* out = sm + G::off_out + (warp - 4) * 8192;
    int g = 0, gg = 0;
    for (int tile = first; tile < a.tiles; tile += stride) {
      const int m0 = (tile % a.mt) * 256 + rank * BM, n0 = (tile / a.mt) * kN;
      const int r = 32 * q4 + lane, row = m0 + r;
      uint64_t sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      for (int kb = 0; kb < nb; ++kb, ++g) {
        const int u = g % G::bufs, e = kb & 3;
        if (e == 0) pair_wait(sc_full + 8 * (gg % G::groups), (gg / G::groups) & 1, abort, a.flags);
        const float* sc = sca + ((gg % G::groups) * 4 + e) * 2 * BM;
        const float sa = sc[0], sb = GATEUP ? sc[BM] : sa;
        pair_wait(acc_full + 8 * u, (g / G::bufs) & 1, abort, a.flags);
        tc::tc_fence_after();
        const uint32_t buf = tl + (uint32_t)(u * 256);
        const uint64_t sa2 = pack2(sa, sa), sb2 = GATEUP ? pack2(sb, sb) : sa2;
        if (e == 3 || kb == nb - 1) {
          if (lane == 0) tc::bar_arrive_at(sc_full + 8 * G::groups + 8 * (gg % G::groups));
          ++gg;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t d[32];
          tc::tmem_ld32(buf + col(c), d);
          tc::tmem_ld32_wait(d);
          if (c == 3) {
            tc::tc_fence_before();
            if (lane == 0) tc::bar_arrive_cluster(acc_empty0 + 8 * u);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) fma2(sum[16 * c + i], d[2 * i], d[2 * i + 1], c < 2 ? sa2 : sb2);
        }
      }
      const bool ok = *reinterpret_cast<volatile int*>(b.abort) == 0;
      if (!GATEUP) {
        if (!ok) continue;
        // Rows of 64 FP16 columns in the 128-byte swizzle.
        if (lane < 2) tc::tma_store_wait_read();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 p = unpack2(sum[4 * c + e]);
            h[e] = half2_bits(p.x, p.y);
          }
          *reinterpret_cast<uint4*>(out + (c >> 3) * 4096 + tc::sw128_offset(lane, c & 7)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
        const int y0 = m0 + 32 * q4, x0 = n0 + (int)c0;
        if (a.N % 8 == 0) {
          tc::fence_async_smem();
          __syncwarp();
          // A lane per store: one lane issuing both takes twice as long.
          if (lane < 2 && y0 < a.T && x0 + 64 * lane < a.N)
            tc::tma_store_2d(&map_y, x0 + 64 * lane, y0, out + 4096 * lane);
        } else {
          // Rows that TMA cannot address (16-byte pitch): two columns per lane.
          __syncwarp();
          for (int i = 0; i < 2 * min(32, a.T - y0); ++i) {
            const int rr = i >> 1, x = x0 + 64 * (i & 1) + 2 * lane;
            const uint32_t v = *reinterpret_cast<const uint32_t*>(out + 4096 * (i & 1) + tc::sw128_offset(rr, lane >> 2) +
                                                                  4 * (lane & 3));
            __half* o = a.y + (size_t)(y0 + rr) * a.N + x;
            if (x < a.N) o[0] = __ushort_as_half((unsigned short)v);
            if (x + 1 < a.N) o[1] = __ushort_as_half((unsigned short)(v >> 16));
          }
          __syncwarp();
        }
      } else {
        float h[64], up[64];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 p = unpack2(sum[i]), q = unpack2(sum[32 + i]);
          h[2 * i] = p.x; h[2 * i + 1] = p.y;
          up[2 * i] = q.x; up[2 * i + 1] = q.y;
        }
        float m = swiglu(h, up);
        if (lane == 0) tc::tma_store_wait_read();
        __syncwarp();
        b.amax[j2 * BM + r] = m;
        asm volatile("barrier.sync 1, %0;" ::"n"(32 * G::promo) : "memory");
        m = fmax_nan(m, b.amax[(j2 ^ 1) * BM + r]);
        const fp8::BlockScale bs = fp8::block_scale(m);
#pragma unroll
        for (int i = 0; i < 64; i += 16) {
          uint32_t c[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            c[e] = fp8::encode4(h[i + 4 * e] * bs.inv, h[i + 4 * e + 1] * bs.inv, h[i + 4 * e + 2] * bs.inv,
                                h[i + 4 * e + 3] * bs.inv);
          *reinterpret_cast<uint4*>(out + 64 * lane + i) = make_uint4(c[0], c[1], c[2], c[3]);
        }
        tc::fence_async_smem();
        // The maxima have been read before the next tile's are written.
        asm volatile("barrier.sync 1, %0;" ::"n"(32 * G::promo) : "memory");
        const int y0 = m0 + 32 * q4, x0 = n0 + (int)c0;  // rows of 64 codes; Is is a multiple of 64
        if (ok && lane == 0 && y0 < a.T && x0 < a.N) tc::tma_store_2d(&map_y, x0, y0, out);
        if (ok && j2 == 0 && row < a.T) a.hs[(size_t)row * a.nbh + n0 / 128] = bs.scale;
      }
    }
    if (lane < 2) tc::tma_store_wait_read();  // the grid's end waits for the writes
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // Both blocks' loads complete on the leading block's barrier.
      const CUtensorMap* mw = GATEUP && rank ? &map_w2 : &map_w;
      int g = 0;
      bool ok = true;
      for (int tile = first; tile < a.tiles && ok; tile += stride) {
        const int m0 = (tile % a.mt) * 256 + rank * BM, n0 = (tile / a.mt) * kN + (GATEUP ? 0 : rank * 128);
        for (int kb = 0; kb < nb; ++kb, ++g) {
          const int s = g % G::stages;
          if (g >= G::stages && !tc::bar_wait_warp(&b.empty[s], ((g / G::stages) - 1) & 1)) {
            if (lane == 0) pair_abort(b, a.flags);
            ok = false;
            break;
          }
          if (tc::elect_one()) {
            uint8_t* st = sm + (size_t)s * G::stage;
            const uint32_t full = tc::map_rank(tc::smem_addr(&b.full[s]), 0);
            if (rank == 0) tc::bar_expect_tx(&b.full[s], 2 * G::stage);
            tc::tma_load_2d_pair(st, &map_x, kb * BK, m0, full);
            tc::tma_load_2d_pair(st + kABytes, mw, kb * BK, n0, full);
          }
          __syncwarp();
        }
      }
      // After a wait that ran out, the loads still in flight land before the
      // block leaves: 2 ms, since no barrier of this block counts them.
      if (!ok) {
        const uint64_t t0 = tc::global_ns();
        for (int i = 0; i < 1000000 && tc::global_ns() - t0 < 2000000ull; ++i) {
        }
      }
    } else if (warp == 1) {
      if (rank == 0) {
        constexpr uint32_t idesc = tc::idesc_f16(256, 256);
        int g = 0;
        bool ok = true;
        for (int tile = first; tile < a.tiles && ok; tile += stride) {
          for (int kb = 0; kb < nb; ++kb, ++g) {
            const int s = g % G::stages, u = g % G::bufs;
            if ((g >= G::bufs && !tc::bar_wait_warp(&b.acc_empty[u], ((g / G::bufs) - 1) & 1)) ||
                !tc::bar_wait_warp(&b.full[s], (g / G::stages) & 1)) {
              if (lane == 0) pair_abort(b, a.flags);
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const uint32_t base = tc::smem_addr(sm + (size_t)s * G::stage);
            const uint64_t ad = tc::sw128_desc(base), bd = tc::sw128_desc(base + kABytes);
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < BK / 32; ++kk)
                tc::mma_f8_pair(tmem + (uint32_t)(u * 256), ad + 2 * kk, bd + 2 * kk, idesc, kk > 0);
              tc::mma_commit_pair(&b.empty[s]);
              tc::mma_commit_pair(&b.acc_full[u]);
            }
            __syncwarp();
          }
        }
      }
    } else if (warp < 4) {
      // Scales: the products xs * ws of a step, [2 weight blocks][128 tokens];
      // a group of four steps at a time, two tokens per lane. Up to two groups
      // ahead of the promotion, which hides the loads.
      const int r0 = (warp - 2) * 64 + lane;
      const bool vec = (nb & 3) == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15) == 0;
      float* sc = reinterpret_cast<float*>(sm + G::off_scale) + r0;
      int g = 0;
      bool ok = true;
      for (int tile = first; tile < a.tiles && ok; tile += stride) {
        const int m0 = (tile % a.mt) * 256 + rank * BM, n0 = (tile / a.mt) * kN;
        const float* pw0 = a.ws + (size_t)(n0 / 128) * nb;
        const float* pw1 = GATEUP ? a.ws2 + (size_t)(n0 / 128) * nb : (n0 + 128 < a.N ? pw0 + nb : nullptr);
        for (int kb = 0; kb < nb; kb += 4, ++g) {
          float x[2][4], w[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool live = m0 + r0 + 32 * i < a.T;
            const float* px = a.xs + (size_t)(m0 + r0 + 32 * i) * nb + kb;
            if (vec) {
              const float4 v = live ? *reinterpret_cast<const float4*>(px) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[i][e] = live && kb + e < nb ? px[e] : 0.0f;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[0][e] = kb + e < nb ? pw0[kb + e] : 0.0f;
            w[1][e] = pw1 && kb + e < nb ? pw1[kb + e] : 0.0f;
          }
          const int s = g % G::groups;
          if (g >= G::groups && !tc::bar_wait_warp(&b.sc_empty[s], ((g / G::groups) - 1) & 1)) {
            if (lane == 0) pair_abort(b, a.flags);
            ok = false;
            break;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) sc[((4 * s + e) * 2 + j) * BM + 32 * i] = x[i][e] * w[j][e];
          __syncwarp();
          if (lane == 0) tc::bar_arrive(&b.sc_full[s]);
        }
      }
    }
  }
  tc::tc_fence_before();
  __syncwarp();
  cluster_sync();  // neither block leaves while the other's MMAs, loads or arrivals can reach it
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc2(tmem, 512);
}

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }
inline int blocks128(int n) { return (n + 127) / 128; }

int code_map(CUtensorMap* m, const void* base, int K, int rows, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)K, (uint64_t)rows};
  const uint64_t str[1] = {(uint64_t)K};
  const uint32_t box[2] = {BK, (uint32_t)box_rows};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

struct Operand {
  const uint8_t* q;
  const float* s;
};

template <int NT, bool GATEUP>
int launch_gemm(GemmArgs a, const Operand& x, const Operand& w, const Operand* w2, int splits, int sms, int dev,
                cudaStream_t st) {
  using G = Geo<NT>;
  {
    static std::mutex mu;
    static bool set[kMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      MOE_CUDA_TRY(cudaFuncSetAttribute(fp8_gemm_kernel<NT, GATEUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)G::smem));
      set[dev] = true;
    }
  }
  int box = 8;  // rows of the token box: the batch's, rounded up
  while (box < BM && box < a.T) box *= 2;
  const int kn = GATEUP ? 128 : NT;
  a.a_bytes = (uint32_t)box * BK;
  a.xs = x.s;
  a.ws = w.s;
  a.ws2 = w2 ? w2->s : nullptr;
  a.nb = blocks128(a.K);
  a.mt = (a.T + BM - 1) / BM;
  a.tiles = a.mt * ((a.N + kn - 1) / kn);
  a.splits = splits;
  CUtensorMap mx, mw, mw2;
  int rc;
  if ((rc = code_map(&mx, x.q, a.K, a.T, box)) != MOE_OK) return rc;
  if ((rc = code_map(&mw, w.q, a.K, a.N, kn)) != MOE_OK) return rc;
  mw2 = mw;
  if (w2 && (rc = code_map(&mw2, w2->q, a.K, a.N, kn)) != MOE_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(splits > 1 ? a.tiles * splits : std::min(a.tiles, sms)));
  cfg.blockDim = dim3(G::threads);
  cfg.dynamicSmemBytes = G::smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (splits > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<NT, GATEUP>, mx, mw, mw2, a);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "fp8 product launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}

// The pair kernel: y or (hq, hs).
template <bool GATEUP>
int launch_pair(GemmArgs a, const Operand& x, const Operand& w, const Operand* w2, int sms, int dev, cudaStream_t st) {
  {
    static std::mutex mu;
    static bool set[kMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      MOE_CUDA_TRY(cudaFuncSetAttribute(fp8_pair_kernel<GATEUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)Pair::smem));
      set[dev] = true;
    }
  }
  const int kn = GATEUP ? 128 : 256;
  a.xs = x.s;
  a.ws = w.s;
  a.ws2 = w2 ? w2->s : nullptr;
  a.nb = blocks128(a.K);
  a.mt = (a.T + 255) / 256;
  a.tiles = a.mt * ((a.N + kn - 1) / kn);
  CUtensorMap mx, mw, mw2, my;
  int rc;
  if ((rc = code_map(&mx, x.q, a.K, a.T, BM)) != MOE_OK) return rc;
  if ((rc = code_map(&mw, w.q, a.K, a.N, 128)) != MOE_OK) return rc;
  mw2 = mw;
  if (w2 && (rc = code_map(&mw2, w2->q, a.K, a.N, 128)) != MOE_OK) return rc;
  my = mx;
  const uint64_t dims[2] = {(uint64_t)a.N, (uint64_t)a.T};
  if (GATEUP) {
    const uint64_t str[1] = {(uint64_t)a.N};
    const uint32_t box[2] = {64, 32};
    if ((rc = encode_tensor_map(&my, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.hq, dims, str, box,
                                CU_TENSOR_MAP_SWIZZLE_NONE)) != MOE_OK)
      return rc;
  } else if (a.N % 8 == 0) {
    const uint64_t str[1] = {(uint64_t)a.N * 2};
    const uint32_t box[2] = {64, 32};
    if ((rc = encode_tensor_map(&my, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.y, dims, str, box,
                                CU_TENSOR_MAP_SWIZZLE_128B)) != MOE_OK)
      return rc;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min(a.tiles, sms / 2)));
  cfg.blockDim = dim3(Pair::threads);
  cfg.dynamicSmemBytes = Pair::smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_pair_kernel<GATEUP>, mx, mw, mw2, my, a);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "fp8 product launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}

int product(const Operand& x, const Operand& w, int T, int N, int K, __half* y, int32_t* flags, cudaStream_t st) {
  if (T <= kGemvMaxTokens) return fp8_gemv(x.q, x.s, T, w.q, w.s, N, K, y, st);
  int dev = 0, sms = 0;
  const int rc = current_device_sms(&dev, &sms);
  if (rc != MOE_OK) return rc;
  GemmArgs a = {};
  a.T = T; a.N = N; a.K = K;
  a.y = y;
  a.flags = flags;
  const Plan p = plan_of(T, N, blocks128(K), sms, false);
  switch (p.nt) {
    case 0: return launch_pair<false>(a, x, w, nullptr, sms, dev, st);
    case 256: return launch_gemm<256, false>(a, x, w, nullptr, p.splits, sms, dev, st);
    case 128: return launch_gemm<128, false>(a, x, w, nullptr, p.splits, sms, dev, st);
    case 64: return launch_gemm<64, false>(a, x, w, nullptr, p.splits, sms, dev, st);
    default: return launch_gemm<32, false>(a, x, w, nullptr, p.splits, sms, dev, st);
  }
}

int gate_up(const Operand& x, const Operand& wg, const Operand& wu, int T, int Is, int H, uint8_t* hq, float* hs,
            int32_t* flags, cudaStream_t st) {
  int dev = 0, sms = 0;
  const int rc = current_device_sms(&dev, &sms);
  if (rc != MOE_OK) return rc;
  GemmArgs a = {};
  a.T = T; a.N = Is; a.K = H;
  a.hq = hq; a.hs = hs;
  a.nbh = blocks128(Is);
  a.flags = flags;
  const Plan p = plan_of(T, Is, blocks128(H), sms, true);
  if (p.nt == 0) return launch_pair<true>(a, x, wg, &wu, sms, dev, st);
  return launch_gemm<256, true>(a, x, wg, &wu, p.splits, sms, dev, st);
}

// Workspace of the FFN after the header: x and h as codes and scales, and for
// a few tokens h in FP32.
struct FfnWs {
  size_t xq, xs, hq, hs, hf, total;
};
FfnWs ffn_ws(int T, int H, int Is) {
  FfnWs w;
  size_t o = kWorkspaceHeader;
  w.xq = o; o += round256((size_t)T * H);
  w.xs = o; o += round256((size_t)T * blocks128(H) * 4);
  w.hq = o; o += round256((size_t)T * Is);
  w.hs = o; o += round256((size_t)T * blocks128(Is) * 4);
  // In every size, so that a workspace for T tokens serves fewer.
  w.hf = o; o += round256((size_t)std::min(T, kGemvMaxTokens) * Is * 4);
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
  return moe::product({static_cast<const uint8_t*>(xq), xs}, {static_cast<const uint8_t*>(wq), ws}, T, N, K,
                      static_cast<__half*>(y), static_cast<int32_t*>(workspace), static_cast<cudaStream_t>(stream));
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
  int32_t* flags = reinterpret_cast<int32_t*>(w8);
  uint8_t *xq = w8 + o.xq, *hq = w8 + o.hq;
  float *xs = reinterpret_cast<float*>(w8 + o.xs), *hs = reinterpret_cast<float*>(w8 + o.hs);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const moe::Operand g = {static_cast<const uint8_t*>(wg), sg}, u = {static_cast<const uint8_t*>(wu), su},
                     d = {static_cast<const uint8_t*>(wd), sd};
  if (T <= moe::kGemvMaxTokens)
    return moe::fp8_gemv_ffn(static_cast<const __half*>(x), T, H, Is, g.q, sg, u.q, su, d.q, sd, xq, xs, hq,
                             hs, reinterpret_cast<float*>(w8 + o.hf), static_cast<__half*>(y), st);
  int rc = moe::launch_quantize_fp8(static_cast<const __half*>(x), T, H, 1, xq, xs, st);
  if (rc != MOE_OK) return rc;
  if ((rc = moe::gate_up({xq, xs}, g, u, T, Is, H, hq, hs, flags, st)) != MOE_OK) return rc;
  return moe::product({hq, hs}, d, T, H, Is, static_cast<__half*>(y), flags, st);
}

}  // extern "C"
