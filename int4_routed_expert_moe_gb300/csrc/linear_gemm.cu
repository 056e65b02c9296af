// y = act(x W^T + bias) + residual on the tensor cores, more than 16 tokens.
//
// Tokens are the MMA's M, rows of W its N. Both operands come by TMA in the
// 128-byte-swizzled K-major layout, in steps of 64 columns (128 bytes), and a
// tile's sums stay in tensor memory until its last step; a second accumulator
// takes the next tile meanwhile. A pipeline stage holds one, two or four steps:
// waiting, handing over and committing cost some 0.2 us each time, more than
// the MMAs of a step of a narrow tile (64 tokens, 2048 x 2048 in tiles of 64
// columns, us: one step per stage 12.0, two 9.5, four 8.3).
//
// linear_gemm_kernel: a block and 128 tokens by NT columns, the K steps of a
// tile split over a cluster where the tiles are few. linear_pair_kernel: two
// blocks and 256 x 256 or 256 x 128. linear_plan picks.
#include <algorithm>
#include <mutex>

#include "common.h"
#include "device.cuh"
#include "kernels.h"
#include "linear.cuh"
#include "linear_plan.h"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int BM = kLinearTokens;
constexpr int BK = 64;
constexpr uint32_t kABytes = BM * BK * 2;
// An accumulator takes 8 steps (512 of K) for FP32 results, 64 (4096) for FP16.
// The tensor cores cut the running sum off every 16 terms, by 3.5 2^-24 of it on
// average, and the errors add up along K: a router's logits over K = 2048 are
// 2.3e-6 off when one accumulator takes all of K (with segments 6.4e-7), and terms
// of one sign, whose cuts all go one way, 7080 2^-24 over K = 65536 (58 and 440),
// nearly as much as FP16's rounding, 2^-11.
constexpr int kSegment = 8;
constexpr int kSegment16 = 64;

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
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(tc::map_rank(a, rank))
               : "memory");
  return v;
}

struct TileArgs {
  int nb;            // steps along K
  int seg;           // steps that one accumulator takes
  int mt, nt, tiles; // token tiles, tiles along N, in all
  int group;         // pair kernel: token tiles walked together along N
  int splits;        // blocks of a cluster share one tile's steps
  uint32_t a_bytes;  // bytes of the token tile's box
  bool y_tma, r_tma; // pair kernel: rows of y / the residual that TMA can address
};

// A block of these kernels takes more than half of an SM's shared memory, and so
// do the library's other kernels with tensor memory: no two are on an SM at
// once, whatever streams they come from. With two there, the blocks of two
// clusters could each hold the columns that the other waits for.
constexpr size_t kSmShared = 228 * 1024;

// Geometry by tile width. Warp 0 issues TMA, warp 1 owns tensor memory and
// issues the MMAs, the others run the epilogue.
template <int NT>
struct Geo {
  static constexpr int epi = NT >= 128 ? 8 : 4;
  static constexpr int cols = NT / (epi / 4);  // per epilogue warp
  static constexpr int threads = 64 + 32 * epi;
  static constexpr int kb = NT == 128 ? 2 : 4;  // steps per stage
  static_assert(kSegment % kb == 0 && kSegment16 % kb == 0, "a segment is whole stages");
  static constexpr uint32_t step = kABytes + (uint32_t)NT * BK * 2, stage = kb * step;
  static constexpr int stages = NT == 128 ? 3 : 2;
  static constexpr uint32_t tmem_cols = 2 * NT;
  static constexpr uint32_t off_ctrl = (uint32_t)stages * stage;
  static constexpr size_t smem = (size_t)off_ctrl + 1024 + 1024;  // control block, alignment
  static_assert(2 * smem > kSmShared, "no second block with tensor memory on the SM");
  static constexpr int red_pitch = NT + 4;                        // floats per row of a partial tile
  static_assert((size_t)BM * red_pitch * 4 <= off_ctrl, "partial tile fits the stage area");
};

struct Bars {
  uint64_t *full, *empty, *acc_full, *acc_empty, *res;
  uint32_t* tmem_slot;
  int* abort;
};
__device__ __forceinline__ Bars bars_at(uint8_t* p, int stages) {
  Bars b;
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  b.full = q; q += stages;
  b.empty = q; q += stages;
  b.acc_full = q; q += 2;
  b.acc_empty = q; q += 2;
  b.res = q; q += 8;
  b.tmem_slot = reinterpret_cast<uint32_t*>(q);
  b.abort = reinterpret_cast<int*>(b.tmem_slot + 1);
  return b;
}
__device__ __forceinline__ bool is_aborted(const Bars& b) { return *reinterpret_cast<volatile int*>(b.abort) != 0; }
__device__ __forceinline__ void set_aborted(const Bars& b, int32_t* flags) {
  atomicOr(flags, 4);
  *reinterpret_cast<volatile int*>(b.abort) = 1;
}
// Bounded wait by every lane of a warp, one verdict; it ends early once another
// role of the block has given up.
__device__ __forceinline__ bool wait(const Bars& b, uint64_t* bar, uint32_t parity, int32_t* flags) {
  bool ok = tc::bar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = tc::global_ns();
    while (!(ok = tc::bar_try_wait(bar, parity))) {
      if (is_aborted(b)) break;
      if (tc::global_ns() - t0 > tc::kWaitNs) {
        set_aborted(b, flags);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// SEG: a tile's steps go into the accumulators in segments, whose sums the
// epilogue warps add in registers.
template <int NT, bool SEG>
__global__ void __launch_bounds__(Geo<NT>::threads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const LinearArgs a, const TileArgs ta) {
  using G = Geo<NT>;
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = tc::align1024(smraw);
  const Bars b = bars_at(sm + G::off_ctrl, G::stages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_w);
    for (int s = 0; s < G::stages; ++s) {
      tc::bar_init(&b.full[s], 1);
      tc::bar_init(&b.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::bar_init(&b.acc_full[s], 1);
      tc::bar_init(&b.acc_empty[s], G::epi);
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

  const int S = ta.splits;
  const int rank = S > 1 ? (int)cluster_rank() : 0;
  const int kb0 = ta.nb * rank / S, kb1 = ta.nb * (rank + 1) / S;
  const int first = (int)blockIdx.x / S, stride = (int)gridDim.x / S;

  if (warp == 0) {
    int g = 0;
    bool ok = true;
    for (int tile = first; tile < ta.tiles && ok; tile += stride) {
      const int m0 = (tile % ta.mt) * BM, n0 = (tile / ta.mt) * NT;
      for (int kb = kb0; kb < kb1; kb += G::kb, ++g) {
        const int s = g % G::stages, n = min(G::kb, kb1 - kb);
        if (g >= G::stages && !(ok = wait(b, &b.empty[s], ((g / G::stages) - 1) & 1, a.flags))) break;
        if (tc::elect_one()) {
          uint8_t* st = sm + (size_t)s * G::stage;
          tc::bar_expect_tx(&b.full[s], (uint32_t)n * (ta.a_bytes + NT * BK * 2));
          for (int i = 0; i < n; ++i) {
            tc::tma_load_2d(st + i * G::step, &map_x, (kb + i) * BK, m0, &b.full[s]);
            tc::tma_load_2d(st + i * G::step + kABytes, &map_w, (kb + i) * BK, n0, &b.full[s]);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0)  // loads still in flight land before the block leaves (bounded)
      for (int i = g > G::stages ? g - G::stages : 0; i < g; ++i)
        tc::bar_wait(&b.full[i % G::stages], (i / G::stages) & 1);
  } else if (warp == 1) {
    constexpr uint32_t idesc = tc::idesc_f16(BM, NT);
    int g = 0, u = 0;
    bool ok = true;
    for (int tile = first; tile < ta.tiles && ok; tile += stride) {
      for (int kb = kb0, e = 0; kb < kb1; kb += G::kb, ++g) {  // e: step of the segment
        const int s = g % G::stages, n = min(G::kb, kb1 - kb);
        if (e == 0 && u >= 2 && !(ok = wait(b, &b.acc_empty[u & 1], ((u >> 1) - 1) & 1, a.flags))) break;
        if (!(ok = wait(b, &b.full[s], (g / G::stages) & 1, a.flags))) break;
        tc::tc_fence_after();
        const uint32_t base = tc::smem_addr(sm + (size_t)s * G::stage);
        const uint64_t ad = tc::sw128_desc(base), bd = tc::sw128_desc(base + kABytes);
        const bool end = e + n >= ta.seg || kb + n >= kb1;
        if (tc::elect_one()) {
#pragma unroll
          for (int i = 0; i < G::kb; ++i)
            if (i < n)
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                tc::mma_f16(tmem + (uint32_t)((u & 1) * NT), ad + i * (G::step >> 4) + 2 * kk,
                            bd + i * (G::step >> 4) + 2 * kk, idesc, e > 0 || i > 0 || kk > 0);
          tc::mma_commit(&b.empty[s]);
          if (end) tc::mma_commit(&b.acc_full[u & 1]);
        }
        __syncwarp();
        e += n;
        if (end) {
          e = 0;
          ++u;
        }
      }
    }
  } else {
    const int q4 = warp & 3, c0 = G::cols * ((warp - 2) >> 2);
    const uint32_t tl = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)c0;
    int u = 0;
    for (int tile = first; tile < ta.tiles; tile += stride, ++u) {
      const int m0 = (tile % ta.mt) * BM, n0 = (tile / ta.mt) * NT;
      const int r = 32 * q4 + lane, row = m0 + r;
      float sum[SEG ? G::cols : 1] = {};
      if constexpr (SEG) {
        bool ok = true;
        for (int left = kb1 - kb0; left > ta.seg; left -= ta.seg, ++u) {
          if (!(ok = wait(b, &b.acc_full[u & 1], (u >> 1) & 1, a.flags))) break;
          tc::tc_fence_after();
#pragma unroll
          for (int c = 0; c < G::cols; c += 32) {
            uint32_t d[32];
            tc::tmem_ld32(tl + (uint32_t)((u & 1) * NT + c), d);
            tc::tmem_ld32_wait(d);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c + i] += __uint_as_float(d[i]);
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(&b.acc_empty[u & 1]);
        }
        if (!ok) break;
      }
      if (!wait(b, &b.acc_full[u & 1], (u >> 1) & 1, a.flags)) break;
      tc::tc_fence_after();
      if (S > 1) {  // partial tile to shared memory (every stage has been consumed)
        float* red = reinterpret_cast<float*>(sm) + (size_t)r * G::red_pitch + c0;
#pragma unroll
        for (int c = 0; c < G::cols; c += 32) {
          uint32_t d[32];
          __syncwarp();
          tc::tmem_ld32(tl + (uint32_t)((u & 1) * NT + c), d);
          tc::tmem_ld32_wait(d);
          if (row < a.T) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(d[i + e]) + (SEG ? sum[SEG ? c + i + e : 0] : 0.0f);
              *reinterpret_cast<float4*>(red + c + i) = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        break;
      }
#pragma unroll
      for (int c = 0; c < G::cols; c += 32) {
        uint32_t d[32];
        __syncwarp();
        tc::tmem_ld32(tl + (uint32_t)((u & 1) * NT + c), d);
        tc::tmem_ld32_wait(d);
        if (c + 32 == G::cols) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(&b.acc_empty[u & 1]);
        }
        if (row < a.T) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(d[i]) + (SEG ? sum[SEG ? c + i : 0] : 0.0f);
          finish(a, row, n0 + c0 + c, v);
        }
      }
    }
  }
  if (S > 1) {
    // The cluster's partial tiles, added in rank order (the same order every
    // time), each block finishing its share of the tile.
    __syncwarp();
    cluster_sync();
    const int m0 = (first % ta.mt) * BM, n0 = (first / ta.mt) * NT;
    const int rows = min(BM, a.T - m0);
    const uint32_t red = tc::smem_addr(sm);
    constexpr int kQ = NT / 8;  // pieces of 8 columns per row
    for (int i = rank * G::threads + (int)threadIdx.x; i < rows * kQ; i += S * G::threads) {
      const int r = i / kQ, c = (i % kQ) * 8;
      if (n0 + c >= a.N) continue;
      float v[8] = {};
      for (int p = 0; p < S; ++p) {
        const uint32_t at = red + (uint32_t)(r * G::red_pitch + c) * 4;
        const float4 f = ld_cluster(at, (uint32_t)p), h = ld_cluster(at + 16, (uint32_t)p);
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
        v[4] += h.x; v[5] += h.y; v[6] += h.z; v[7] += h.w;
      }
      finish(a, m0 + r, n0 + c, v);
    }
    __syncwarp();
    cluster_sync();  // nobody leaves while its partial tile is read
  }
  tc::gemm_teardown(tmem, G::tmem_cols);
}

// ---- SM pairs: 256 tokens by 256 or 128 rows of W ----------------------------
// Two blocks of a cluster run one tile with cta_group::2 MMAs: each holds its
// 128 tokens (A) and half of the weight rows (B), and each accumulates its
// tokens against all rows. Warps: 0 TMA, 1 tensor memory and (in the leading
// block) MMA issue, 4-11 epilogue (a lane quarter, half of the columns each).
//
// Measured: 8192 x 8192 x 4096, FP16 out, 292 us (1.88 PFLOP/s, 98 % of the
// measured BF16 rate; the tensor pipe is active 96 % of the SMs' time); with
// bias, SiLU and residual 311 us, 92 %: the epilogue's passes through shared
// memory take bandwidth from the MMAs' operands, which need all of it. Under
// sustained load the power limit takes them to 335 and 360 us (cuBLAS without
// epilogue 285 and 328). FP32 out 318 us: 268 MB more to write. 16 tiles of
// tokens go along N together (kGroup), us: 4 318, 8 308, 16 303, 32 (all) 324:
// the tiles in flight then read 43 MB, which stays in L2.
constexpr int kGroup = 16;
template <int NT>
struct Pair {
  static constexpr int epi = 8, threads = 384;
  static constexpr int cols = NT / 2;  // per epilogue warp
  static constexpr int kb = NT == 256 ? 1 : 2;  // steps per stage (256: two 3 % slower, 128: one 17 % slower)
  static_assert(kSegment % kb == 0 && kSegment16 % kb == 0, "a segment is whole stages");
  static constexpr uint32_t step = kABytes + (uint32_t)(NT / 2) * BK * 2, stage = kb * step;
  static constexpr int stages = NT == 256 ? 6 : 4;
  static constexpr uint32_t tmem_cols = 2 * NT;
  static constexpr uint32_t off_out = stages * stage;  // [epi][32 rows][128 bytes]
  static constexpr uint32_t off_ctrl = off_out + epi * 4096;
  static constexpr size_t smem = (size_t)off_ctrl + 1024 + 1024;
  static_assert(smem <= 232448, "shared memory of a block");
  static_assert(2 * smem > kSmShared, "no second block with tensor memory on the SM");
};

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// 16 bytes of an epilogue warp's staging area: 32 rows of 128 bytes in the
// 128-byte swizzle, 64 FP16 columns (chunk c: 32 of them) or 32 FP32 columns.
template <typename Y>
__device__ __forceinline__ uint8_t* piece(uint8_t* out, int c, int lane, int i) {
  return out + tc::sw128_offset(lane, (sizeof(Y) == 2 ? 4 * c : 0) + i);
}

// Tile number to (token tile, tile along N): `group` token tiles go along N
// together, so that the tiles in flight share few rows of both operands.
__device__ __forceinline__ void place(const TileArgs& t, int tile, int& m, int& n) {
  const int g = tile / (t.group * t.nt), r = tile - g * t.group * t.nt;
  const int wide = min(t.group, t.mt - g * t.group);
  m = g * t.group + r % wide;
  n = r / wide;
}

template <typename Y, int NT, bool SEG>
__global__ void __launch_bounds__(Pair<NT>::threads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_r,
                       const LinearArgs a, const TileArgs ta) {
  using G = Pair<NT>;
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = tc::align1024(smraw);
  const Bars b = bars_at(sm + G::off_ctrl, G::stages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_w);
    tc::tma_prefetch_desc(&map_y);
    tc::tma_prefetch_desc(&map_r);
    for (int s = 0; s < G::stages; ++s) {
      tc::bar_init(&b.full[s], 1);
      tc::bar_init(&b.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::bar_init(&b.acc_full[s], 1);
      tc::bar_init(&b.acc_empty[s], 2 * G::epi);
    }
    for (int s = 0; s < G::epi; ++s) tc::bar_init(&b.res[s], 1);
    *b.abort = 0;
    tc::bar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc2(b.tmem_slot, G::tmem_cols);
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = *b.tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const int nb = ta.nb;
  const int first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
  // Sums of segments in registers, 128 of them with 256 columns (a thread spills 32
  // to 40 bytes). 384 x 168 registers at launch = 128 x 72 + 256 x 216.
  constexpr bool kSplitRegs = SEG && NT == 256;
  if (kSplitRegs && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0) {
    // Both blocks' loads complete on the leading block's barrier.
    int g = 0;
    bool ok = true;
    for (int tile = first; tile < ta.tiles && ok; tile += stride) {
      int m0, n0;
      place(ta, tile, m0, n0);
      m0 = m0 * 256 + rank * BM;
      n0 = n0 * NT + rank * (NT / 2);
      for (int kb = 0; kb < nb; kb += G::kb, ++g) {
        const int s = g % G::stages, n = min(G::kb, nb - kb);
        if (g >= G::stages && !(ok = wait(b, &b.empty[s], ((g / G::stages) - 1) & 1, a.flags))) break;
        if (tc::elect_one()) {
          uint8_t* st = sm + (size_t)s * G::stage;
          const uint32_t full = tc::map_rank(tc::smem_addr(&b.full[s]), 0);
          if (rank == 0) tc::bar_expect_tx(&b.full[s], (uint32_t)n * 2 * G::step);
          for (int i = 0; i < n; ++i) {
            tc::tma_load_2d_pair(st + i * G::step, &map_x, (kb + i) * BK, m0, full);
            tc::tma_load_2d_pair(st + i * G::step + kABytes, &map_w, (kb + i) * BK, n0, full);
          }
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
      constexpr uint32_t idesc = tc::idesc_f16(256, NT);
      int g = 0, u = 0;
      bool ok = true;
      for (int tile = first; tile < ta.tiles && ok; tile += stride) {
        for (int kb = 0, e = 0; kb < nb; kb += G::kb, ++g) {  // e: step of the segment
          const int s = g % G::stages, n = min(G::kb, nb - kb);
          if (e == 0 && u >= 2 && !(ok = wait(b, &b.acc_empty[u & 1], ((u >> 1) - 1) & 1, a.flags))) break;
          if (!(ok = wait(b, &b.full[s], (g / G::stages) & 1, a.flags))) break;
          tc::tc_fence_after();
          const uint32_t base = tc::smem_addr(sm + (size_t)s * G::stage);
          const uint64_t ad = tc::sw128_desc(base), bd = tc::sw128_desc(base + kABytes);
          const bool end = e + n >= ta.seg || kb + n >= nb;
          if (tc::elect_one()) {
#pragma unroll
            for (int i = 0; i < G::kb; ++i)
              if (i < n)
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk)
                  mma_f16_pair(tmem + (uint32_t)((u & 1) * NT), ad + i * (G::step >> 4) + 2 * kk,
                               bd + i * (G::step >> 4) + 2 * kk, idesc, e > 0 || i > 0 || kk > 0);
            tc::mma_commit_pair(&b.empty[s]);
            if (end) tc::mma_commit_pair(&b.acc_full[u & 1]);
          }
          __syncwarp();
          e += n;
          if (end) {
            e = 0;
            ++u;
          }
        }
      }
    }
  } else if (warp >= 4) {
    if constexpr (kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    constexpr int kBox = 128 / (int)sizeof(Y);                  // columns per staged row
    constexpr int kPass = kBox, kChunks = kPass / 32;           // columns and chunks per staging pass
    const int q4 = warp & 3, e8 = warp - 4, j2 = e8 >> 2;
    const uint32_t tl = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(G::cols * j2);
    const uint32_t acc_empty0 = tc::map_rank(tc::smem_addr(&b.acc_empty[0]), 0);
    uint8_t* out = sm + G::off_out + e8 * 4096;
    int u = 0, loads = 0;
    for (int tile = first; tile < ta.tiles; tile += stride, ++u) {
      int y0, x0;
      place(ta, tile, y0, x0);
      y0 = y0 * 256 + rank * BM + 32 * q4;
      x0 = x0 * NT + G::cols * j2;
      const int row = y0 + lane;
      float sum[SEG ? G::cols : 1] = {};
      if constexpr (SEG) {
        for (int left = nb; left > ta.seg; left -= ta.seg, ++u) {
          wait(b, &b.acc_full[u & 1], (u >> 1) & 1, a.flags);  // given up: the stores below are left out
          tc::tc_fence_after();
#pragma unroll
          for (int c = 0; c < G::cols; c += 32) {
            uint32_t d[32];
            tc::tmem_ld32(tl + (uint32_t)((u & 1) * NT + c), d);
            tc::tmem_ld32_wait(d);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c + i] += __uint_as_float(d[i]);
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::bar_arrive_cluster(acc_empty0 + 8 * (u & 1));
        }
      }
      bool got = false;
#pragma unroll (SEG ? G::cols / kPass : 1)
      for (int p = 0; p < G::cols / kPass; ++p) {
        const int xp = x0 + p * kPass;
        // The stores of the last pass have read the staging area; the
        // residual's tile comes into it, and the results take its place.
        if (lane == 0) tc::tma_store_wait_read();
        __syncwarp();
        const bool some = y0 < a.T && xp < a.N, load = some && ta.r_tma;
        if (load) {
          if (lane == 0) {
            tc::fence_async_smem();
            tc::bar_expect_tx(&b.res[e8], 4096u);
            tc::tma_load_2d(out, &map_r, xp, y0, &b.res[e8]);
          }
          __syncwarp();
        }
        if (!got) got = wait(b, &b.acc_full[u & 1], (u >> 1) & 1, a.flags);
        tc::tc_fence_after();
        if (load && !wait(b, &b.res[e8], loads++ & 1, a.flags)) got = false;
        const bool last = p == G::cols / kPass - 1;
#pragma unroll (SEG ? kChunks : 1)
        for (int c = 0; c < kChunks; ++c) {
          uint32_t d[32];
          __syncwarp();
          tc::tmem_ld32(tl + (uint32_t)((u & 1) * NT + p * kPass + 32 * c), d);
          tc::tmem_ld32_wait(d);
          if (last && c == kChunks - 1) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive_cluster(acc_empty0 + 8 * (u & 1));
          }
          const int n = xp + 32 * c;
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(d[i]) + (SEG ? sum[SEG ? p * kPass + 32 * c + i : 0] : 0.0f);
          if (a.bias) add_bias(a, n, v);
          activate<sizeof(Y) == 2>(a.act, v);
          if (a.residual && !ta.r_tma && row < a.T) {
            const Y* r = static_cast<const Y*>(a.residual) + (size_t)row * (size_t)a.ldr + n;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n + i < a.N) v[i] += (float)r[i];
          }
          if (sizeof(Y) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4* s = reinterpret_cast<uint4*>(piece<Y>(out, c, lane, i));
              if (load) {
                const uint4 q = *s;
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 f = __half22float2(u32_as_h2(w[e]));
                  v[8 * i + 2 * e] += f.x;
                  v[8 * i + 2 * e + 1] += f.y;
                }
              }
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const half2 f = __floats2half2_rn(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]);
                h[e] = *reinterpret_cast<const uint32_t*>(&f);
              }
              *s = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float4* s = reinterpret_cast<float4*>(piece<Y>(out, c, lane, i));
              float4 f = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
              if (load) {
                const float4 q = *s;
                f.x += q.x; f.y += q.y; f.z += q.z; f.w += q.w;
              }
              *s = f;
            }
          }
        }
        if (!got || is_aborted(b)) continue;
        if (ta.y_tma) {
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0 && some) tc::tma_store_2d(&map_y, xp, y0, out);
        } else {
          // Rows that TMA cannot address (pitch no multiple of 16 bytes): one element per lane.
          __syncwarp();
          for (int rr = 0; rr < min(32, a.T - y0); ++rr)
#pragma unroll
            for (int j = 0; j < kPass / 32; ++j) {
              const int x = 32 * j + lane, col = x * (int)sizeof(Y);
              const Y v = *reinterpret_cast<const Y*>(out + tc::sw128_offset(rr, col >> 4) + (col & 15));
              if (xp + x < a.N) static_cast<Y*>(a.y)[(size_t)(y0 + rr) * (size_t)a.ldy + xp + x] = v;
            }
          __syncwarp();
        }
      }
    }
    if (lane == 0) tc::tma_store_wait_read();  // the grid's end waits for the writes
  }
  tc::tc_fence_before();
  __syncwarp();
  cluster_sync();  // neither block leaves while the other's MMAs, loads or arrivals can reach it
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc2(tmem, G::tmem_cols);
}

// A row-major matrix [rows][cols], rows ld elements apart, in boxes of 128-byte rows.
int row_map(CUtensorMap* m, const void* base, bool f32, int cols, int rows, long long ld, int box_rows) {
  const int esz = f32 ? 4 : 2;
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t str[1] = {(uint64_t)ld * esz};
  const uint32_t box[2] = {128u / esz, (uint32_t)box_rows};
  return encode_tensor_map(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dims, str,
                           box, CU_TENSOR_MAP_SWIZZLE_128B);
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Launch(unsigned grid, int threads, size_t smem, int cluster, cudaStream_t st) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
};

template <int NT, bool SEG>
int launch_gemm(const LinearArgs& a, int splits, int sms, int dev, cudaStream_t st) {
  using G = Geo<NT>;
  static std::mutex mu;
  static bool set[kMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      MOE_CUDA_TRY(cudaFuncSetAttribute(linear_gemm_kernel<NT, SEG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::smem));
      set[dev] = true;
    }
  }
  int box = 8;  // rows of the token box: the batch's, rounded up
  while (box < BM && box < a.T) box *= 2;
  TileArgs t = {};
  t.nb = (a.K + BK - 1) / BK;
  t.seg = !SEG ? t.nb : a.y32 ? kSegment : kSegment16;
  t.mt = (a.T + BM - 1) / BM;
  t.tiles = t.mt * ((a.N + NT - 1) / NT);
  t.splits = splits;
  t.a_bytes = (uint32_t)box * BK * 2;
  CUtensorMap mx, mw;
  int rc;
  if ((rc = row_map(&mx, a.x, false, a.K, a.T, a.ldx, box)) != MOE_OK) return rc;
  if ((rc = row_map(&mw, a.w, false, a.K, a.N, a.K, NT)) != MOE_OK) return rc;
  const Launch l((unsigned)(splits > 1 ? t.tiles * splits : std::min(t.tiles, sms)), G::threads, G::smem, splits, st);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, linear_gemm_kernel<NT, SEG>, mx, mw, a, t);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "moe_linear launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}

// Whether a tile's sum is taken in segments.
bool segments(const LinearArgs& a) { return a.y32 || a.K > kSegment16 * BK; }

template <int NT>
int launch_gemm(const LinearArgs& a, int splits, int sms, int dev, cudaStream_t st) {
  return segments(a) ? launch_gemm<NT, true>(a, splits, sms, dev, st) : launch_gemm<NT, false>(a, splits, sms, dev, st);
}

template <typename Y, int NT, bool SEG>
int launch_pair(const LinearArgs& a, int sms, int dev, cudaStream_t st) {
  static std::mutex mu;
  static bool set[kMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      MOE_CUDA_TRY(cudaFuncSetAttribute(linear_pair_kernel<Y, NT, SEG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)Pair<NT>::smem));
      // The register split must not ask for more than the block is launched with: it would wait forever.
      cudaFuncAttributes fa;
      MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, linear_pair_kernel<Y, NT, SEG>));
      if (SEG && NT == 256 && fa.numRegs * Pair<NT>::threads < 128 * 72 + 256 * 216)
        return fail(MOE_ERR_UNSUPPORTED, "moe_linear: the pair kernel was built with %d registers per thread", fa.numRegs);
      set[dev] = true;
    }
  }
  constexpr bool f32 = sizeof(Y) == 4;
  TileArgs t = {};
  t.nb = (a.K + BK - 1) / BK;
  t.seg = !SEG ? t.nb : f32 ? kSegment : kSegment16;
  t.mt = (a.T + 255) / 256;
  t.nt = (a.N + NT - 1) / NT;
  t.tiles = t.mt * t.nt;
  t.group = kGroup;
  t.splits = 1;
  // A store is cut off at N in steps of 16 bytes: what it wrote past N would
  // not be left as it was.
  t.y_tma = a.ldy * (long long)sizeof(Y) % 16 == 0 && a.N * sizeof(Y) % 16 == 0;
  t.r_tma = a.residual && a.ldr * (long long)sizeof(Y) % 16 == 0;
  CUtensorMap mx, mw, my, mr;
  int rc;
  if ((rc = row_map(&mx, a.x, false, a.K, a.T, a.ldx, BM)) != MOE_OK) return rc;
  if ((rc = row_map(&mw, a.w, false, a.K, a.N, a.K, NT / 2)) != MOE_OK) return rc;
  my = mr = mx;
  if (t.y_tma && (rc = row_map(&my, a.y, f32, a.N, a.T, a.ldy, 32)) != MOE_OK) return rc;
  if (t.r_tma && (rc = row_map(&mr, a.residual, f32, a.N, a.T, a.ldr, 32)) != MOE_OK) return rc;
  const Launch l((unsigned)(2 * std::min(t.tiles, sms / 2)), Pair<NT>::threads, Pair<NT>::smem, 2, st);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, linear_pair_kernel<Y, NT, SEG>, mx, mw, my, mr, a, t);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "moe_linear launch: %s", cudaGetErrorString(e));
  return MOE_OK;
}

template <int NT>
int launch_pair(const LinearArgs& a, int sms, int dev, cudaStream_t st) {
  if (a.y32) return launch_pair<float, NT, true>(a, sms, dev, st);
  return segments(a) ? launch_pair<__half, NT, true>(a, sms, dev, st) : launch_pair<__half, NT, false>(a, sms, dev, st);
}

int launch_plan(const LinearArgs& a, const LinearPlan& p, int sms, int dev, cudaStream_t st) {
  if (p.pair) return p.nt == 256 ? launch_pair<256>(a, sms, dev, st) : launch_pair<128>(a, sms, dev, st);
  switch (p.nt) {
    case 128: return launch_gemm<128>(a, p.splits, sms, dev, st);
    case 64: return launch_gemm<64>(a, p.splits, sms, dev, st);
    default: return launch_gemm<32>(a, p.splits, sms, dev, st);
  }
}

}  // namespace

int linear_gemm(const LinearArgs& a, cudaStream_t st) {
  int dev = 0, sms = 0;
  const int rc = current_device_sms(&dev, &sms);
  if (rc != MOE_OK) return rc;
  return launch_plan(a, linear_plan(a.T, a.N, (a.K + BK - 1) / BK, sms), sms, dev, st);
}

}  // namespace moe
