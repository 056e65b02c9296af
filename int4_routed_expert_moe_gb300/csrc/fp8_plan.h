// Which kernel and tile a block-scaled FP8 product of more than 16 tokens runs
// on (see fp8_gemm.cu). Host code alone: a test compiles it by itself.
#pragma once

#include <algorithm>

namespace moe {

constexpr int kPlanTokens = 128;  // tokens per tile of a block
constexpr int kMaxSplits = 8;     // portable cluster size

// The kernel a product runs on: pairs (nt = 0), or single blocks with tiles of
// nt columns and the K steps of a tile split over a cluster.
struct Plan {
  int nt, splits;
};
// The cheapest by a model of the time (us), fitted to runs of every choice at
// 17 to 512 tokens against 4096 x 2048, 2048 x 4096, 1001 x 2064, 512 x 1024
// and 8192 x 8192 (us measured by choice, e.g. 64 tokens, 4096 x 2048: nt/splits
// 128/4 6.1, 64/2 6.3, 32/1 6.9, 128/2 7.4, 256/4 8.1; 512 tokens, 8192 x 8192:
// pairs 28.9, 256/1 35, 128/1 51):
//   single blocks: 3.2 to start and end; a step takes 0.235 (barriers, issue) or
//   what its bytes need at 68 GB/ms per SM; joining a split costs 0.5 and
//   0.0125 per column;
//   pairs: 4.2 to start and end, 0.38 per step, 1.5 per tile after the first
//   (gate/up 2.0: SiLU and the quantisation). The products' runs alone were
//   fitted; gate/up takes their terms and that one of its own.
inline Plan plan_of(int T, int N, int nb, int sms, bool gateup) {
  const int mt = (T + kPlanTokens - 1) / kPlanTokens, kn_pair = gateup ? 128 : 256;
  const int pair_tiles = ((T + 255) / 256) * ((N + kn_pair - 1) / kn_pair);
  const int pair_waves = (pair_tiles + sms / 2 - 1) / (sms / 2);
  const float per_tile = gateup ? 2.0f : 1.5f;
  Plan best = {0, 1};
  float t_best = 4.2f + (float)pair_waves * (0.38f * (float)nb + per_tile) - per_tile;
  const float a_bytes = 128.0f * (float)std::min(T, kPlanTokens);
  for (int nt = gateup ? 256 : 32; nt <= 256; nt *= 2) {
    const int kn = gateup ? 128 : nt, tiles = mt * ((N + kn - 1) / kn);
    const float step = std::max(0.235f, (128.0f * (float)nt + a_bytes) / 68000.0f);
    for (int s = 1; s <= kMaxSplits && s <= nb; s *= 2) {
      // A split tile's blocks start together: about sms / 2 blocks fit in
      // clusters of eight at a time, 9/10 of the SMs in clusters of four.
      if (s > 1 && (long long)tiles * s > (s == 8 ? sms / 2 : s == 4 ? sms * 9 / 10 : sms)) break;
      const int steps = (nb + s - 1) / s;
      const int waves = (tiles + sms - 1) / sms;
      const float t = 3.2f + (float)waves * (float)steps * step + (s > 1 ? 0.5f + 0.0125f * (float)nt : 0.0f) +
                      (float)(waves - 1) * per_tile +
                      (s == 1 && !gateup && N % 8 ? (float)waves * 0.03f * (float)nt : 0.0f);  // scattered 2-byte stores
      if (t < t_best) {
        t_best = t;
        best = {nt, s};
      }
    }
  }
  return best;
}

}  // namespace moe
