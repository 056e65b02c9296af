// Which kernel and tile the FP16 product of more than 16 tokens runs on (see
// linear_gemm.cu). Host code alone: a test compiles it by itself.
#pragma once

#include <algorithm>

namespace moe {

constexpr int kLinearTokens = 128;     // tokens per tile of a block
constexpr int kLinearMaxSplits = 8;    // portable cluster size

// Pairs (nt = 0), or single blocks with tiles of nt columns and the K steps of
// a tile split over a cluster.
struct LinearPlan {
  int nt, splits;
};
// The cheapest by a model of the time (us); nb: steps of 64 along K. Fitted to
// runs of every choice at 13 batch sizes from 17 to 8192 against 12 matrices
// from 64 x 2048 to 8192 x 8192 (us measured by choice, e.g. 64 tokens, 2048 x
// 2048: 64/4 7.3, 32/2 8.4, 64/1 12.0, pairs 13.7; 1000 tokens, 8192 x 8192:
// pairs 79, 128/1 133); over them its choice is 0.7 % slower than the best:
//   single blocks: 4.05 to start and end; a step takes its barriers and MMAs
//   (0.21 to 0.28), or what its bytes need at 113 GB/ms per SM and 14.4 GB/ms
//   in all; joining a split costs 0.5, 0.076 per block and 0.018 per column of
//   a full tile; outputs stored one by one (N odd) 0.11 per column;
//   pairs: 4.7 to start and end, 0.3 per step, 1.16 at least per tile.
inline LinearPlan linear_plan(int T, int N, int nb, int sms) {
  const int mt = (T + kLinearTokens - 1) / kLinearTokens;
  const int pair_tiles = ((T + 255) / 256) * ((N + 255) / 256);
  const int pair_waves = (pair_tiles + sms / 2 - 1) / (sms / 2);
  LinearPlan best = {0, 1};
  float t_best = 4.7f + (float)pair_waves * std::max(0.3f * (float)nb, 1.16f);
  const float rows = (float)std::min(T, kLinearTokens), full = rows / (float)kLinearTokens;
  for (int nt = 32; nt <= 128; nt *= 2) {
    const int tiles = mt * ((N + nt - 1) / nt);
    const float bytes = 128.0f * ((float)nt + rows);
    const float least = nt == 32 ? 0.21f : nt == 64 ? 0.26f : 0.28f;
    for (int s = 1; s <= kLinearMaxSplits && s <= nb; s *= 2) {
      // A split tile's blocks start together: about sms / 2 blocks fit in
      // clusters of eight at a time, 9/10 of the SMs in clusters of four.
      if (s > 1 && (long long)tiles * s > (s == 8 ? sms / 2 : s == 4 ? sms * 9 / 10 : sms)) break;
      const int steps = (nb + s - 1) / s, waves = (tiles + sms - 1) / sms;
      const float blocks = (float)std::min((long long)tiles * s, (long long)sms);
      const float step = std::max(least, std::max(bytes / 113000.0f, blocks * bytes / 14.4e6f));
      const float t = 4.05f + (float)(waves * steps) * step + 0.44f * (float)(waves - 1) +
                      (s > 1 ? 0.5f + 0.076f * (float)s + 0.018f * (float)nt * full : 0.0f) +
                      (s == 1 && N % 8 ? (float)waves * 0.11f * (float)std::min(nt, N) * full : 0.0f);
      if (t < t_best) {
        t_best = t;
        best = {nt, s};
      }
    }
  }
  return best;
}

}  // namespace moe
