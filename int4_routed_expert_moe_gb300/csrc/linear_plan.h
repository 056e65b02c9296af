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
// The cheapest by a model of the time (us); nb: steps of 64 along K.
inline LinearPlan linear_plan(int T, int N, int nb, int sms) {
  const int mt = (T + kLinearTokens - 1) / kLinearTokens;
  const int pair_tiles = ((T + 255) / 256) * ((N + 255) / 256);
  const int pair_waves = (pair_tiles + sms / 2 - 1) / (sms / 2);
  const float per_tile = 0.5f;
  LinearPlan best = {0, 1};
  float t_best = 5.0f + (float)pair_waves * (0.38f * (float)nb + per_tile);
  const float a_bytes = 128.0f * (float)std::min(T, kLinearTokens);
  for (int nt = 32; nt <= 128; nt *= 2) {
    const int tiles = mt * ((N + nt - 1) / nt);
    const float step = std::max(0.2f, (128.0f * (float)nt + a_bytes) / 68000.0f);
    for (int s = 1; s <= kLinearMaxSplits && s <= nb; s *= 2) {
      if (s > 1 && (long long)tiles * s > (s == 8 ? sms / 2 : s == 4 ? sms * 9 / 10 : sms)) break;
      const int steps = (nb + s - 1) / s, waves = (tiles + sms - 1) / sms;
      const float t = 3.2f + (float)waves * ((float)steps * step + per_tile) + (s > 1 ? 0.5f + 0.0125f * (float)nt : 0.0f);
      if (t < t_best) {
        t_best = t;
        best = {nt, s};
      }
    }
  }
  return best;
}

}  // namespace moe
