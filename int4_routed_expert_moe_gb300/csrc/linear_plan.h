// Which kernel and tile the FP16 product of more than 16 tokens runs on (see
// linear_gemm.cu). Host code alone: a test compiles it by itself.
#pragma once

#include <algorithm>

namespace moe {

constexpr int kLinearTokens = 128;     // tokens per tile of a block
constexpr int kLinearMaxSplits = 8;    // portable cluster size

// Tiles of nt columns, on pairs of SMs (256 tokens) or on single blocks (128
// tokens) that share a tile's K steps in a cluster of `splits`.
struct LinearPlan {
  bool pair;
  int nt, splits;
};
// The cheapest by a model of the time (us); nb: steps of 64 along K. Fitted to
// runs of every choice, FP16 results, operands in L2 from the run before, at 13
// batch sizes from 17 to 8192 against 12 matrices from 64 x 2048 to 8192 x 8192
// (us measured by choice, e.g. 64 tokens, 2048 x 2048: 64/4 6.6, 32/1 7.2, 128/4
// 7.5, pairs 13.8 and 8.6; 8192 tokens, 256 x 2048: pairs of 128 columns 10.4,
// 128/1 12.6, 64/1 16.0, pairs of 256 16.0); over them its choice is 0.5 % slower
// than the best. x from memory and FP32 results take longer (the last pairs of 128
// columns 13.0 with FP32 results and a bias, 14.9 with x from memory too):
//   single blocks: 3.75 to start and end; a step takes its barriers and MMAs
//   (0.113 to 0.23), or what its bytes need at 153 GB/ms per SM and 20.7 GB/ms
//   in all; joining a split costs 0.37, 0.15 per block and 0.02 per column of a
//   full tile; outputs stored one by one (N odd) 0.13 per column;
//   pairs: 5.0 (256 columns) and 3.55 (128) to start and end, 0.279 and 0.185 per
//   step, 1.45 and 0.83 at least per tile.
inline LinearPlan linear_plan(int T, int N, int nb, int sms) {
  LinearPlan best = {true, 256, 1};
  float t_best = 0.0f;
  for (int nt = 256; nt >= 128; nt /= 2) {
    const int tiles = ((T + 255) / 256) * ((N + nt - 1) / nt), waves = (tiles + sms / 2 - 1) / (sms / 2);
    const float t = nt == 256 ? 5.0f + (float)waves * std::max(0.279f * (float)nb, 1.45f)
                              : 3.55f + (float)waves * std::max(0.185f * (float)nb, 0.83f);
    if (nt == 256 || t < t_best) {
      t_best = t;
      best.nt = nt;
    }
  }
  const int mt = (T + kLinearTokens - 1) / kLinearTokens;
  const float rows = (float)std::min(T, kLinearTokens), full = rows / (float)kLinearTokens;
  for (int nt = 32; nt <= 128; nt *= 2) {
    const int tiles = mt * ((N + nt - 1) / nt);
    const float bytes = 128.0f * ((float)nt + rows);
    const float least = nt == 32 ? 0.113f : nt == 64 ? 0.145f : 0.23f;
    for (int s = 1; s <= kLinearMaxSplits && s <= nb; s *= 2) {
      // A split tile's blocks start together: about sms / 2 blocks fit in
      // clusters of eight at a time, 9/10 of the SMs in clusters of four.
      if (s > 1 && (long long)tiles * s > (s == 8 ? sms / 2 : s == 4 ? sms * 9 / 10 : sms)) break;
      const int steps = (nb + s - 1) / s, waves = (tiles + sms - 1) / sms;
      const float blocks = (float)std::min((long long)tiles * s, (long long)sms);
      const float step = std::max(least, std::max(bytes / 153000.0f, blocks * bytes / 20.7e6f));
      const float t = 3.75f + (float)(waves * steps) * step + 0.52f * (float)(waves - 1) +
                      (s > 1 ? 0.37f + 0.15f * (float)s + 0.02f * (float)nt * full : 0.0f) +
                      (s == 1 && N % 8 ? (float)waves * 0.13f * (float)std::min(nt, N) * full : 0.0f);
      if (t < t_best) {
        t_best = t;
        best = {false, nt, s};
      }
    }
  }
  return best;
}

}  // namespace moe
