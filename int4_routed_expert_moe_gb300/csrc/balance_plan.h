// How the balance loss shares a batch out (see balance.cu). Host code alone: a
// test compiles it by itself.
#pragma once

#include <algorithm>

namespace moe {

constexpr int kMinChunk = 32;  // tokens
// Threads of a block by the values a lane holds, so that its registers suffice
// (1024 threads spill: 32768 x 256 19.4 us against 17.1; backward with 32 values and
// 16-byte loads 12 to 16 bytes of a thread do), and chunks at most: what fills the
// 152 SMs of a GB300 once, with two blocks per SM backward.
constexpr int threads_of(int nv) { return nv == 8 ? 768 : nv == 16 ? 512 : 256; }
constexpr int back_threads_of(int nv) { return nv == 32 ? 256 : 512; }
constexpr int max_chunks(int E) { return E > 512 ? 304 : 152; }  // not decreasing in E
constexpr int back_chunks(int E) { return E > 256 && E <= 512 ? 152 : 304; }
// A batch of up to 3 rounds of a block's tokens and 16 sequences is one chunk,
// and so one block: 256 tokens of 64 experts 6.4 us, 1024 in 32 chunks 9.3.
constexpr int kAloneRounds = 3;
constexpr int kAloneSequences = 16;
constexpr int kFusedRows = 40960;  // chunks times experts that one launch joins

// Lanes that share a token, and the values of each.
constexpr int lanes_of(int E) { return E <= 64 ? 8 : E <= 128 ? 16 : 32; }
constexpr int values_of(int E) { return E <= 256 ? 8 : E <= 512 ? 16 : 32; }
// Sequences that a block takes at a time.
constexpr int sequences_of(int lanes, int values) { return 1024 / (lanes * values); }

struct BalancePlan {
  int chunk, chunks;  // tokens per block, blocks
  bool fused;         // forward: one launch
};
inline BalancePlan balance_plan(int T, int E, int S, bool back) {
  BalancePlan p;
  const int most = back ? back_chunks(E) : max_chunks(E);
  p.chunk = std::max(kMinChunk, (T + most - 1) / most);
  if (!back && S <= kAloneSequences) {
    const int groups = threads_of(values_of(E)) / lanes_of(E);
    if (T <= kAloneRounds * groups) p.chunk = kAloneRounds * groups;
  }
  p.chunks = std::max(1, (T + p.chunk - 1) / p.chunk);
  p.fused = p.chunks * E <= kFusedRows;
  return p;
}

}  // namespace moe
