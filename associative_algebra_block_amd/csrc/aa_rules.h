// Rules by which the launchers choose a kernel from a call's sizes, as plain
// host functions: the launchers and the CPU tests of the rules share them.
#pragma once

#include <stdint.h>

namespace aa {

// An HSA dispatch counts the threads of a grid dimension in 32 bits.
constexpr int64_t kMaxGridThreads = (int64_t(1) << 32) - 1;

// The append that turns values in LDS: tokens and threads of a workgroup.
constexpr int kTurnTokens = 64, kTurnThreads = 256;
inline int64_t append_turn_workgroups(int64_t n) { return (n + kTurnTokens - 1) / kTurnTokens; }

// Whether n tokens are turned.  From 8 D tokens on the turning surely repays its
// waits: with 8 bf16 heads of 128 and pages of 64, 512, 1024, 4096 and 40000 tokens
// of a prompt take 5.6, 8.8, 26 and 408 us one by one and 4.7, 5.0, 8.3 and 69
// turned; with 32 float32 heads of 24, 128, 256 and 1024 take 3.3, 4.1, 9.2 and
// 3.3, 3.4, 3.8.  Calls of more threads than a grid holds go one by one.
inline bool append_turns(int64_t n, int head_dim) {
  return n >= 8 * int64_t(head_dim) && append_turn_workgroups(n) * kTurnThreads <= kMaxGridThreads;
}

// The kernels of a mixture-of-experts call: waves per 16-column strip of gate and
// up (kMoeUpWaves a workgroup, up_parts workgroups a pair, pairs in rows of eight
// or one a row), and strips and waves a workgroup of the down projection.
constexpr int kMoeUpWaves = 8;
struct MoeRule {
  int up_waves;
  uint32_t up_parts;
  bool rows_of_eight;
  int down_strips, down_waves;
};
inline MoeRule moe_rule(bool q2xq2, int q, int64_t D, int64_t F, int top_k, int64_t M) {
  MoeRule r;
  const uint64_t pairs = uint64_t(M) * uint64_t(top_k), strips = uint64_t(F / 16);
  const int groups = q2xq2 ? 4 : q < 2 ? q : 2;   // of a leaf, at most
  // Waves a strip: as many as repay their join.  Measured (us of the whole call)
  // with 1, 2, 4 and 8, for sums of 8 steps of 32 rows (q = 16, 2048 -> 768) at 384
  // strips 13.5, 12.5, 12.2, 13.2; at 768 14.3, 13.7, 14.7, 15.6; at 1536 16.2, 16.5,
  // 17.2, 22.3.  For 16 and more steps (Q2 x Q2, 768 -> 2048) at 256 strips 18.5,
  // 15.5, 14.4, 13.4; at 1280 20.8, 19.9, 18.6, 20.9; at 5120 36.0, 33.3, 39.1, 51.1;
  // at 10240 47.5, 52.4, 64.4, 89.8.
  const bool long_sums = groups * (D / q) >= 16 * 32;
  const uint64_t all_strips = pairs * strips;
  r.up_waves = long_sums && all_strips <= 256 ? 8 : all_strips <= (long_sums ? 1536 : 512) ? 4
               : all_strips <= (long_sums ? 8192 : 1024) ? 2 : 1;
  r.up_parts = uint32_t((strips * r.up_waves + kMoeUpWaves - 1) / kMoeUpWaves);
  r.rows_of_eight = r.up_parts % 8 && pairs >= 16;
  // Two strips a workgroup, which share the hidden activation's loads, where there
  // are enough of them, else one, with four or, for long sums, sixteen waves:
  // (2 strips x 8 waves, 1 x 4, 1 x 16) take for 1, 5, 10 and 20 tokens of Q2 x Q2
  // experts (48, 240, 480, 960 strips, 128 steps) 14.9, 15.3, 13.4; 20.7, 20.5, 18.6;
  // 24.7, 26.5, 27.4; 33.3, 35.8, 41.7 us; for 2 and 16 tokens of q = 16, 2048 -> 768
  // (256, 2048 strips, 32 steps) 14.0, 13.9, 15.5 and 31.2, 32.4, 59.5.  Short sums
  // of very many strips do with four waves: 32 tokens (4096 strips) 50.8 and 52.3.
  // Workgroups of 16 waves are one on each of the 256 units, so more of them take
  // two turns: q = 2, 640 -> 1440, 7 tokens (280 strips, 276 steps) 39.8 us, 2 x 8 35.1.
  const int64_t steps = top_k * int64_t(groups) * ((F / q + 31) / 32);
  const uint64_t all_out = uint64_t(M) * uint64_t(D / 16);
  if (all_out >= 1536 && steps <= 64) r.down_strips = 2, r.down_waves = 4;
  else if (all_out >= 400 || (steps > 64 && all_out > 256)) r.down_strips = 2, r.down_waves = 8;
  else r.down_strips = 1, r.down_waves = steps <= 64 ? 4 : 16;
  return r;
}

}  // namespace aa
