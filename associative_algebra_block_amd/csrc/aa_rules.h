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

// Whether n tokens are turned.  From about 8 D tokens on the turning repays its
// waits: with 8 heads of 128 and pages of 64, 512, 1024, 4096 and 40000 tokens of
// a prompt take 5.6, 8.7, 26 and 524 us one by one and 7.3, 7.7, 10.3 and 96
// turned; with 32 heads of 24, 128, 256 and 1024 take 3.3, 4.1, 8.4 and 3.9, 3.9,
// 4.6.  Calls of more threads than a grid holds go one by one.
inline bool append_turns(int64_t n, int head_dim) {
  return n >= 8 * int64_t(head_dim) && append_turn_workgroups(n) * kTurnThreads <= kMaxGridThreads;
}

}  // namespace aa
