// The append's rule at every token count near its borders: calls that are
// turned fit a grid, and the rule asks for at least 8 tokens a feature.
#include <stdio.h>

#include "aa_rules.h"

int main() {
  int checks = 0;
  const int64_t edges[] = {1, 64, 8 * 8, 8 * 128, 8 * 256, int64_t(1) << 30, (int64_t(1) << 31) - 1};
  for (const int64_t edge : edges)
    for (int64_t n = edge - 200; n <= edge + 200; ++n) {
      if (n < 1 || n >= int64_t(1) << 31) continue;
      for (int d = 8; d <= 256; d += 8) {
        ++checks;
        const bool turns = aa::append_turns(n, d);
        const int64_t threads = aa::append_turn_workgroups(n) * aa::kTurnThreads;
        if (turns && threads > aa::kMaxGridThreads) {
          fprintf(stderr, "%lld tokens, head dim %d: a grid of %lld threads\n", (long long)n, d, (long long)threads);
          return 1;
        }
        if (turns && n < 8 * d) return fprintf(stderr, "%lld tokens of %d turned\n", (long long)n, d), 1;
        if (!turns && n >= 8 * d && n < (int64_t(1) << 30) - aa::kTurnTokens)
          return fprintf(stderr, "%lld tokens of %d not turned\n", (long long)n, d), 1;
      }
    }
  printf("append rule holds: %d\n", checks);
  return 0;
}
