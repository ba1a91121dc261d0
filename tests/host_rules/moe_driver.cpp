// Prints, for each "q2xq2 q D F top_k M" of the standard input, the kernels that
// the rule takes: waves a strip of gate and up, pairs in rows of eight, strips
// and waves of the down projection, and whether a last strip is alone.
#include <stdio.h>

#include "aa_rules.h"

int main() {
  int law, q, k;
  long long D, F, M;
  while (scanf("%d %d %lld %lld %d %lld", &law, &q, &D, &F, &k, &M) == 6) {
    const aa::MoeRule r = aa::moe_rule(law != 0, q, D, F, k, M);
    printf("%d %d %d %d %d\n", r.up_waves, int(r.rows_of_eight), r.down_strips, r.down_waves,
           int(D / q / 16 % r.down_strips != 0));
  }
  return 0;
}
