// The in-place forms of the LayerNorm entry points (S = X, dX = dS) with
// stand-in launchers, and overlaps beside them that stay refused.
#include <stdint.h>
#include <stdio.h>

#include "aa.h"

template <typename T = void>
static T* P(uint64_t k) { return reinterpret_cast<T*>(k << 40); }

static int wrong = 0;
static void expect(aa_status_t got, aa_status_t want, const char* what) {
  if (got == want) return;
  ++wrong;
  fprintf(stderr, "%s: got %s, want %s (%s)\n", what, aa_status_string(got), aa_status_string(want), aa_last_error());
}

int main() {
  float *g = P<float>(3), *b = P<float>(4), *mu = P<float>(7), *r = P<float>(8);
  const auto fwd = [&](void* S, void* Y) {
    return aa_layernorm_fwd(P(1), P(2), g, b, S, Y, mu, r, 8, 768, 1e-5f, AA_F32, AA_BF16, AA_BF16, nullptr);
  };
  expect(fwd(P(5), P(6)), AA_OK, "S of its own");
  expect(fwd(P(1), P(6)), AA_OK, "S = X");
  expect(fwd(P(1), P(1)), AA_ERR_INVALID_ARG, "Y = S = X");
  expect(fwd(P<char>(1) + 16, P(6)), AA_ERR_INVALID_ARG, "S beside X's start");
  const auto bwd = [&](const void* dS, void* dX) {
    return aa_layernorm_bwd(P(1), P(2), g, mu, r, dS, dX, nullptr, nullptr, 8, 768, AA_F32, AA_BF16, nullptr, 0, nullptr);
  };
  expect(bwd(P(9), P(10)), AA_OK, "dX of its own");
  expect(bwd(P(9), P(9)), AA_OK, "dX = dS");
  expect(bwd(P(9), P(2)), AA_ERR_INVALID_ARG, "dX = dY");
  expect(bwd(P(9), P<char>(9) + 16), AA_ERR_INVALID_ARG, "dX beside dS's start");
  if (!wrong) printf("in-place calls passed\n");
  return wrong != 0;
}
