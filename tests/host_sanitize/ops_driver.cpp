// Drives the LayerNorm, paged-attention and mixture-of-experts entry points
// through their host checks with stand-in launchers (ops_stub_launch.cpp),
// under AddressSanitizer and UndefinedBehaviorSanitizer: sizes at the limits
// (products near 2^63), absent operands, overlaps.  Device pointers are plain
// addresses that nothing dereferences.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "aa.h"

namespace aa {
extern int g_launches;
}

static int g_checks = 0;

static void expect(aa_status_t got, aa_status_t want, int launched, int want_launched, const char* what, int line) {
  ++g_checks;
  if (got != want || launched != want_launched || (want != AA_OK && aa_last_error()[0] == '\0')) {
    fprintf(stderr, "line %d: %s: got %s (%d launched), want %s (%s)\n", line, what, aa_status_string(got), launched,
            aa_status_string(want), aa_last_error());
    exit(1);
  }
}
#define EXPECT(call, want, launches)                                                       \
  do {                                                                                     \
    const int before = aa::g_launches;                                                     \
    const aa_status_t st = (call);                                                         \
    expect(st, want, aa::g_launches - before, launches, #call, __LINE__);                  \
  } while (0)

template <typename T = void>
static T* P(uint64_t k) { return reinterpret_cast<T*>(k << 40); }

int main() {
  float *g = P<float>(3), *b = P<float>(4), *mu = P<float>(7), *r = P<float>(8);
  const int64_t big = (int64_t(1) << 31) - 1;
  EXPECT(aa_layernorm_fwd(P(1), P(2), g, b, P(5), P(6), mu, r, 8, 768, 1e-5f, AA_F32, AA_BF16, AA_BF16, nullptr), AA_OK, 1);
  EXPECT(aa_layernorm_fwd(P(1), P(2), g, b, P(1), P(600), mu, r, big, 16384, 0.0f, AA_BF16, AA_BF16, AA_F32, nullptr),
         AA_ERR_INVALID_ARG, 0);   // rows so many that X runs into the others
  EXPECT(aa_layernorm_fwd(P(1), nullptr, nullptr, nullptr, nullptr, P(600), nullptr, nullptr, big, 16384, 0.0f, AA_F32,
                          AA_F32, AA_F32, nullptr), AA_OK, 1);
  EXPECT(aa_layernorm_fwd(P(1), nullptr, g, b, P(5), P(6), mu, r, 8, 768, 1e-5f, AA_F32, AA_BF16, AA_BF16, nullptr),
         AA_ERR_INVALID_ARG, 0);
  EXPECT(aa_layernorm_fwd(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 1, 0.0f, AA_F32,
                          AA_F32, AA_F32, nullptr), AA_OK, 0);
  size_t n = 0;
  EXPECT(aa_layernorm_bwd_workspace(8, 768, &n), AA_OK, 0);
  EXPECT(aa_layernorm_bwd(P(1), P(2), g, mu, r, nullptr, P(9), P<float>(10), P<float>(11), 8, 768, AA_F32, AA_BF16,
                          P(12), n, nullptr), AA_OK, 1);
  EXPECT(aa_layernorm_bwd(P(1), P(2), g, mu, r, P(9), P(9), nullptr, nullptr, 8, 768, AA_F32, AA_BF16, nullptr, 0,
                          nullptr), AA_OK, 1);
  EXPECT(aa_layernorm_bwd(P(1), P(2), g, mu, r, nullptr, P(9), P<float>(10), nullptr, 8, 768, AA_F32, AA_BF16, P(12),
                          n - 1, nullptr), AA_ERR_INVALID_ARG, 0);
  EXPECT(aa_layernorm_bwd(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, P<float>(10), P<float>(11), 0,
                          768, AA_F32, AA_BF16, nullptr, 0, nullptr), AA_OK, 1);   // writes zeros

  const int32_t *table = P<int32_t>(5), *pos = P<int32_t>(6), *len = P<int32_t>(6);
  EXPECT(aa_kv_append(P(1), P(2), 1024, 2048, AA_F32, P(3), P(4), 100, 64, 8, 128, table, 3, 10, nullptr, pos, 3,
                      nullptr), AA_OK, 1);
  EXPECT(aa_kv_append(P(1), P(2), big, big, AA_F32, P(3), P(1 << 22), big, 4096, 1024, 256, table, big, big, P<int32_t>(9),
                      pos, big, nullptr), AA_ERR_INVALID_ARG, 0);   // a cache larger than the address space leaves
  EXPECT(aa_kv_append(P(1), P(2), 1024, 1024, AA_F32, P(3), P(4), 100, 64, 8, 128, table, 3, 10, nullptr, pos, 4,
                      nullptr), AA_ERR_SHAPE, 0);
  EXPECT(aa_attn_decode_workspace(3, 32, 8, 128, 64, 1000, &n), AA_OK, 0);
  EXPECT(aa_attn_decode(P(1), 4096, AA_BF16, P(3), P(4), 100, 64, 32, 8, 128, table, 3, 1000, len, 0.1f, P(7), AA_F32,
                        P(8), n, nullptr), AA_OK, 1);
  EXPECT(aa_attn_decode(P(1), 4096, AA_BF16, P(3), P(4), 100, 64, 32, 8, 128, table, 3, 1000, len, 0.1f, P(7), AA_F32,
                        P(8), n - 1, nullptr), AA_ERR_INVALID_ARG, 0);
  EXPECT(aa_attn_decode(P(1), 4096, AA_BF16, P(3), P(4), 100, 64, 32, 8, 128, table, big, 1000, len, 0.1f, P(7), AA_F32,
                        P(8), n, nullptr), AA_ERR_UNSUPPORTED, 0);

  aa_plan_t up = nullptr, down = nullptr;
  EXPECT(aa_plan_create(&up, AA_LAW_QQ, 16, 2048, 768, AA_TYPES_POS_MOD, 0, AA_BF16, AA_BF16), AA_OK, 0);
  EXPECT(aa_plan_create(&down, AA_LAW_QQ, 16, 768, 2048, AA_TYPES_POS_MOD, 0, AA_BF16, AA_F32), AA_OK, 0);
  EXPECT(aa_moe_ffn_workspace(up, down, 128, 8, 16, &n), AA_OK, 0);
  EXPECT(aa_moe_ffn_fwd(up, down, P(1), P(2), 128, 8, 1, P(3), P(4), P(5), P(6), nullptr, nullptr, 16, INT64_MAX, nullptr,
                        P(9), n, nullptr), AA_OK, 1);
  EXPECT(aa_moe_ffn_fwd(up, down, P(1), P(2), 128, 8, 1, P(3), P(4), P(5), P(6), P<int32_t>(7), P<float>(8), 16, 0,
                        nullptr, P(9), n - 1, nullptr), AA_ERR_INVALID_ARG, 0);
  EXPECT(aa_moe_ffn_fwd(up, down, P(1), P(2), 128, 8, 1, P(3), P(4), P(5), P(6), nullptr, nullptr, INT64_MAX, 0, nullptr,
                        P(9), n, nullptr), AA_ERR_UNSUPPORTED, 0);
  EXPECT(aa_plan_destroy(up), AA_OK, 0);
  EXPECT(aa_plan_destroy(down), AA_OK, 0);
  printf("host checks passed: %d\n", g_checks);
  return 0;
}
