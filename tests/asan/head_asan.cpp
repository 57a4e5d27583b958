// Host AddressSanitizer and UndefinedBehaviorSanitizer driver for the output layer's losses (test infrastructure): every
// refusal of their entry points, and the workspace plan with its range choosers over the whole range of sizes, ends
// included.  Nothing here reaches a kernel launch.  Built and run by tests/test_head_asan_cpu.py.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "head.h"
#include "qlora.h"

static int g_fail = 0;
#define EXPECT(call, want)                                                                               \
  do {                                                                                                   \
    const int rc_ = (call);                                                                              \
    if (rc_ != (want)) {                                                                                 \
      printf("line %d: %s returned %d, expected %d (%s)\n", __LINE__, #call, rc_, (want), qlora_last_error()); \
      g_fail = 1;                                                                                        \
    }                                                                                                    \
  } while (0)
#define HOLDS(cond)                                                                                      \
  do {                                                                                                   \
    if (!(cond)) {                                                                                       \
      printf("line %d: %s fails at T=%lld V=%lld K=%lld\n", __LINE__, #cond, (long long)T, (long long)V, (long long)K); \
      g_fail = 1;                                                                                        \
    }                                                                                                    \
  } while (0)

// Of one size: the plan's choices and its bytes, against what the parts must hold.
static void plan(int64_t T, int64_t V, int64_t K) {
  const int tr = qlora::head_tile_rows(T, V);
  HOLDS(tr == 64 || tr == 128 || tr == 256);
  if (T > 0) {
    const int s = qlora::head_logit_ranges(T, V, K, tr);
    HOLDS(s >= 1 && s <= 16 && s <= (K + 127) / 128);
    const int64_t fours = (K + 127) / 128, per = (fours + s - 1) / s;
    HOLDS((s - 1) * per < fours);  // no range is empty
  }
  const int d = qlora::head_dw_ranges(T, V, K, 1);
  HOLDS(d >= 1 && d <= 256 && (d == 1 || d <= (T + 127) / 128));
  HOLDS(qlora::head_dw_ranges(T, V, K, 2) == 1);
  for (int64_t n = 0; n <= T; n = n < 3 ? n + 1 : n * 3 + 7) {
    const int per = qlora::head_dw_steps((int)n, d);
    HOLDS(per >= 1 && (int64_t)per * 128 * d >= n);
  }
  for (int dx = 0; dx < 2; ++dx)
    for (int dw = 0; dw < 2; ++dw) {
      size_t one = 0, most = 0;
      EXPECT(qlora_head_workspace_bytes(T, V, K, 0, dx, dw, &one), QLORA_OK);
      EXPECT(qlora_head_workspace_bytes(T, V, K, QLORA_MAX_TARGETS, dx, dw, &most), QLORA_OK);
      HOLDS(most >= one && one >= (size_t)T * K * 2 + (size_t)T * 12);
    }
}

int main() {
  void *F = (void *)0x10000;  // aligned, never dereferenced: each call below fails before using it
  char *M = (char *)F + 8, *O = (char *)F + 2;  // misaligned
  qlora_bf16 *b = (qlora_bf16 *)F;
  float *f = (float *)F;
  int64_t *y = (int64_t *)F;
  int32_t *x = (int32_t *)F;
  const size_t big = (size_t)1 << 62;

  EXPECT(qlora_head_ce(b, -1, b, 100, 64, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 0, 64, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 60, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, INT64_MAX, b, 100, 64, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, INT64_MIN, b, 100, 64, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, INT64_MAX, 64, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, INT64_MAX - 7, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 1 << 21, 1 << 14, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(nullptr, 8, b, 100, 64, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, nullptr, 100, 64, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, nullptr, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, y, f, nullptr, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce((qlora_bf16 *)M, 8, b, 100, 64, y, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, (int64_t *)O, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, y, (float *)O, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, y, f, f, (qlora_bf16 *)M, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, y, f, f, b, (qlora_bf16 *)M, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, y, f, f, b, b, M, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, y, f, f, b, b, nullptr, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_ce(b, 8, b, 100, 64, y, f, f, b, b, F, 0, nullptr), QLORA_EWORKSPACE);
  EXPECT(qlora_head_distill(b, 8, b, 100, 64, x, f, 0, 1.f, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_distill(b, 8, b, 100, 64, x, f, INT32_MAX, 1.f, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_distill(b, 8, b, 100, 64, x, f, 4, 0.f, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_distill(b, 8, b, 100, 64, nullptr, f, 4, 1.f, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_distill(b, 8, b, 100, 64, x, (float *)O, 4, 1.f, f, f, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_distill(b, 8, b, 100, 64, x, f, 4, 1.f, f, f, b, b, F, 0, nullptr), QLORA_EWORKSPACE);
  size_t n = 0;
  EXPECT(qlora_head_workspace_bytes(8, 100, 64, 0, 1, 1, nullptr), QLORA_EINVAL);
  EXPECT(qlora_head_workspace_bytes(8, 100, 64, INT32_MIN, 1, 1, &n), QLORA_EINVAL);
  EXPECT(qlora_head_workspace_bytes(INT64_MAX, INT64_MAX, INT64_MAX - 7, 0, 1, 1, &n), QLORA_EINVAL);

  const int64_t top = (int64_t)1 << 22;
  const int64_t Ts[] = {0, 1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1001, 4096, 32768, 32769, 100000, top - 1, top};
  const int64_t Vs[] = {1, 2, 63, 64, 127, 128, 129, 255, 256, 257, 1000, 32000, 50257, 128256, 1048577, top - 1, top};
  const int64_t Ks[] = {8, 16, 120, 128, 136, 1024, 2056, 4096, 8192, 65536, top - 8, top};
  int plans = 0;
  for (int64_t T : Ts)
    for (int64_t V : Vs)
      for (int64_t K : Ks) {
        const bool fits = V * K <= (int64_t)1 << 34 && T * K < (int64_t)1 << 31;
        EXPECT(qlora_head_workspace_bytes(T, V, K, 0, 0, 0, &n), fits ? QLORA_OK : QLORA_EINVAL);
        if (fits) plan(T, V, K), ++plans;
      }
  printf("%d plans\n", plans);
  printf(g_fail ? "head asan driver FAILED\n" : "head asan driver ok\n");
  return g_fail;
}
