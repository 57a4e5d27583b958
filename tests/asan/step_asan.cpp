// Host AddressSanitizer and UndefinedBehaviorSanitizer driver for the embedding, the layer norm and the adapters by token
// (test infrastructure): every refusal of their entry points, and the workspace plans with their choosers over the whole
// range of sizes, ends included.  Nothing here reaches a kernel launch.  Built and run by tests/test_step_asan_cpu.py.
#include <stdint.h>
#include <stdio.h>

#include "qlora.h"
#include "step.h"

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
      printf("line %d: %s fails at T=%lld %lld x %lld\n", __LINE__, #cond, (long long)T, (long long)K, (long long)N); \
      g_fail = 1;                                                                                        \
    }                                                                                                    \
  } while (0)

// Of one size: the plans' choices and their bytes, against what the parts must hold.
static void plan(int64_t T, int64_t K, int64_t N, int32_t pool, int32_t r) {
  for (int64_t n : {K, N}) {
    const int s = qlora::adapt_ranges(T, pool, r, n);
    HOLDS(s >= 1 && s <= 8 && s <= (n + 511) / 512);
    size_t e = 0;
    EXPECT(qlora_embed_workspace_bytes(T, n, &e), QLORA_OK);
    const int piece = qlora::embed_piece(T);
    HOLDS(piece >= 1 && piece <= 32);
    const int64_t pieces = (T + piece - 1) / piece;
    HOLDS(e >= (size_t)T * 8 + (pieces > 1 ? (size_t)pieces * 2 * n * 4 : 0));
    if (n <= qlora::kNormMax) {
      size_t b = 0;
      EXPECT(qlora_layer_norm_workspace_bytes(T, n, &b), QLORA_OK);
      const int groups = qlora::norm_bwd_groups(T, n);
      HOLDS(groups >= 1 && groups <= 256 && b == (size_t)groups * 2 * n * 4);
    }
  }
  const int piece = qlora::adapt_piece(T, K, N);
  HOLDS(piece >= 128 && piece <= 1024 && (T > 512 || piece == 512));
  // groups cut into pieces have room: two groups a token longer than a piece, and one group of all tokens
  const int64_t slots = qlora::adapt_slots(T, piece);
  HOLDS(T <= piece || slots >= (T + piece - 1) / piece);
  HOLDS(T < 2 * (piece + 1) || slots >= 4);
  size_t f = 0, b = 0;
  EXPECT(qlora_adapters_workspace_bytes(T, K, N, pool, r, 0, &f), QLORA_OK);
  EXPECT(qlora_adapters_workspace_bytes(T, K, N, pool, r, 1, &b), QLORA_OK);
  HOLDS(f >= (size_t)T * 4 + (size_t)T * r * 4 && b >= f + (size_t)pool * r * (K + N) * 2 + (size_t)slots * r * (K + N) * 4);
}

int main() {
  void *F = (void *)0x10000;  // aligned, never dereferenced: each call below fails before using it
  char *M = (char *)F + 8, *O = (char *)F + 2;  // misaligned
  qlora_bf16 *b = (qlora_bf16 *)F, *m = (qlora_bf16 *)M;
  float *f = (float *)F;
  int64_t *y = (int64_t *)F;
  int32_t *x = (int32_t *)F;
  const size_t big = (size_t)1 << 62;
  size_t n = 0;

  EXPECT(qlora_embed(y, INT64_MIN, b, 100, 64, 1.f, b, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed(y, 8, b, INT64_MAX, 64, 1.f, b, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed(y, 8, b, 100, INT64_MAX - 7, 1.f, b, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed(nullptr, 8, b, 100, 64, 1.f, b, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed(y, 8, m, 100, 64, 1.f, b, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed(y, 8, b, 100, 64, 1.f, nullptr, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed_bwd((int64_t *)O, b, 8, 100, 64, 1.f, 0, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed_bwd(y, b, INT64_MAX, 100, 64, 1.f, 0, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed_bwd(y, b, 8, 100, 64, 1.f, 0, nullptr, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed_bwd(y, b, 8, 100, 64, 1.f, 1, b, M, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed_bwd(y, b, 8, 100, 64, 1.f, 1, b, F, 0, nullptr), QLORA_EWORKSPACE);
  EXPECT(qlora_embed_workspace_bytes(8, 64, nullptr), QLORA_EINVAL);
  EXPECT(qlora_embed_workspace_bytes(INT64_MAX, INT64_MAX, &n), QLORA_EINVAL);

  EXPECT(qlora_layer_norm(b, INT64_MAX, 64, f, f, 1, 1e-5f, b, f, f, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm(b, 8, INT64_MAX - 7, f, f, 1, 1e-5f, b, f, f, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm(b, 8, 64, nullptr, f, 1, 1e-5f, b, f, f, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm(b, 8, 64, f, M, 1, 1e-5f, b, f, f, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm(b, 8, 64, f, f, INT32_MIN, 1e-5f, b, f, f, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm(b, 8, 64, f, f, 1, -1.f, b, f, f, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm(b, 8, 64, f, f, 1, 1e-5f, b, (float *)O, f, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm_bwd(b, b, 8, 64, f, 1, nullptr, f, b, f, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm_bwd(b, b, 8, 64, f, 1, f, f, m, f, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm_bwd(b, b, 8, 64, f, 1, f, f, b, f, f, F, 0, nullptr), QLORA_EWORKSPACE);
  EXPECT(qlora_layer_norm_workspace_bytes(8, 64, nullptr), QLORA_EINVAL);
  EXPECT(qlora_layer_norm_workspace_bytes(INT64_MAX, 64, &n), QLORA_EINVAL);

  EXPECT(qlora_adapters_fwd(b, INT64_MAX, 64, b, b, 72, 3, 16, x, f, x, b, b, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_fwd(b, 8, INT64_MAX - 7, b, b, 72, 3, 16, x, f, x, b, b, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_fwd(b, 8, 64, b, b, INT64_MIN, 3, 16, x, f, x, b, b, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_fwd(b, 8, 64, b, b, 72, INT32_MAX, 16, x, f, x, b, b, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_fwd(b, 8, 64, b, b, 72, 3, INT32_MIN, x, f, x, b, b, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_fwd(b, 8, 64, b, b, 72, 3, 16, x, nullptr, x, b, b, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_fwd(b, 8, 64, b, b, 72, 3, 16, x, f, x, m, b, f, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_fwd(b, 8, 64, b, b, 72, 3, 16, x, f, x, b, b, f, F, 0, nullptr), QLORA_EWORKSPACE);
  EXPECT(qlora_adapters_bwd(b, nullptr, 8, 64, b, b, 72, 3, 16, x, f, x, f, b, b, b, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_bwd(b, b, 8, 64, b, b, 72, 3, 16, x, f, x, f, b, b, m, b, F, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_bwd(b, b, 8, 64, b, b, 72, 3, 16, x, f, x, f, b, b, b, b, M, big, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_bwd(b, b, 8, 64, b, b, 72, 3, 16, x, f, x, f, b, b, b, b, F, 0, nullptr), QLORA_EWORKSPACE);
  EXPECT(qlora_adapters_workspace_bytes(8, 64, 72, 3, 16, 1, nullptr), QLORA_EINVAL);
  EXPECT(qlora_adapters_workspace_bytes(INT64_MIN, 64, 72, 3, 16, 1, &n), QLORA_EINVAL);

  const int64_t top = (int64_t)1 << 22;
  const int64_t Ts[] = {0, 1, 2, 16, 63, 64, 65, 128, 129, 512, 513, 1023, 1025, 2048, 4097, 8192, 8193, 100000, top - 1, top};
  const int64_t Ns[] = {8, 64, 120, 1000, 2048, 4104, 8192, 16384, 32768, 32776, 1 << 20, top};
  const int32_t pools[] = {1, 2, 31, 64, 1000}, ranks[] = {8, 24, 64, 128};
  int plans = 0;
  for (int64_t T : Ts)
    for (int64_t K : Ns)
      for (int64_t N : Ns)
        for (int32_t pool : pools)
          for (int32_t r : ranks) {
            const bool fits = T * K < (int64_t)1 << 32 && T * N < (int64_t)1 << 32 && pool * K <= 1 << 27 && pool * N <= 1 << 27;
            EXPECT(qlora_adapters_workspace_bytes(T, K, N, pool, r, 0, &n), fits ? QLORA_OK : QLORA_EINVAL);
            if (fits) plan(T, K, N, pool, r), ++plans;
          }
  printf("%d plans\n", plans);
  printf(g_fail ? "step asan driver FAILED\n" : "step asan driver ok\n");
  return g_fail;
}
