// step.h -- launchers of what a step has beside the NF4 linears and the losses: embedding, layer norm, adapters by token
// (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace qlora {

// Rows by key: order[p] is the row at place p of the rows sorted by key, equal keys by row; key[p] its key.  A key
// outside [0, n_keys) counts as n_keys and comes last.
constexpr int64_t kOrderChunk = 8192;  // rows that are ranked against each other at most; longer lists merge sorted chunks
struct Order {
  int32_t *order = nullptr, *key = nullptr;    // [T]
  int32_t *order2 = nullptr, *key2 = nullptr;  // [T], others between passes of the merge (T > kOrderChunk only)
};

// Embedding.
hipError_t launch_embed(const int64_t *tokens, int64_t T, const bf16_t *W, int64_t V, int64_t D, float scale, bf16_t *Y,
                        hipStream_t s);
// The gradient of up to kEmbedFew tokens.
constexpr int64_t kEmbedFew = 128;
hipError_t launch_embed_few(const int64_t *tokens, int64_t T, const bf16_t *dY, int64_t V, int64_t D, float scale, bool add,
                            bf16_t *dW, hipStream_t s);
// Of more: entries of the sorted list that one wave adds up.
int embed_piece(int64_t T);
hipError_t launch_embed_order(const int64_t *tokens, int64_t T, int64_t V, const Order &o, bf16_t *fill, int64_t fill_n,
                              hipStream_t s);
int embed_passes(int64_t T);  // of the merge
hipError_t launch_embed_merge(int64_t T, int pass, const Order &o, hipStream_t s);
hipError_t launch_embed_sum(const Order &o, int64_t T, const bf16_t *dY, int64_t V, int64_t D, float scale, bool add,
                            bf16_t *dW, float *part, hipStream_t s);
hipError_t launch_embed_join(const Order &o, int64_t T, int64_t V, int64_t D, float scale, bool add, bf16_t *dW,
                             const float *part, hipStream_t s);

// Layer norm.  The weights are binary32 where f32 is set, else bf16.
constexpr int64_t kNormMax = 32768;
hipError_t launch_norm(const bf16_t *X, int64_t T, int64_t D, const void *w, const void *b, bool f32, float eps, bf16_t *Y,
                       float *mean, float *rstd, hipStream_t s);
int norm_bwd_groups(int64_t T, int64_t D);  // workgroups, each with binary32 sums [2][D] in `part`
hipError_t launch_norm_bwd(const bf16_t *X, const bf16_t *dY, int64_t T, int64_t D, const void *w, bool f32,
                           const float *mean, const float *rstd, bf16_t *dX, float *part, hipStream_t s);
bool norm_bwd_few(int64_t T, int64_t D);  // few rows: all of the backward in one launch (unless dX is dY itself)
hipError_t launch_norm_few(const bf16_t *X, const bf16_t *dY, int64_t T, int64_t D, const void *w, bool f32,
                           const float *mean, const float *rstd, bf16_t *dX, void *dw, void *db, hipStream_t s);
bool norm_bwd_columns(int64_t D);  // the sums come from a kernel of their own, which goes first (dX may be dY itself)
hipError_t launch_norm_columns(const bf16_t *X, const bf16_t *dY, int64_t T, int64_t D, const float *mean, const float *rstd,
                               float *part, hipStream_t s);
hipError_t launch_norm_reduce(const float *part, int groups, int64_t D, bool f32, void *dw, void *db, hipStream_t s);

// Adapters by token.  The tokens' rows, grouped by adapter: order holds the tokens in groups, group a at start[a] ..
// start[a + 1] - 1 (group n_pool: those without an adapter), each in the order of the batch.
constexpr int kPoolMax = 1000;
constexpr int64_t kAdaptSmall = 64;  // up to so many tokens the forward's workgroups group them by themselves
constexpr int64_t kAdaptFew = 128;   // tokens of a backward whose last two products are one launch
constexpr int64_t kAdaptChunk = 8192;  // tokens that one workgroup groups
__host__ __device__ inline int64_t adapt_chunks(int64_t T) { return (T + kAdaptChunk - 1) / kAdaptChunk; }
struct AdaptRows {
  const int32_t *index = nullptr;  // [T] adapter of each token
  int64_t T = 0;
  int n_pool = 0, r = 0;
  const int32_t *rank = nullptr;   // [n_pool] or null (r)
  const float *scale = nullptr;    // [n_pool]
  int32_t *order = nullptr, *start = nullptr;  // [T], [n_pool + 2]; null: at most kAdaptSmall tokens
  int32_t *counts = nullptr;                   // [chunks][n_pool + 1]; null: one chunk
};
// Groups the tokens and, for each non-null `to`, transposes a pool: from [n_pool][rows][cols] to [n_pool][cols][rows]; the
// ranks are t0's rows and t1's columns.
struct AdaptTurn {
  const bf16_t *from = nullptr;
  bf16_t *to = nullptr;
  int64_t rows = 0, cols = 0;
  int tile_rows = 0, tile_cols = 0;  // of a workgroup (this and the workgroups of a pool are set at the launch)
  uint32_t blocks = 0;
};
hipError_t launch_adapt_count(const AdaptRows &a, hipStream_t s);  // the counts, before the plan
hipError_t launch_adapt_plan(const AdaptRows &a, AdaptTurn t0, AdaptTurn t1, hipStream_t s);
// U[split][t][j] = (scale) P[t] . Q_a[j] over a range of K, Q [n_pool][r][K]: ranges of K (their sums come apart).
int adapt_ranges(int64_t T, int n_pool, int r, int64_t K);
hipError_t launch_adapt_shrink(const AdaptRows &a, const bf16_t *P, int64_t K, const bf16_t *Q, bool scaled, int ranges,
                               float *U, hipStream_t s);
// out[t] = bf16(base[t] + (scale) U[t] . Q_a^T), Q [n_pool][N][r], U the sum of its ranges (also to U_out unless null).
hipError_t launch_adapt_expand(const AdaptRows &a, const float *U, int ranges, const bf16_t *Q, int64_t N, bool scaled,
                               const bf16_t *base, bf16_t *out, float *U_out, hipStream_t s);
// Gradients of the pools: dA[a][j][k] = sum over the group's tokens of dU[t][j] X[t][k], dB[a][n][j] = scale times that of
// U[t][j] dY[t][n].  Groups are cut into pieces of `piece` tokens; those of a group of several go to part.
int adapt_piece(int64_t T, int64_t n_in, int64_t n_out);
inline int64_t adapt_slots(int64_t T, int piece) { return 2 * (T / piece); }  // pieces of groups of several, at most
struct AdaptGrads {
  const float *dU = nullptr, *U = nullptr;
  int dU_ranges = 1;  // that are not added yet (kAdaptFew tokens at most)
  const bf16_t *X = nullptr, *dY = nullptr;
  int64_t n_in = 0, n_out = 0;
  float *part_a = nullptr, *part_b = nullptr;  // [slots][r][n_in], [slots][n_out][r]
  bf16_t *dA = nullptr, *dB = nullptr;
};
hipError_t launch_adapt_grads(const AdaptRows &a, const AdaptGrads &g, int piece, hipStream_t s);
// Up to kAdaptFew tokens: dX, as launch_adapt_expand forms it from dU and Q, and the gradients, which are one piece.
hipError_t launch_adapt_back(const AdaptRows &a, const AdaptGrads &g, int piece, const bf16_t *Q, const bf16_t *base,
                             bf16_t *dX, hipStream_t s);
hipError_t launch_adapt_reduce(const AdaptRows &a, const AdaptGrads &g, int piece, hipStream_t s);

}  // namespace qlora
