// step.h -- launchers of what a step has beside the NF4 linears and the losses: embedding, layer norm, adapters by token
// (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace qlora {

// Rows by key: order[p] is the row at place p of the rows sorted by key, equal keys by row; key[p] its key.  A key
// outside [0, n_keys) counts as n_keys and comes last.
constexpr int64_t kOrderChunk = 8192;  // rows that are ranked against each other; longer lists merge such chunks
struct Order {
  int32_t *order = nullptr, *key = nullptr;    // [T]
  int32_t *order2 = nullptr, *key2 = nullptr;  // [T], of the chunks before they are merged (T > kOrderChunk only)
};

// Embedding.
hipError_t launch_embed(const int64_t *tokens, int64_t T, const bf16_t *W, int64_t V, int64_t D, float scale, bf16_t *Y,
                        hipStream_t s);
// Entries of the sorted list that one wave adds up, and the bytes of the sums that cross from one such piece to the next.
int embed_piece(int64_t T);
hipError_t launch_embed_order(const int64_t *tokens, int64_t T, int64_t V, const Order &o, bf16_t *fill, int64_t fill_n,
                              hipStream_t s);
hipError_t launch_embed_merge(int64_t T, const Order &o, hipStream_t s);
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
hipError_t launch_norm_reduce(const float *part, int groups, int64_t D, bool f32, void *dw, void *db, hipStream_t s);

}  // namespace qlora
