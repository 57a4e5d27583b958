// step_abi.hip -- the C ABI of the embedding, the layer norm and the adapters by token: argument checks, workspace
// planning, kernel sequencing, as abi.hip does for the linear layer.
#include "abi.h"
#include "qlora.h"
#include "step.h"

using namespace qlora;

namespace {

bool aligned_to(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_tokens(int64_t T) {
  if (T < 0 || T > kMaxDim) return fail(QLORA_EINVAL, "T must be in [0, 2^22] (got %lld)", (long long)T);
  return QLORA_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
  if (bytes < need) return fail(QLORA_EWORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
  if (need && (!ws || !aligned_to(ws, kAlign)))
    return fail(QLORA_EINVAL, "workspace must be non-NULL and 256-byte aligned");
  return QLORA_OK;
}

// Parts of a workspace, one behind the other.
struct Parts {
  size_t total = 0;
  size_t take(size_t bytes) {
    const size_t at = total;
    total = up(total + bytes, kAlign);
    return at;
  }
};

// ------------------------------------------------------------------ embedding
int check_embed(int64_t T, int64_t V, int64_t D) {
  if (int rc = check_tokens(T)) return rc;
  if (V < 1 || V > kMaxDim || D < 8 || D > kMaxDim || D % 8 != 0)
    return fail(QLORA_EINVAL, "need n_vocab >= 1 and n_in a positive multiple of 8, each at most 2^22 (got %lld x %lld)",
                (long long)V, (long long)D);
  if (V * D > kMaxWeights || T * D >= (int64_t)1 << 32)
    return fail(QLORA_EINVAL, "n_vocab x n_in must be at most 2^34 and T x n_in below 2^32 (got T=%lld, %lld x %lld)",
                (long long)T, (long long)V, (long long)D);
  return QLORA_OK;
}

struct EmbedPlan {
  size_t order = 0, key = 0, order2 = 0, key2 = 0, part = 0, total = 0;
};

EmbedPlan embed_plan(int64_t T, int64_t D) {
  EmbedPlan p;
  Parts w;
  p.order = w.take((size_t)T * 4);
  p.key = w.take((size_t)T * 4);
  if (T > kOrderChunk) {
    p.order2 = w.take((size_t)T * 4);
    p.key2 = w.take((size_t)T * 4);
  }
  const int64_t pieces = ceil_div(T, embed_piece(T));
  if (pieces > 1) p.part = w.take((size_t)pieces * 2 * D * 4);
  p.total = w.total;
  return p;
}

// ----------------------------------------------------------------- layer norm
int check_norm(int64_t T, int64_t D, int weights) {
  if (int rc = check_tokens(T)) return rc;
  if (D < 8 || D > kNormMax || D % 8 != 0)
    return fail(QLORA_EINVAL, "n_in must be a multiple of 8 in [8, %d] (got %lld)", (int)kNormMax, (long long)D);
  if (T * D >= (int64_t)1 << 32)
    return fail(QLORA_EINVAL, "T x n_in must be below 2^32 (got %lld x %lld)", (long long)T, (long long)D);
  if (weights != QLORA_WEIGHT_BF16 && weights != QLORA_WEIGHT_F32)
    return fail(QLORA_EINVAL, "weight_type must be QLORA_WEIGHT_BF16 or QLORA_WEIGHT_F32 (got %d)", weights);
  return QLORA_OK;
}

// ------------------------------------------------------------------- adapters
int check_adapters(int64_t T, int64_t n_in, int64_t n_out, int32_t n_pool, int32_t r) {
  if (int rc = check_tokens(T)) return rc;
  if (n_in < 8 || n_in > kMaxDim || n_in % 8 || n_out < 8 || n_out > kMaxDim || n_out % 8)
    return fail(QLORA_EINVAL, "n_in and n_out must be positive multiples of 8, at most 2^22 (got %lld, %lld)",
                (long long)n_in, (long long)n_out);
  if (n_pool < 1 || n_pool > kPoolMax)
    return fail(QLORA_EINVAL, "n_pool must be in [1, %d] (got %d)", kPoolMax, (int)n_pool);
  if (r < 8 || r > QLORA_MAX_RANK || r % 8)
    return fail(QLORA_EINVAL, "r must be a multiple of 8 in [8, %d] (got %d)", QLORA_MAX_RANK, (int)r);
  if (n_pool * n_in > (int64_t)1 << 27 || n_pool * n_out > (int64_t)1 << 27)
    return fail(QLORA_EINVAL, "n_pool x n_in and n_pool x n_out must be at most 2^27");
  if (T * n_in >= (int64_t)1 << 32 || T * n_out >= (int64_t)1 << 32)
    return fail(QLORA_EINVAL, "T x n_in and T x n_out must be below 2^32");
  return QLORA_OK;
}

struct AdaptPlan {
  int ranges_u = 1, ranges_du = 1, piece = 0;
  size_t order = 0, start = 0, counts = 0, u = 0, du = 0, du_sum = 0, at = 0, bt = 0, part_a = 0, part_b = 0, total = 0;
};

AdaptPlan adapt_plan(int64_t T, int64_t n_in, int64_t n_out, int32_t n_pool, int32_t r, bool backward) {
  AdaptPlan p;
  Parts w;
  p.order = w.take((size_t)T * 4);
  p.start = w.take((size_t)(n_pool + 2) * 4);
  if (T > kAdaptChunk) p.counts = w.take((size_t)adapt_chunks(T) * (n_pool + 1) * 4);
  p.ranges_u = adapt_ranges(T, n_pool, r, n_in);
  p.u = w.take((size_t)p.ranges_u * T * r * 4);
  if (backward) {
    p.ranges_du = adapt_ranges(T, n_pool, r, n_out);
    p.du = w.take((size_t)p.ranges_du * T * r * 4);
    p.du_sum = p.ranges_du > 1 ? w.take((size_t)T * r * 4) : p.du;
    p.at = w.take((size_t)n_pool * r * n_in * 2);
    p.bt = w.take((size_t)n_pool * r * n_out * 2);
    p.piece = adapt_piece(T, n_in, n_out);
    const size_t slots = (size_t)adapt_slots(T, p.piece);
    p.part_a = w.take(slots * r * n_in * 4);
    p.part_b = w.take(slots * r * n_out * 4);
  }
  p.total = w.total;
  return p;
}

int check_pool(const void *X, const void *A, const void *B, const int32_t *rank, const float *scale, const int32_t *index,
               int64_t T) {
  if (!A || !B || !scale) return fail(QLORA_EINVAL, "A_pool, B_pool and scale must not be NULL");
  if (T > 0 && (!X || !index)) return fail(QLORA_EINVAL, "X and index must not be NULL");
  if (!aligned16(X) || !aligned16(A) || !aligned16(B))
    return fail(QLORA_EINVAL, "X, A_pool and B_pool must be 16-byte aligned");
  if (!aligned_to(rank, 4) || !aligned_to(scale, 4) || !aligned_to(index, 4))
    return fail(QLORA_EINVAL, "rank, scale and index must be 4-byte aligned");
  return QLORA_OK;
}

}  // namespace

extern "C" {

int qlora_adapters_workspace_bytes(int64_t T, int64_t n_in, int64_t n_out, int32_t n_pool, int32_t r, int backward,
                                   size_t *bytes) {
  if (!bytes) return fail(QLORA_EINVAL, "bytes is NULL");
  if (int rc = check_adapters(T, n_in, n_out, n_pool, r)) return rc;
  *bytes = adapt_plan(T, n_in, n_out, n_pool, r, backward != 0).total;
  return QLORA_OK;
}

int qlora_adapters_fwd(const qlora_bf16 *X, int64_t T, int64_t n_in, const qlora_bf16 *A_pool, const qlora_bf16 *B_pool,
                       int64_t n_out, int32_t n_pool, int32_t r, const int32_t *rank, const float *scale,
                       const int32_t *index, const qlora_bf16 *base, qlora_bf16 *Y, float *U_out, void *ws, size_t ws_bytes,
                       void *stream) {
  int rc = check_adapters(T, n_in, n_out, n_pool, r);
  if (rc) return rc;
  if ((rc = check_pool(X, A_pool, B_pool, rank, scale, index, T))) return rc;
  if (T > 0 && !Y) return fail(QLORA_EINVAL, "Y must not be NULL");
  if (!aligned16(base) || !aligned16(Y) || !aligned16(U_out))
    return fail(QLORA_EINVAL, "base, Y and U_out must be 16-byte aligned");
  const AdaptPlan p = adapt_plan(T, n_in, n_out, n_pool, r, false);
  if ((rc = check_workspace(ws, ws_bytes, p.total))) return rc;
  if ((rc = check_device(nullptr))) return rc;
  if (T == 0) return QLORA_OK;
  hipStream_t s = (hipStream_t)stream;
  char *w = (char *)ws;
  AdaptRows a;
  a.index = index;
  a.T = T;
  a.n_pool = n_pool;
  a.r = r;
  a.rank = rank;
  a.scale = scale;
  if (T > kAdaptSmall) {
    a.order = (int32_t *)(w + p.order);
    a.start = (int32_t *)(w + p.start);
    if (T > kAdaptChunk) {
      a.counts = (int32_t *)(w + p.counts);
      LAUNCH("adapters_count", launch_adapt_count(a, s));
    }
    LAUNCH("adapters_plan", launch_adapt_plan(a, AdaptTurn(), AdaptTurn(), s));
  }
  const bool direct = U_out && p.ranges_u == 1;
  float *U = direct ? U_out : (float *)(w + p.u);
  LAUNCH("adapters_shrink", launch_adapt_shrink(a, X, n_in, A_pool, false, p.ranges_u, U, s));
  LAUNCH("adapters_expand",
         launch_adapt_expand(a, U, p.ranges_u, B_pool, n_out, true, base, Y, direct ? nullptr : U_out, s));
  return QLORA_OK;
}

int qlora_adapters_bwd(const qlora_bf16 *X, const qlora_bf16 *dY, int64_t T, int64_t n_in, const qlora_bf16 *A_pool,
                       const qlora_bf16 *B_pool, int64_t n_out, int32_t n_pool, int32_t r, const int32_t *rank,
                       const float *scale, const int32_t *index, const float *U, const qlora_bf16 *base, qlora_bf16 *dX,
                       qlora_bf16 *dA, qlora_bf16 *dB, void *ws, size_t ws_bytes, void *stream) {
  int rc = check_adapters(T, n_in, n_out, n_pool, r);
  if (rc) return rc;
  if ((rc = check_pool(X, A_pool, B_pool, rank, scale, index, T))) return rc;
  if (T > 0 && !dY) return fail(QLORA_EINVAL, "dY must not be NULL");
  if (!aligned16(dY) || !aligned16(U) || !aligned16(base) || !aligned16(dX) || !aligned16(dA) || !aligned16(dB))
    return fail(QLORA_EINVAL, "dY, U, base, dX, dA and dB must be 16-byte aligned");
  const AdaptPlan p = adapt_plan(T, n_in, n_out, n_pool, r, true);
  if ((rc = check_workspace(ws, ws_bytes, p.total))) return rc;
  if ((rc = check_device(nullptr))) return rc;
  const bool dx = dX && T > 0;
  if (!dx && !dA && !dB) return QLORA_OK;
  hipStream_t s = (hipStream_t)stream;
  char *w = (char *)ws;
  AdaptRows a;
  a.index = index;
  a.T = T;
  a.n_pool = n_pool;
  a.r = r;
  a.rank = rank;
  a.scale = scale;
  a.order = (int32_t *)(w + p.order);
  a.start = (int32_t *)(w + p.start);
  AdaptTurn ta, tb;  // A [r][n_in] to [n_in][r] for dX, B [n_out][r] to [r][n_out] for dU
  if (dx) {
    ta.from = A_pool;
    ta.to = (bf16_t *)(w + p.at);
    ta.rows = r;
    ta.cols = n_in;
  }
  if (T > 0 && (dx || dA)) {
    tb.from = B_pool;
    tb.to = (bf16_t *)(w + p.bt);
    tb.rows = n_out;
    tb.cols = r;
  }
  if (T > kAdaptChunk) {
    a.counts = (int32_t *)(w + p.counts);
    LAUNCH("adapters_count", launch_adapt_count(a, s));
  }
  LAUNCH("adapters_plan", launch_adapt_plan(a, ta, tb, s));
  AdaptGrads g;
  g.X = X;
  g.dY = dY;
  g.n_in = n_in;
  g.n_out = n_out;
  g.part_a = (float *)(w + p.part_a);
  g.part_b = (float *)(w + p.part_b);
  g.dA = dA;
  g.dB = dB;
  g.U = U;
  if (T > 0) {
    // (the gradients of the pools take u and du whole: ranges of du are added where dX is formed)
    if (dB && !U) {
      float *u = (float *)(w + p.u);
      LAUNCH("adapters_shrink", launch_adapt_shrink(a, X, n_in, A_pool, false, 1, u, s));
      g.U = u;
    }
    const bool few = T <= kAdaptFew && dx && (dA || dB);
    if (dx || dA) {
      float *du = (float *)(w + p.du), *sum = (float *)(w + p.du_sum);
      const int ranges = dx ? p.ranges_du : 1;
      LAUNCH("adapters_shrink", launch_adapt_shrink(a, dY, n_out, tb.to, true, ranges, du, s));
      g.dU = du;
      if (few) {
        g.dU_ranges = ranges;
        LAUNCH("adapters_back", launch_adapt_back(a, g, p.piece, ta.to, base, dX, s));
        return QLORA_OK;
      }
      if (dx)
        LAUNCH("adapters_expand", launch_adapt_expand(a, du, ranges, ta.to, n_in, false, base, dX,
                                                      dA && ranges > 1 ? sum : nullptr, s));
      if (ranges > 1) g.dU = sum;
    }
  }
  if (dA || dB) LAUNCH("adapters_grads", launch_adapt_grads(a, g, p.piece, s));
  if ((dA || dB) && T > p.piece) LAUNCH("adapters_reduce", launch_adapt_reduce(a, g, p.piece, s));
  return QLORA_OK;
}

int qlora_embed(const int64_t *tokens, int64_t T, const qlora_bf16 *W, int64_t n_vocab, int64_t n_in, float scale,
                qlora_bf16 *Y, void *stream) {
  int rc = check_embed(T, n_vocab, n_in);
  if (rc) return rc;
  if (!W || !aligned16(W)) return fail(QLORA_EINVAL, "W must be non-NULL and 16-byte aligned");
  if (T > 0 && (!tokens || !Y)) return fail(QLORA_EINVAL, "tokens and Y must not be NULL");
  if (!aligned_to(tokens, 8)) return fail(QLORA_EINVAL, "tokens must be 8-byte aligned");
  if (!aligned16(Y)) return fail(QLORA_EINVAL, "Y must be 16-byte aligned");
  if ((rc = check_device(nullptr))) return rc;
  if (T == 0) return QLORA_OK;
  hipStream_t s = (hipStream_t)stream;
  LAUNCH("embed", launch_embed(tokens, T, W, n_vocab, n_in, scale, Y, s));
  return QLORA_OK;
}

int qlora_embed_workspace_bytes(int64_t T, int64_t n_in, size_t *bytes) {
  if (!bytes) return fail(QLORA_EINVAL, "bytes is NULL");
  if (int rc = check_embed(T, 1, n_in)) return rc;
  *bytes = embed_plan(T, n_in).total;
  return QLORA_OK;
}

int qlora_embed_bwd(const int64_t *tokens, const qlora_bf16 *dY, int64_t T, int64_t n_vocab, int64_t n_in, float scale,
                    int accumulate, qlora_bf16 *dW, void *ws, size_t ws_bytes, void *stream) {
  int rc = check_embed(T, n_vocab, n_in);
  if (rc) return rc;
  if (!dW || !aligned16(dW)) return fail(QLORA_EINVAL, "dW must be non-NULL and 16-byte aligned");
  if (T > 0 && (!tokens || !dY)) return fail(QLORA_EINVAL, "tokens and dY must not be NULL");
  if (!aligned_to(tokens, 8)) return fail(QLORA_EINVAL, "tokens must be 8-byte aligned");
  if (!aligned16(dY)) return fail(QLORA_EINVAL, "dY must be 16-byte aligned");
  const EmbedPlan p = embed_plan(T, n_in);
  if ((rc = check_workspace(ws, ws_bytes, p.total))) return rc;
  if ((rc = check_device(nullptr))) return rc;
  hipStream_t s = (hipStream_t)stream;
  char *w = (char *)ws;
  Order o;
  o.order = (int32_t *)(w + p.order);
  o.key = (int32_t *)(w + p.key);
  o.order2 = (int32_t *)(w + p.order2);
  o.key2 = (int32_t *)(w + p.key2);
  float *part = (float *)(w + p.part);
  const bool add = accumulate != 0;
  if (T == 0 && add) return QLORA_OK;
  if (T > 0 && T <= kEmbedFew) {
    LAUNCH("embed_few", launch_embed_few(tokens, T, dY, n_vocab, n_in, scale, add, dW, s));
    return QLORA_OK;
  }
  LAUNCH("embed_order", launch_embed_order(tokens, T, n_vocab, o, dW, add ? 0 : n_vocab * n_in, s));
  if (T == 0) return QLORA_OK;
  for (int pass = 0; pass < embed_passes(T); ++pass) LAUNCH("embed_merge", launch_embed_merge(T, pass, o, s));
  LAUNCH("embed_sum", launch_embed_sum(o, T, dY, n_vocab, n_in, scale, add, dW, part, s));
  if (T > embed_piece(T)) LAUNCH("embed_join", launch_embed_join(o, T, n_vocab, n_in, scale, add, dW, part, s));
  return QLORA_OK;
}

int qlora_layer_norm(const qlora_bf16 *X, int64_t T, int64_t n_in, const void *weight, const void *bias, int weight_type,
                     float eps, qlora_bf16 *Y, float *mean, float *rstd, void *stream) {
  int rc = check_norm(T, n_in, weight_type);
  if (rc) return rc;
  if (!(eps >= 0.f) || eps > 3e38f) return fail(QLORA_EINVAL, "eps must be finite and not negative (got %g)", (double)eps);
  if (!weight || !aligned16(weight) || !aligned16(bias))
    return fail(QLORA_EINVAL, "weight must be non-NULL, weight and bias 16-byte aligned");
  if (T > 0 && (!X || !Y)) return fail(QLORA_EINVAL, "X and Y must not be NULL");
  if (!aligned16(X) || !aligned16(Y)) return fail(QLORA_EINVAL, "X and Y must be 16-byte aligned");
  if (!aligned_to(mean, 4) || !aligned_to(rstd, 4)) return fail(QLORA_EINVAL, "mean and rstd must be 4-byte aligned");
  if ((rc = check_device(nullptr))) return rc;
  if (T == 0) return QLORA_OK;
  hipStream_t s = (hipStream_t)stream;
  LAUNCH("layer_norm", launch_norm(X, T, n_in, weight, bias, weight_type == QLORA_WEIGHT_F32, eps, Y, mean, rstd, s));
  return QLORA_OK;
}

int qlora_layer_norm_workspace_bytes(int64_t T, int64_t n_in, size_t *bytes) {
  if (!bytes) return fail(QLORA_EINVAL, "bytes is NULL");
  if (int rc = check_norm(T, n_in, QLORA_WEIGHT_F32)) return rc;
  *bytes = (size_t)norm_bwd_groups(T, n_in) * 2 * n_in * 4;
  return QLORA_OK;
}

int qlora_layer_norm_bwd(const qlora_bf16 *X, const qlora_bf16 *dY, int64_t T, int64_t n_in, const void *weight,
                         int weight_type, const float *mean, const float *rstd, qlora_bf16 *dX, void *dweight, void *dbias,
                         void *ws, size_t ws_bytes, void *stream) {
  int rc = check_norm(T, n_in, weight_type);
  if (rc) return rc;
  if (!weight || !aligned16(weight)) return fail(QLORA_EINVAL, "weight must be non-NULL and 16-byte aligned");
  if (T > 0 && (!X || !dY || !mean || !rstd)) return fail(QLORA_EINVAL, "X, dY, mean and rstd must not be NULL");
  if (!aligned16(X) || !aligned16(dY) || !aligned16(dX) || !aligned16(dweight) || !aligned16(dbias))
    return fail(QLORA_EINVAL, "X, dY, dX, dweight and dbias must be 16-byte aligned");
  if (!aligned_to(mean, 4) || !aligned_to(rstd, 4)) return fail(QLORA_EINVAL, "mean and rstd must be 4-byte aligned");
  const bool sums = dweight || dbias;
  const int groups = norm_bwd_groups(T, n_in);
  if (sums && (rc = check_workspace(ws, ws_bytes, (size_t)groups * 2 * n_in * 4))) return rc;
  if ((rc = check_device(nullptr))) return rc;
  if (!sums && (!dX || T == 0)) return QLORA_OK;
  hipStream_t s = (hipStream_t)stream;
  const bool f32 = weight_type == QLORA_WEIGHT_F32;
  float *part = sums ? (float *)ws : nullptr;
  if (sums && norm_bwd_few(T, n_in) && dX != dY) {
    LAUNCH("layer_norm_bwd", launch_norm_few(X, dY, T, n_in, weight, f32, mean, rstd, dX, dweight, dbias, s));
    return QLORA_OK;
  }
  // (without rows: the sums are zero)
  const bool columns = norm_bwd_columns(n_in);
  if (sums && columns) LAUNCH("layer_norm_columns", launch_norm_columns(X, dY, T, n_in, mean, rstd, part, s));
  if (dX || !columns) LAUNCH("layer_norm_bwd", launch_norm_bwd(X, dY, T, n_in, weight, f32, mean, rstd, dX, part, s));
  if (sums) LAUNCH("layer_norm_reduce", launch_norm_reduce(part, groups, n_in, f32, dweight, dbias, s));
  return QLORA_OK;
}

}  // extern "C"
