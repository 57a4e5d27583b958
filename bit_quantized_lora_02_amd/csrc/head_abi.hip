// head_abi.hip -- the C ABI of the output layer's losses: argument checks, workspace planning, kernel sequencing, as
// abi.hip does for the other entry points.
#include "abi.h"
#include "head.h"
#include "qlora.h"

using namespace qlora;

namespace {

// E (2 bytes per row and column of the vocabulary), or without gradients the tile statistics, is held for a block of
// rows at a time, of at most this many bytes: at 4096 rows of a 128256-wide vocabulary the products run at full size (256
// tiles of dX), so larger blocks would gain logits and dX nothing and smaller ones would leave compute units idle.  dW
// reads and writes its carried sums once per block, which larger ones would save some of.
constexpr size_t kHeadBlockBytes = (size_t)1 << 30;

struct HeadPlan {
  HeadBlocks b = {};
  int64_t ntile = 0;
  int64_t ldx = 0;  // rows per block of the laid out X
  size_t off_n = 0, off_ranges = 0, off_xt = 0, off_list = 0, off_ref = 0, off_col = 0, off_zt = 0, off_pt = 0,
         off_bucket = 0, off_target = 0, off_stat = 0, off_scale = 0, off_z = 0, off_e = 0, off_part = 0, off_xs = 0,
         off_sums = 0, total = 0;
  int ranges = 1;      // of the logit product's reduction
  int dw_ranges = 1;   // of the dW product's
};

HeadPlan head_plan(int64_t T, int64_t V, int64_t K, int32_t k, bool dx, bool dw) {
  HeadPlan p;
  const bool grad = dx || dw;
  // (a block holds at least 256 rows where there are several, and then the vocabulary is wide: the tile follows from T, V)
  p.b.tile_rows = head_tile_rows(T, V);
  p.ntile = ceil_div(V, kHeadStat);
  const int64_t tiles = ceil_div(V, head_tile_cols(p.b.tile_rows));
  p.b.lde = ceil_div(V, kHeadPad) * kHeadPad;
  const size_t row = grad ? (size_t)p.b.lde * 2 : (size_t)p.ntile * sizeof(float2);
  int64_t most = (int64_t)(kHeadBlockBytes / row) / 256 * 256;
  most = most < 256 ? 256 : most;
  p.b.count = T <= most ? 1 : ceil_div(T, most);
  p.b.tb = p.b.count == 1 ? (T < 1 ? 1 : T) : (int64_t)up((size_t)ceil_div(T, p.b.count), 256);
  p.b.count = T < 1 ? 1 : ceil_div(T, p.b.tb);
  p.b.te = (int64_t)up((size_t)p.b.tb, 16);
  p.ldx = (int64_t)up((size_t)T, 16);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up(off + bytes, kAlign);
    return at;
  };
  p.off_n = take(4);
  p.off_ranges = take((size_t)p.b.count * 16);
  p.off_xt = take((size_t)ceil_div(K, 128) * p.ldx * 256);
  p.off_list = take((size_t)T * 4);
  p.off_ref = take((size_t)T * 4);
  p.off_col = take((size_t)T * 4);
  if (k > 0) {
    p.off_zt = take((size_t)T * k * 4);
    p.off_pt = take((size_t)T * k * 4);
    const size_t tr = p.b.tile_rows, row_tiles = ((size_t)p.b.tb + tr - 1) / tr;
    p.off_bucket = take(row_tiles * (size_t)(tiles + 1) * 4);
    p.off_target = take(row_tiles * tr * (size_t)k * 4);
  }
  p.off_stat = take((size_t)p.b.tb * p.ntile * sizeof(float2));
  p.off_scale = take((size_t)p.b.tb * sizeof(float4));
  p.ranges = p.b.count == 1 && T > 0 ? head_logit_ranges(T, V, K, p.b.tile_rows) : 1;
  if (p.ranges > 1) p.off_z = take((size_t)p.ranges * T * p.b.lde * 4);
  if (grad) p.off_e = take((size_t)p.b.te * p.b.lde * 2);
  if (dx) p.off_part = take(head_part_floats(p.b.tb, K, p.b.tile_rows) * 4);
  if (dw) {
    p.off_xs = take(up((size_t)p.b.tb, 128) * K * 2);
    p.dw_ranges = head_dw_ranges(T, V, K, p.b.count);
    if (p.b.count > 1 || p.dw_ranges > 1) p.off_sums = take((size_t)V * K * p.dw_ranges * 4);
  }
  p.total = off;
  return p;
}

int check_head_sizes(int64_t T, int64_t V, int64_t K) {
  if (T < 0 || T > kMaxDim) return fail(QLORA_EINVAL, "T must be in [0, 2^22] (got %lld)", (long long)T);
  if (V < 1 || V > kMaxDim || K < 8 || K > kMaxDim || K % 8 != 0)
    return fail(QLORA_EINVAL, "need n_vocab >= 1 and n_in a positive multiple of 8, each at most 2^22 (got %lld x %lld)",
                (long long)V, (long long)K);
  // (T n_in: no kernel needs this limit, offsets into X, its copies and dX are 64 bits wide or within a block of 32 columns;
  // larger batches have not been run)
  if (V * K > kMaxWeights || T * K >= (int64_t)1 << 31)
    return fail(QLORA_EINVAL, "n_vocab x n_in must be at most 2^34 and T x n_in below 2^31 (got T=%lld, %lld x %lld)",
                (long long)T, (long long)V, (long long)K);
  return QLORA_OK;
}

bool aligned_to(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Either labels (k = 0) or index and logit (k >= 1 teacher logits per row).
int head_loss(const qlora_bf16 *X, int64_t T, const qlora_bf16 *W, int64_t V, int64_t K, const int64_t *labels,
              const int32_t *index, const float *logit, int32_t k, float tau, const float *weight, float *loss,
              qlora_bf16 *dX, qlora_bf16 *dW, void *ws, size_t ws_bytes, void *stream) {
  int rc = check_head_sizes(T, V, K);
  if (rc) return rc;
  if (!W || !aligned16(W)) return fail(QLORA_EINVAL, "W must be non-NULL and 16-byte aligned");
  if (T > 0 && (!X || !loss)) return fail(QLORA_EINVAL, "X and loss must not be NULL");
  if (!aligned16(X) || !aligned16(dX) || !aligned16(dW))
    return fail(QLORA_EINVAL, "X, dX and dW must be 16-byte aligned");
  if (!aligned_to(loss, 4) || !aligned_to(weight, 4))
    return fail(QLORA_EINVAL, "loss and weight must be 4-byte aligned");
  const HeadPlan p = head_plan(T, V, K, k, dX != nullptr, dW != nullptr);
  if (ws_bytes < p.total) return fail(QLORA_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, p.total);
  if (!ws || !aligned_to(ws, kAlign)) return fail(QLORA_EINVAL, "workspace must be non-NULL and 256-byte aligned");
  if ((rc = check_device(nullptr))) return rc;
  if (T == 0 && !dW) return QLORA_OK;
  hipStream_t s = (hipStream_t)stream;
  char *w = (char *)ws;
  int32_t *n = (int32_t *)(w + p.off_n), *list = (int32_t *)(w + p.off_list);
  HeadRows rows;
  rows.n = n;
  rows.ranges = nullptr;
  rows.tile_rows = p.b.tile_rows;
  rows.list = list;
  rows.ref = (float *)(w + p.off_ref);
  rows.refcol = (int32_t *)(w + p.off_col);
  rows.zt = k > 0 ? (float *)(w + p.off_zt) : nullptr;
  rows.pt = k > 0 ? (float *)(w + p.off_pt) : nullptr;
  rows.bucket = k > 0 ? (int32_t *)(w + p.off_bucket) : nullptr;
  rows.target = k > 0 && p.ranges == 1 ? (uint32_t *)(w + p.off_target) : nullptr;
  const bool grad = dX || dW;
  float2 *stat = (float2 *)(w + p.off_stat);
  float4 *scale = (float4 *)(w + p.off_scale);
  bf16_t *E = grad ? (bf16_t *)(w + p.off_e) : nullptr;
  float *part = dX ? (float *)(w + p.off_part) : nullptr;
  bf16_t *Xs = dW ? (bf16_t *)(w + p.off_xs) : nullptr;
  float *sums = p.off_sums ? (float *)(w + p.off_sums) : nullptr;
  bf16_t *Xt = (bf16_t *)(w + p.off_xt);
  int32_t *ranges = (int32_t *)(w + p.off_ranges);
  const float c = 1.44269504f / tau;
  const int64_t lde = p.b.lde, te = p.b.te;
  LAUNCH("head_prep", launch_head_prep(X, T, W, V, K, labels, index, logit, k, tau, n, list, ranges, p.b, rows, loss, dX,
                                       Xt, p.ldx, s));
  const bool sorted = k > 0 && p.ranges == 1;  // the targets go by the product's tiles
  float *zpart = p.ranges > 1 ? (float *)(w + p.off_z) : nullptr;
  const bool few = k > 0 && head_few_targets(T, k, p.b.tile_rows);
  if (k > 0 && !few) LAUNCH("head_list", launch_head_list(rows, T, K, n, list, ranges, p.b, s));
  for (int64_t b = 0; b < p.b.count; ++b) {
    const int64_t row0 = b * p.b.tb, tb = T - row0 < p.b.tb ? T - row0 : p.b.tb;
    rows.ranges = ranges + 4 * b;
    if (tb > 0 && sorted && !few) LAUNCH("head_bucket", launch_head_bucket(rows, row0, tb, index, k, V, s));
    if (tb > 0)
      LAUNCH("head_logits", launch_head_logits(rows, row0, tb, Xt, p.ldx, W, V, K, c, stat, p.ntile, E, lde, te, k,
                                               p.ranges, zpart, s));
    if (tb > 0 && zpart)
      LAUNCH("head_soft", launch_head_soft(rows, row0, tb, zpart, p.ranges, V, c, stat, p.ntile, index, k, E, lde, te, s));
    if (tb > 0 || dW)
      LAUNCH("head_combine", launch_head_combine(rows, row0, tb, stat, p.ntile, V, labels, index, k, tau, weight, loss,
                                                 scale, E, lde, te, X, K, Xs, s));
    if (tb > 0 && dX) {
      LAUNCH("head_dx", launch_head_dx(rows, row0, tb, E, lde, te, W, V, K, scale, part, dX, s));
      LAUNCH("head_dx_reduce", launch_head_reduce(rows, row0, tb, part, W, K, scale, dX, s));
    }
    if (dW && tb > 0) {
      LAUNCH("head_scale", launch_head_scale(rows, row0, tb, scale, E, lde, te, s));
      if (k > 0) LAUNCH("head_put", launch_head_put(rows, row0, tb, V, index, k, scale, E, te, s));
    }
    if (dW)
      LAUNCH("head_dw",
             launch_head_dw(rows, row0, tb, E, lde, te, Xs, V, K, sums, b == 0, b + 1 == p.b.count && p.dw_ranges == 1,
                            p.dw_ranges, dW, s));
    if (dW && p.dw_ranges > 1)
      LAUNCH("head_dw_reduce", launch_head_dw_reduce(rows, tb, sums, p.dw_ranges, V, K, dW, s));
  }
  return QLORA_OK;
}

}  // namespace

extern "C" {

int qlora_head_workspace_bytes(int64_t T, int64_t n_vocab, int64_t n_in, int32_t k, int need_dx, int need_dw,
                               size_t *bytes) {
  if (!bytes) return fail(QLORA_EINVAL, "bytes is NULL");
  if (int rc = check_head_sizes(T, n_vocab, n_in)) return rc;
  if (k < 0 || k > QLORA_MAX_TARGETS) return fail(QLORA_EINVAL, "k must be in [0, %d] (got %d)", QLORA_MAX_TARGETS, (int)k);
  *bytes = head_plan(T, n_vocab, n_in, k, need_dx != 0, need_dw != 0).total;
  return QLORA_OK;
}

int qlora_head_ce(const qlora_bf16 *X, int64_t T, const qlora_bf16 *W, int64_t n_vocab, int64_t n_in,
                  const int64_t *labels, const float *weight, float *loss, qlora_bf16 *dX, qlora_bf16 *dW, void *ws,
                  size_t ws_bytes, void *stream) {
  if (T > 0 && !labels) return fail(QLORA_EINVAL, "labels must not be NULL");
  if (!aligned_to(labels, 8)) return fail(QLORA_EINVAL, "labels must be 8-byte aligned");
  return head_loss(X, T, W, n_vocab, n_in, labels, nullptr, nullptr, 0, 1.f, weight, loss, dX, dW, ws, ws_bytes,
                   stream);
}

int qlora_head_distill(const qlora_bf16 *X, int64_t T, const qlora_bf16 *W, int64_t n_vocab, int64_t n_in,
                       const int32_t *index, const float *logit, int32_t k, float tau, const float *weight,
                       float *loss, qlora_bf16 *dX, qlora_bf16 *dW, void *ws, size_t ws_bytes, void *stream) {
  if (k < 1 || k > QLORA_MAX_TARGETS) return fail(QLORA_EINVAL, "k must be in [1, %d] (got %d)", QLORA_MAX_TARGETS, (int)k);
  if (!(tau >= 1e-4f && tau <= 1e4f)) return fail(QLORA_EINVAL, "tau must be in [1e-4, 1e4] (got %g)", (double)tau);
  if (T > 0 && (!index || !logit)) return fail(QLORA_EINVAL, "index and logit must not be NULL");
  if (!aligned_to(index, 4) || !aligned_to(logit, 4)) return fail(QLORA_EINVAL, "index and logit must be 4-byte aligned");
  return head_loss(X, T, W, n_vocab, n_in, nullptr, index, logit, k, tau, weight, loss, dX, dW, ws, ws_bytes, stream);
}

}  // extern "C"
