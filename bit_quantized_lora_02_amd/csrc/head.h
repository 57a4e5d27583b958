// head.h -- sizes and tables shared by the output layer's loss kernels (head_gemm.hip, head_loss.hip) and the
// C ABI (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlora {

typedef uint16_t bf16_t;

// One loss over the output layer z = X W^T: the rows that count, their targets, and what the kernels hand on.
//
// The rows of X that count (a target inside the vocabulary) are numbered 0 .. n-1 in the order of X; `list` gives
// row i's place in X.  Work goes by blocks of `tb` such rows.  With c = log2(e) / tau, a row's unit u is its first
// target's logit ref = z[refcol] (or, where some logit is so far above it that bf16 would overflow, a larger one),
// and E[v] = exp2((z[v] - u) c) is what is kept of logit v.
struct HeadRows {
  const int32_t *n;       // rows that count
  const int32_t *ranges;  // for the block at hand: the dX product's ranges of its first rows, of the others (which take
                          // 128-row tiles), number of first rows; that number in the logit product
  int tile_rows;          // rows of the products' tiles
  const int32_t *list;  // [T] their rows in X
  float *ref;           // [T] by row of X: the logit of the row's first target
  int32_t *refcol;      // [T] by row of X: that target's column
  // several targets (NULL for one):
  float *zt;             // [T][k] their logits, from the product's tiles; then their entries of E before rounding
  float *pt;             // [T][k] their probabilities
  int32_t *bucket;       // [row tiles][ntile + 1] where each output tile's targets start in `target`
  uint32_t *target;      // [row tiles][rows of a tile * k]: target | column in the tile << 8 | row in the tile << 16
};

// Rows of E are padded with zero columns to a multiple of this.
constexpr int kHeadPad = 128;
// Where a wave's columns of E sum to this or more, they take a unit of their own instead of the row's reference.
constexpr float kHeadRange = 1.0995116e12f;  // 2^40
// Columns per entry of the softmax statistics: a wave's share of a tile, 64, or 128 in the 256 x 256 tile.
constexpr int kHeadStat = 64;
__host__ __device__ inline int head_stat_cols(bool wide_tile) { return wide_tile ? 128 : kHeadStat; }

// Rows of X per tile of the logit and dX products.  Few rows take narrow tiles: the padding rows' MFMA work would cost
// more than the wider tile's operand reuse gains.  So do small outputs, whose 256-wide tiles would not occupy half of the
// chip: a 128-row tile takes 0.6 of the time of a 256-row one (1910 x 1890 x 3232: logits with their sums 50 us in
// 256-row tiles, 44 in 128-row ones; 600 x 8000 x 2048: 46 and 32; but 512 x 32000 x 4096, 250 tiles: 115 and 159).
inline int head_tile_rows(int64_t T, int64_t V) {
  if (T <= 64) return 64;
  return T <= 128 || (V + 255) / 256 * ((T + 255) / 256) <= 128 ? 128 : 256;
}
// Columns of a tile (of the vocabulary in the logit product, of X in the dX product).
// Up to 64 rows the products are bound by the stream of W, and the smaller tile gives every CU some of it.
__host__ __device__ inline int head_tile_cols(int tile_rows) { return tile_rows == 64 ? 128 : 256; }

// Most ranges of the dX product's reduction (one per lane of half a wave when they are chosen), and workgroups of the
// narrow tile that run at once (three per CU).
constexpr int kHeadRanges = 32, kHeadSlots64 = 768;

// Ranges of the logit product's reduction over K for T rows: more than one where the output has too few tiles to
// occupy the chip (a small vocabulary, few rows).  In microseconds: a 32-deep step of a 64-row tile takes 0.25 and 0.001
// for each workgroup that shares the memory, from about 450 of them on their 8 KB of W at 5.3 TB/s (250 workgroups 0.51,
// 375 0.71, 750 1.16); one of a 128-row tile 0.5 and 0.002 for each that streams other rows of W (T = 100: 125 workgroups
// 0.7, 250 1.0; T = 1910: 240 0.6).  Splitting costs a launch, about 5, and the binary32 sums, written and read once
// at about 4.5 TB/s.  (16 x 32000 x 4096: 57 us in two ranges, 60 in one; 64 x 64000 x 4096: 111 in two, 96 in one.)
inline int head_logit_ranges(int64_t T, int64_t V, int64_t K, int tile_rows) {
  const int64_t cols = head_tile_cols(tile_rows), tiles_m = (V + cols - 1) / cols;
  const int64_t tiles = tiles_m * ((T + tile_rows - 1) / tile_rows);
  const int64_t slots = tile_rows == 64 ? kHeadSlots64 : 256, fours = (K + 127) / 128;
  if (tile_rows == 256 || tiles * 2 > slots) return 1;
  auto step = [&](int s) {
    const float streams = (float)(tiles_m * s), some = 0.25f + 0.001f * streams, many = 0.00155f * streams;
    return tile_rows == 128 ? 0.5f + 0.002f * streams : some > many ? some : many;
  };
  const float sums = (float)(T * V) * 8.f / 4.5e6f;
  int best = 1;
  float least = 4.f * (float)fours * step(1);
  for (int s = 2; s <= 16 && s <= fours && tiles * s <= slots; ++s) {
    const float cost = 4.f * (float)((fours + s - 1) / s) * step(s) + 5.f + sums * (float)s;
    if (cost < least) least = cost, best = s;
  }
  const int64_t per = (fours + best - 1) / best;
  return (int)((fours + per - 1) / per);
}

// A teacher's targets of one row tile and at most this many: one of k_head_prep's workgroups numbers the rows and sorts
// the targets while the others take the rows, which saves one launch or two.
constexpr int kHeadFewTargets = 4096;
__host__ __device__ inline bool head_few_targets(int64_t T, int k, int tile_rows) {
  return T <= tile_rows && T * k <= kHeadFewTargets;
}

// How the counted rows are taken in blocks.
struct HeadBlocks {
  int64_t tb, count;  // rows per block (the last: what is left of T), blocks
  int64_t lde;        // columns of E: V rounded up to kHeadPad
  int tile_rows;
  int64_t te;         // rows of E's blocks of columns (E is [lde / 32][te][32])
};

hipError_t launch_head_prep(const bf16_t *X, int64_t T, const bf16_t *W, int64_t V, int64_t K, const int64_t *labels,
                            const int32_t *index, const float *logit, int k, float tau, int32_t *n, int32_t *list,
                            int32_t *ranges, const HeadBlocks &blocks, const HeadRows &rows, float *loss, bf16_t *dX,
                            bf16_t *Xt, int64_t ldx, hipStream_t s);
// Without labels and unless head_few_targets: numbers the rows after launch_head_prep.
hipError_t launch_head_list(const HeadRows &rows, int64_t T, int64_t K, int32_t *n, int32_t *list, int32_t *ranges,
                            const HeadBlocks &blocks, hipStream_t s);
// Sorts the targets of a block's counted rows by the output tile of the logit product they fall into.
hipError_t launch_head_bucket(const HeadRows &rows, int64_t row0, int64_t tb, const int32_t *index, int k, int64_t V,
                              hipStream_t s);
// Losses, the targets' entries of E, and per row of the block (scale) the factor, what the first target's entry lost in
// rounding, the factor's fraction and that target's column; rows of X times the factor's power of two (Xs, for dW).
hipError_t launch_head_combine(const HeadRows &rows, int64_t row0, int64_t tb, const float2 *stat, int64_t ntile,
                               int64_t V, const int64_t *labels, const int32_t *index, int k, float tau,
                               const float *weight, float *loss, float4 *scale, bf16_t *E, int64_t lde, int64_t te,
                               const bf16_t *X, int64_t K, bf16_t *Xs, hipStream_t s);
hipError_t launch_head_scale(const HeadRows &rows, int64_t row0, int64_t tb, const float4 *scale, bf16_t *E, int64_t lde,
                             int64_t te, hipStream_t s);
hipError_t launch_head_put(const HeadRows &rows, int64_t row0, int64_t tb, int64_t V, const int32_t *index, int k,
                           const float4 *scale, bf16_t *E, int64_t te, hipStream_t s);
hipError_t launch_head_reduce(const HeadRows &rows, int64_t row0, int64_t tb, const float *part, const bf16_t *W,
                              int64_t K, const float4 *scale, bf16_t *dX, hipStream_t s);

// Rows that go to tiles of `tile_rows`: all, but for 128 or fewer behind the last whole 256-row tile, which take
// 128-row tiles.  (With all rows in them a 128-row tile takes 0.57 to 0.64 of the time of a 256-row one in the logit product
// and 0.55 to 0.57 in the dX product, 4096 x 128256 x 4096 and 2048 x 128256 x 8192; the rules that choose by it take 0.6
// or 0.62 and 0.57.)
__device__ inline int head_whole_rows(int n, int tile_rows) {
  const int rest = n % 256;
  return tile_rows == 256 && rest >= 1 && rest <= 128 ? n - rest : n;
}
// Columns of the vocabulary (of V) that the dW product takes in 256-wide tiles, `tiles_m` tiles of X's columns each:
// all, but where the last round of 256 workgroups would be half empty its tiles are cut in two.
__host__ __device__ inline int head_whole_columns(int64_t V, int tiles_m) {
  const int tiles = (int)((V + 255) / 256), rounds = (int)((int64_t)tiles * tiles_m / 256);
  const int64_t rest = (int64_t)tiles * tiles_m - (int64_t)rounds * 256;
  const int keep = (int)((int64_t)rounds * 256 / tiles_m);
  return rest >= 1 && rest <= 128 && keep * 256 < V ? keep * 256 : (int)V;
}

// Ranges of the dW product's reduction over T rows (one block of them): more than one where even the narrow tiles leave
// half of the chip idle (a small W).  In microseconds, as for the logits: 0.5 a step, a launch, the binary32 sums.
inline int head_dw_ranges(int64_t T, int64_t V, int64_t K, int64_t blocks) {
  const int64_t tiles_m = (K + 255) / 256, tiles = tiles_m * ((V + 127) / 128), fours = (T + 127) / 128;
  if (blocks > 1 || tiles * 2 > 256) return 1;
  const float sums = (float)(V * K) * 8.f / 4.5e6f;
  int best = 1;
  float least = 2.f * (float)fours;
  for (int s = 2; s <= fours && tiles * s <= 256; ++s) {
    const float cost = 2.f * (float)((fours + s - 1) / s) + 5.f + sums * (float)s;
    if (cost < least) least = cost, best = s;
  }
  return best;
}
// Those of n counted rows: all of the same length but the last, none empty.
__host__ __device__ inline int head_dw_steps(int n, int ranges) {  // 128-row steps of one
  const int deep = n > 128 ? (n + 127) / 128 : 1;
  return (deep + ranges - 1) / ranges;
}

// The dX product's partial sums: of the whole tiles' rows first, where they have any.
__host__ __device__ inline int64_t head_first_sums(int64_t whole, int ranges, int64_t K) {
  return ranges > 1 ? ranges * whole * K : 0;
}
// Room in floats for them: ranges * tiles is at most 4 times the slots, in either pass.
inline size_t head_part_floats(int64_t tb, int64_t K, int tile_rows) {
  const size_t bn = tile_rows, slots = bn == 64 ? kHeadSlots64 : 256;
  const size_t most = 4 * slots * (bn + (bn == 256 ? 128 : 0)) * head_tile_cols(tile_rows);
  const size_t all = kHeadRanges * (size_t)tb * K;
  return all < most ? all : most;
}

hipError_t launch_head_logits(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *Xt, int64_t ldx,
                              const bf16_t *W, int64_t V, int64_t K, float c, float2 *stat, int64_t ntile, bf16_t *E,
                              int64_t lde, int64_t te, int k, int ranges, float *part, hipStream_t s);
// Where the logits came as the partial sums of several ranges: their statistics, E, and the targets' logits.
hipError_t launch_head_soft(const HeadRows &rows, int64_t row0, int64_t tb, const float *part, int ranges, int64_t V,
                            float c, float2 *stat, int64_t ntile, const int32_t *index, int k, bf16_t *E, int64_t lde,
                            int64_t te, hipStream_t s);
hipError_t launch_head_dx(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *E, int64_t lde, int64_t te,
                          const bf16_t *W, int64_t V, int64_t K, const float4 *scale, float *part, bf16_t *dX,
                          hipStream_t s);
hipError_t launch_head_dw(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *E, int64_t lde, int64_t te,
                          const bf16_t *Xs, int64_t V, int64_t K, float *sums, bool first, bool last, int ranges,
                          bf16_t *dW, hipStream_t s);
// dW from the sums of several ranges.
hipError_t launch_head_dw_reduce(const HeadRows &rows, int64_t tb, const float *sums, int ranges, int64_t V, int64_t K,
                                 bf16_t *dW, hipStream_t s);

}  // namespace qlora
