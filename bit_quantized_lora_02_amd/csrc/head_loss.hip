// head_loss.hip -- the row-wise kernels of the output layer's losses: which rows count and their targets' logits
// (k_head_prep, k_head_list), the targets by output tile (k_head_bucket), the statistics of logits that came in ranges
// (k_head_soft), the loss, the row's factor and the targets' gradient (k_head_combine), the factor for dW (k_head_scale,
// k_head_put), and the sums of the dX and dW products' ranges (k_head_reduce, k_head_dw_reduce).
//
// For a row with logits z, targets v_i with probabilities p_i (one target with p = 1: cross entropy), temperature
// tau and c = log2(e) / tau, everything is taken against the first target r (the most probable one):
//   -log q_r = log(sum_v exp((z_v - z_r) / tau)) = log1p(rest),  rest = sum over v != r
//   loss = tau^2 (sum_i p_i (log p_i - (z_i - z_r) / tau) + log1p(rest)),
// which keeps the digits of a loss near zero, where log-sum-exp minus z_r would cancel.  With the row's unit u = z_r,
// E_v = exp2((z_v - u) c) and S = 1 + rest, the gradient by the logits is
//   G_v = w tau (q_v - P_v) = (w tau / S) (E_v - S P_v),   P_v = sum of the p_i whose target is v,
// so the product kernels take E with only the targets' entries replaced by E_v - S P_v (at r: (1 - P_r) - P_r rest,
// again without cancellation), and the row factor w tau / S is applied to dX in binary32 afterwards (dW: see
// k_head_scale).  Entries are rounded to bf16 for the matrix unit; at r, whose entry outweighs the others, dX also gets the
// remainder.
#include <type_traits>

#include "device.h"
#include "head.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kScanRows = 8;  // consecutive rows per thread and pass of the numbering

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}

__device__ __forceinline__ bool target_ok(int64_t v, int64_t V) { return v >= 0 && v < V; }

// Reduction ranges of the dX product, by one wave: `tiles` output tiles of `steps` 64-deep steps on `slots` workgroups
// that run at once, lane s - 1 looking at s ranges.  A round of workgroups costs its steps plus about 10 (first
// loads, output), a 128-row tile's 0.57 of a 256-row one's; more than one range also costs the binary32 partial sums,
// written and read once: about 20 steps' time for 256 tiles of 256 x 256.
struct Split {
  int ranges;
  float cost;  // in steps
};
__device__ __forceinline__ Split wave_split(int tiles, int steps, int tile_rows, int lane) {
  const int s = (lane & (kHeadRanges - 1)) + 1, slots = tile_rows == 64 ? kHeadSlots64 : 256;
  const int rounds = (tiles * s + slots - 1) / slots;
  const float elems = (float)(tile_rows * head_tile_cols(tile_rows));
  float cost = (float)rounds * ((float)steps / (float)s + 10.f) * (tile_rows == 128 ? 0.57f : 1.f) +
               (s > 1 ? 20.f * elems / (256.f * 65536.f) * (float)(tiles * s) : 0.f);
  if (s > 1 && (steps < 8 * s || tiles * s > 4 * slots)) cost = INFINITY;
  Split best = {s, cost};
#pragma unroll
  for (int o = kHeadRanges / 2; o > 0; o >>= 1) {
    const Split other = {__shfl_xor(best.ranges, o), __shfl_xor(best.cost, o)};
    if (other.cost < best.cost || (other.cost == best.cost && other.ranges < best.ranges)) best = other;
  }
  return best;
}

// For n rows: the first of them in tiles of tile_rows, the others in tiles of 128 rows where tile_rows is 256 (the rows
// behind the last whole tile, or, of few tiles, all: 300 x 32000 x 4096 with the sums 120 us in 256-row tiles, 101 in
// 128-row ones), and the ranges of both, all of the same length but the last, none empty (0: no such rows).
__device__ __forceinline__ void dx_ranges(int n, int64_t K, int64_t lde, int tile_rows, int lane, int32_t *out) {
  const int cols = head_tile_cols(tile_rows), tiles_m = (int)((K + cols - 1) / cols), fours = (int)(lde / 128);
  auto split = [&](int rows, int tr) { return wave_split((rows + tr - 1) / tr * tiles_m, fours * 2, tr, lane); };
  Split first = split(n, tile_rows), second = {0, 0.f};
  int whole = n;
  if (tile_rows == 256) {
    const int some = head_whole_rows(n, 256);
    if (some < n && some > 0) {
      const Split a = split(some, 256), b = split(n - some, 128);
      if (a.cost + b.cost < first.cost) first = a, first.cost += b.cost, second = b, whole = some;
    }
    const Split all = split(n, 128);
    if (all.cost < first.cost) first = {0, 0.f}, second = all, whole = 0;
  }
  auto even = [&](int r) {
    const int per = r > 0 ? (fours + r - 1) / r : 1;
    return r > 0 ? (fours + per - 1) / per : 0;
  };
  if (lane == 0) out[0] = even(first.ranges), out[1] = even(second.ranges), out[2] = whole;
}

// s[j] = the sum over r = 0 .. ranges - 1, in order, of p[r * step + j], D of the ranges asked for at a time (FULL: also of
// the last ones, some of them twice).
template <int D, bool FULL, int N>
__device__ __forceinline__ void add_ranges(const float *p, int64_t step, int ranges, float (&s)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = 0.f;
  int r = 0;
  auto add = [&](auto count) {
    constexpr int C = decltype(count)::value;
    float4 a[C][N / 4];
#pragma unroll
    for (int q = 0; q < C; ++q)
#pragma unroll
      for (int j = 0; j < N / 4; ++j)
        a[q][j] = *reinterpret_cast<const float4 *>(p + (FULL ? min(r + q, ranges - 1) : r + q) * step + 4 * j);
#pragma unroll
    for (int q = 0; q < C; ++q)
#pragma unroll
      for (int j = 0; j < N / 4; ++j)
        if (!FULL || r + q < ranges)
          s[4 * j] += a[q][j].x, s[4 * j + 1] += a[q][j].y, s[4 * j + 2] += a[q][j].z, s[4 * j + 3] += a[q][j].w;
    r += C;
  };
  while (r + (FULL ? 1 : D) <= ranges) add(std::integral_constant<int, D>());
  while (r < ranges) add(std::integral_constant<int, 1>());
}

// Of n rows, those that the logit product takes in 256-row tiles, `tiles_m` of the vocabulary; the others go to tiles of
// 128 rows: those behind the last whole tile (see second_pass), or all, where fewer rounds of workgroups at 0.62 of the time
// make up for them (rows that do not count are known only here: 256 of 512 rows x 32000 x 4096 in 125 wide tiles 119 us, in
// 250 narrow ones 104; 240 of 600 x 30000 x 1024 30 and 23).
__device__ __forceinline__ int logit_whole(int n, int tiles_m) {
  const int whole = head_whole_rows(n, 256);
  auto rounds = [](int items, int slots) { return (float)((items + slots - 1) / slots); };
  const int wide = tiles_m * ((whole + 255) / 256), busy = wide % 256;
  float cost = (float)(wide / 256);
  if (whole == n)
    cost += busy > 0 ? 1.f : 0.f;
  else if (busy > 0 && tiles_m <= 2 * (256 - busy))
    cost += fmaxf(1.f, 0.6f * rounds(tiles_m, 256 - busy));
  else
    cost += (busy > 0 ? 1.f : 0.f) + 0.6f * rounds(tiles_m, 256);
  return 0.62f * rounds(tiles_m * ((n + 127) / 128), 256) < cost ? 0 : whole;
}

// Numbers the rows with counts(t), in order, by one workgroup of `threads`; then the blocks' ways through the products.
template <int threads, class Counts>
__device__ __forceinline__ void number_rows(int64_t T, int64_t K, Counts counts, int32_t *__restrict__ n,
                                            int32_t *__restrict__ list, int32_t *__restrict__ ranges,
                                            const HeadBlocks &blocks) {
  __shared__ int s_wave[threads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base = 0;
  for (int64_t t0 = 0; t0 < T; t0 += threads * kScanRows) {
    const int64_t mine = t0 + (int64_t)tid * kScanRows;
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < kScanRows; ++j)
      if (mine + j < T && counts(mine + j)) bits |= 1u << j;
    int before = __popc(bits);  // inclusive sum over the wave, then over the waves
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(before, o);
      if (lane >= o) before += up;
    }
    if (lane == 63) s_wave[wave] = before;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < threads / 64; ++w) {
      if (w < wave) before += s_wave[w];
      total += s_wave[w];
    }
    int at = base + before - __popc(bits);
#pragma unroll
    for (int j = 0; j < kScanRows; ++j)
      if (bits >> j & 1) list[at++] = (int32_t)(mine + j);
    base += total;
    __syncthreads();
  }
  if (tid == 0) *n = base;
  for (int64_t b = wave; b < blocks.count; b += threads / 64) {
    const int64_t row0 = b * blocks.tb, tb = T - row0 < blocks.tb ? T - row0 : blocks.tb;
    const int64_t have = base - row0 < tb ? base - row0 : tb;
    if (have <= 0) continue;
    dx_ranges((int)have, K, blocks.lde, blocks.tile_rows, lane, ranges + 4 * b);
    if (lane == 0) ranges[4 * b + 3] = logit_whole((int)have, (int)((blocks.lde + 255) / 256));
  }
}

// One workgroup's counting sort of a row tile's targets by output tile of the logit product: `have` rows of the block's
// list from `first`, into rows.bucket and rows.target at row tile `tile`.  (The order within an output tile is that of
// the LDS counters; every target's logit goes to a place of its own, so no result depends on it.)
template <int threads>
__device__ __forceinline__ void sort_targets(const HeadRows &rows, int64_t tile, int64_t first, int have, int tile_rows,
                                             int tile_cols, int ntile, const int32_t *__restrict__ index, int k,
                                             int64_t V, int *s_count /* [ntile] */) {
  __shared__ int s_sum[threads / 64], s_row[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < have; i += threads) s_row[i] = ((volatile const int32_t *)rows.list)[first + i];
  have *= k;
  for (int i = tid; i < ntile; i += threads) s_count[i] = 0;
  __syncthreads();
  const uint32_t per_k = 0xffffffffu / (uint32_t)k + 1;  // e / k = e per_k / 2^32 for e < 2^16 (k = 1: per_k = 0)
  auto each = [&](auto use) {
#pragma unroll 8
    for (int e = tid; e < have; e += threads) {
      const int nj = k == 1 ? e : (int)__umulhi((uint32_t)e, per_k), j = e - nj * k;
      const int64_t v = index[(int64_t)s_row[nj] * k + j];
      if (target_ok(v, V)) use((int)v, nj, j);
    }
  };
  each([&](int v, int, int) { atomicAdd(&s_count[v / tile_cols], 1); });
  __syncthreads();
  // exclusive sums over the tiles, a run of `per` of them per thread
  const int per = (ntile + threads - 1) / threads, i0 = tid * per;
  int mine = 0;
  for (int i = i0; i < i0 + per && i < ntile; ++i) mine += s_count[i];
  int before = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(before, o);
    if (lane >= o) before += up;
  }
  if (lane == 63) s_sum[wave] = before;
  __syncthreads();
  for (int w = 0; w < wave; ++w) before += s_sum[w];
  int at = before - mine;
  int32_t *bucket = rows.bucket + tile * (ntile + 1);
  for (int i = i0; i < i0 + per && i < ntile; ++i) {
    const int c = s_count[i];
    bucket[i] = s_count[i] = at;
    at += c;
  }
  if (i0 < ntile && i0 + per >= ntile) bucket[ntile] = at;
  __syncthreads();
  uint32_t *target = rows.target + tile * tile_rows * k;
  each([&](int v, int nj, int j) {
    target[atomicAdd(&s_count[v / tile_cols], 1)] = (uint32_t)j | (uint32_t)(v % tile_cols) << 8 | (uint32_t)nj << 16;
  });
}

// Workgroup 0 numbers the rows that count: with labels, or where the teacher's targets are few (head_few_targets), which
// it then also sorts; k_head_list and k_head_bucket do it otherwise.  The other workgroups' waves take a row of X each:
// its first target (the label, or the teacher's most probable one; the first of equals) and that target's logit by a
// dot product (binary32 FMA), the teacher's softmax, and the row in the blocks of 32 columns that the logit product
// reads (zeros past K); or, for a row that does not count, its zero loss and gradient.  Bound by its loads: 4096 x 4096
// 24 us (X, the targets' rows of W and the copy, 4.2 TB/s), a single row 4.
__global__ __launch_bounds__(kPrepThreads) void k_head_prep(const bf16_t *__restrict__ X, int64_t T,
                                                            const bf16_t *__restrict__ W, int64_t V, int64_t K,
                                                            const int64_t *__restrict__ labels,
                                                            const int32_t *__restrict__ index,
                                                            const float *__restrict__ logit, int k, float tau,
                                                            int32_t *n, int32_t *list, int32_t *__restrict__ ranges,
                                                            HeadBlocks blocks, HeadRows rows, int tile_cols, int ntile,
                                                            float *__restrict__ loss, bf16_t *__restrict__ dX,
                                                            bf16_t *__restrict__ Xt, int64_t ldx) {
  extern __shared__ int s_count[];  // [ntile] where workgroup 0 sorts the targets
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x == 0) {
    if (labels) {
      number_rows<kPrepThreads>(T, K, [&](int64_t t) { return target_ok(labels[t], V); }, n, list, ranges, blocks);
    } else if (head_few_targets(T, k, blocks.tile_rows)) {
      __shared__ int s_counts[256];  // (the most rows of a tile)
      for (int t = tid; t < T; t += kPrepThreads) s_counts[t] = 0;
      __syncthreads();
#pragma unroll 4
      for (int e = tid; e < (int)T * k; e += kPrepThreads)
        if (target_ok(index[e], V) && logit[e] != -INFINITY) s_counts[e / k] = 1;
      __syncthreads();
      number_rows<kPrepThreads>(T, K, [&](int64_t t) { return s_counts[t] != 0; }, n, list, ranges, blocks);
      __syncthreads();
      if (rows.target)
        sort_targets<kPrepThreads>(rows, 0, 0, *(volatile const int32_t *)n, blocks.tile_rows, tile_cols, ntile, index, k,
                                   V, s_count);
    }
    return;
  }
  const int64_t t = (int64_t)(blockIdx.x - 1) * (kPrepThreads / 64) + wave;
  if (t >= T) return;
  int64_t y;
  if (labels) {
    y = labels[t];
    if (!target_ok(y, V)) y = -1;
  } else {  // the teacher's softmax over the row's targets, up to four per lane (NaN is taken for +inf: either counts and
            // leaves the row's probabilities NaN)
    float tl[4], top = -INFINITY;
    int id[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = lane + 64 * j;
      id[j] = i < k ? index[t * k + i] : -1;
      tl[j] = target_ok(id[j], V) ? logit[t * k + i] : -INFINITY;
      if (tl[j] != tl[j]) tl[j] = INFINITY;
      top = fmaxf(top, tl[j]);
    }
    top = wave_max(top);
    int first = 256;
    float e[4], sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      e[j] = tl[j] == -INFINITY ? 0.f : expf((tl[j] - top) / tau);
      sum += e[j];
      if (tl[j] == top) first = min(first, lane + 64 * j);
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) first = min(first, __shfl_xor(first, o));
    y = -1;
    if (top > -INFINITY) {
      y = index[t * k + first];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (lane + 64 * j < k) rows.pt[t * k + lane + 64 * j] = e[j] / sum;
    }
  }
  if (y < 0) {
    if (lane == 0) {
      loss[t] = 0.f;
      rows.refcol[t] = -1;
    }
    if (dX)
      for (int64_t at = 8 * lane; at < K; at += 512)
        *reinterpret_cast<u32x4_t *>(dX + t * K + at) = u32x4_t{0u, 0u, 0u, 0u};
    return;
  }
  const bf16_t *x = X + t * K, *w = W + y * K;
  float z = 0.f;
  const int64_t end = (K + 127) / 128 * 128;
  auto dot = [&](auto deep) {  // `deep` pieces of 512 columns asked for before the first is used
    constexpr int D = decltype(deep)::value;
    for (int64_t at0 = 8 * lane; at0 < end; at0 += 512 * D) {
      u32x4_t xv[D], wv[D];
#pragma unroll
      for (int q = 0; q < D; ++q) {
        const int64_t at = at0 + 512 * q, from = at < K ? at : 0;
        xv[q] = *reinterpret_cast<const u32x4_t *>(x + from);
        wv[q] = *reinterpret_cast<const u32x4_t *>(w + from);
      }
#pragma unroll
      for (int q = 0; q < D; ++q) {
        const int64_t at = at0 + 512 * q;
        if (at >= K) xv[q] = wv[q] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z = fmaf(bf16_lo_to_f32(xv[q][e]), bf16_lo_to_f32(wv[q][e]), z);
          z = fmaf(bf16_hi_to_f32(xv[q][e]), bf16_hi_to_f32(wv[q][e]), z);
        }
        if (at < end) *reinterpret_cast<u32x4_t *>(Xt + (at / 32 * ldx + t) * 32 + at % 32) = xv[q];
      }
    }
  };
  // (short rows ask for no more than they have: 5719 x 456 took 12.7 us with eight pieces, 8.9 with two; a single row of
  // 4096 5.7 us with four, 4.1 with eight)
  if (end <= 1024)
    dot(std::integral_constant<int, 2>());
  else
    dot(std::integral_constant<int, 8>());
  z = wave_sum(z);
  if (lane == 0) {
    rows.ref[t] = z;
    rows.refcol[t] = (int32_t)y;
  }
}

// Numbers the rows whose first target k_head_prep found, by one workgroup: 4096 rows 8 us.
constexpr int kListThreads = 1024;
__global__ __launch_bounds__(kListThreads) void k_head_list(int64_t T, int64_t K, const int32_t *__restrict__ refcol,
                                                            int32_t *__restrict__ n, int32_t *__restrict__ list,
                                                            int32_t *__restrict__ ranges, HeadBlocks blocks) {
  number_rows<kListThreads>(T, K, [&](int64_t t) { return refcol[t] >= 0; }, n, list, ranges, blocks);
}

// One workgroup per tile of rows of the block: 4096 rows of 64 targets 20 to 26 us (by the clock), of
// latency, beside products of 6200.
constexpr int kBucketThreads = 1024;
__global__ __launch_bounds__(kBucketThreads) void k_head_bucket(HeadRows rows, int64_t row0, int64_t tb, int tile_cols,
                                                                int ntile, const int32_t *__restrict__ index, int k,
                                                                int64_t V) {
  extern __shared__ int s_count[];  // [ntile]
  int64_t n = *rows.n - row0;
  n = n < tb ? n : tb;
  const int64_t n0 = (int64_t)blockIdx.x * rows.tile_rows;
  if (n0 >= n) return;
  sort_targets<kBucketThreads>(rows, blockIdx.x, row0 + n0, (int)(n - n0 < rows.tile_rows ? n - n0 : rows.tile_rows),
                               rows.tile_rows, tile_cols, ntile, index, k, V, s_count);
}

// A workgroup per counted row and 2048 columns: z from the ranges' sums, in order, then what the product's epilogue does
// with it (see logit_items), a lane taking eight columns.
// (Only narrow tiles' reductions are split: every entry of the statistics is of kHeadStat columns.)  Bound by the sums'
// read: 1910 x 1890 in two ranges 8.5 us, launch included.
__global__ __launch_bounds__(256) void k_head_soft(HeadRows rows, int64_t row0, int64_t tb,
                                                   const float *__restrict__ part, int ranges, int64_t V, float c,
                                                   float2 *__restrict__ stat, int64_t ntile,
                                                   const int32_t *__restrict__ index, int k, bf16_t *__restrict__ E,
                                                   int64_t lde, int64_t te) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t i = blockIdx.x;
  int64_t n = *rows.n - row0;
  n = n < tb ? n : tb;
  if (i >= n) return;
  const int64_t t = rows.list[row0 + i];
  const float ref = rows.ref[t], uc = ref * c;
  const int rc = rows.refcol[t];
  const float *const p = part + i * lde;
  for (int j = tid; blockIdx.y == 0 && j < k; j += 256) {
    const int64_t v = index[t * k + j];
    float z = 0.f;
    if (target_ok(v, V))
#pragma unroll 4
      for (int r = 0; r < ranges; ++r) z += p[(int64_t)r * n * lde + v];
    rows.zt[t * k + j] = z;
  }
  const int64_t v = ((int64_t)blockIdx.y * 256 + tid) * 8;
  const bool in = v < lde;  // lde % 128 == 0: a group's lanes are all in or all out
  float z[8], e[8], sum = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) z[q] = 0.f;
  if (in) add_ranges<4, false>(p + v, n * lde, ranges, z);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (!in || v + q >= V || v + q == rc) z[q] = -INFINITY;
    e[q] = __builtin_amdgcn_exp2f(fmaf(z[q], c, -uc));
    sum += e[q];
  }
  for (int o = 1; o < kHeadStat / 8; o <<= 1) sum += __shfl_xor(sum, o);
  float u = ref;
  const bool over = !(sum < kHeadRange);
  if (__any(over)) {
    float top = z[0];
#pragma unroll
    for (int q = 1; q < 8; ++q) top = fmaxf(top, z[q]);
    for (int o = 1; o < kHeadStat / 8; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    u = over ? top : ref;
    sum = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      e[q] = __builtin_amdgcn_exp2f((z[q] - u) * c);
      sum += e[q];
    }
    for (int o = 1; o < kHeadStat / 8; o <<= 1) sum += __shfl_xor(sum, o);
  }
  if (v < V && lane % (kHeadStat / 8) == 0) stat[i * ntile + v / kHeadStat] = make_float2(u, sum);
  if (E && in)
    *reinterpret_cast<u32x4_t *>(E + (v / 32 * te + i) * 32 + v % 32) =
        u32x4_t{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7])};
}

// One wave per counted row of the block.  Bound by latency: 3686 rows of a 128256-wide vocabulary 14 us, with 64 targets
// each 27.
__global__ __launch_bounds__(256) void k_head_combine(HeadRows rows, int64_t row0, int64_t tb,
                                                      const float2 *__restrict__ stat, int64_t ntile, int64_t V,
                                                      const int64_t *__restrict__ labels,
                                                      const int32_t *__restrict__ index, int k, float tau,
                                                      const float *__restrict__ weight, float *__restrict__ loss,
                                                      float4 *__restrict__ scale, bf16_t *__restrict__ E, int64_t lde,
                                                      int64_t te, const bf16_t *__restrict__ X, int64_t K,
                                                      bf16_t *__restrict__ Xs) {
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // row of the block
  int64_t n = *rows.n - row0;
  n = n < 0 ? 0 : n < tb ? n : tb;
  if (i >= n) {  // the dW product's steps go to the next 128 rows (at least one such group)
    if (Xs && i < (n > 0 ? (n + 127) / 128 * 128 : 128)) {
      for (int64_t at = 8 * lane; at < K; at += 512)
        *reinterpret_cast<u32x4_t *>(Xs + i * K + at) = u32x4_t{0u, 0u, 0u, 0u};
      if (n == 0 && i == 0)
        for (int64_t v = 8 * lane; v < lde; v += 512)
          *reinterpret_cast<u32x4_t *>(E + (v / 32 * te) * 32 + v % 32) = u32x4_t{0u, 0u, 0u, 0u};
    }
    return;
  }
  const int64_t t = rows.list[row0 + i];
  const float ref = rows.ref[t], c = 1.44269504f / tau;
  const float2 *st = stat + i * ntile;
  const int stat_cols = head_stat_cols(rows.tile_rows == 256 && i < rows.ranges[3]);
  const int entries = (int)((V + stat_cols - 1) / stat_cols);
  float u = ref, sum = 0.f;
#pragma unroll 4
  for (int j = lane; j < entries; j += 64) {
    const float2 v = st[j];
    u = fmaxf(u, v.x);
    // (units are the reference or above it, but where the columns hold a NaN: theirs is the largest of the others, their sum
    // NaN, and the row's loss and gradients are to be)
    sum += v.x > ref ? 0.f : v.y;
  }
  u = wave_max(u);
  float S, eref = 1.f, rest, nlogq;
  const bool wide = u != ref;  // some tile's logits are far above the reference: the row takes the largest unit
  if (!wide) {
    rest = ref == INFINITY ? NAN : wave_sum(sum);  // (against +inf every finite logit's term is 0)
    nlogq = log1pf(rest);
  } else {
    sum = 0.f;
    for (int j = lane; j < entries; j += 64) sum += st[j].y * exp2f((st[j].x - u) * c);
    rest = wave_sum(sum);
    eref = exp2f((ref - u) * c);
    nlogq = logf(rest + eref) + (u - ref) / tau;
  }
  S = rest + eref;
  const int32_t rc = rows.refcol[t];
  // sum_i p_i (log p_i - (z_i - z_r) / tau).  At the first target's column z_i is z_r, though the product's and the dot's
  // sums of it differ in their last places, which would outweigh the loss of a sure row.
  float h = 0.f;
  if (!labels)
    for (int j = lane; j < k; j += 64) {
      const float p = rows.pt[t * k + j];
      const float z = index[t * k + j] == rc ? 0.f : (rows.zt[t * k + j] - ref) / tau;
      if (p != 0.f) h += p * (logf(p) - z);
    }
  h = wave_sum(h);
  if (lane == 0) loss[t] = tau * tau * (h + nlogq);
  if (!E) return;
  auto e = [&](int64_t v) { return E + (v / 32 * te + i) * 32 + v % 32; };
  if (wide) {  // bring the row's tiles to one unit (a factor below binary32's range is applied in two halves)
    for (int64_t at = 8 * lane; at < lde; at += 512) {
      const float d = exp2f(0.5f * (st[min(at / stat_cols, (int64_t)entries - 1)].x - u) * c);
      u32x4_t v = *reinterpret_cast<u32x4_t *>(e(at));
#pragma unroll
      for (int w = 0; w < 4; ++w) v[w] = pack_bf16x2(bf16_lo_to_f32(v[w]) * d * d, bf16_hi_to_f32(v[w]) * d * d);
      *reinterpret_cast<u32x4_t *>(e(at)) = v;
    }
    __threadfence_block();  // the targets' entries below follow these stores
  }
  const float f = (weight ? weight[t] : 1.f) * tau / S;
  // The first target's entry is the row's largest as a rule; what its rounding to bf16 leaves goes to dX in binary32.
  int ex;
  const float fm = frexpf(f, &ex);
  auto first_target = [&](float g) {
    const bf16_t r = f32_to_bf16(g);
    *e(rc) = r;
    scale[i] = make_float4(f, g - bf16_lo_to_f32(r), fm, __int_as_float(rc));
  };
  if (labels) {
    if (lane == 0) first_target(-rest);
  } else {
    for (int i0 = 0; i0 < k; i0 += 64) {
      const int me = i0 + lane;
      const int32_t v = me < k ? index[t * k + me] : -1;
      float P = 0.f;  // all of the row's probability at this column
      for (int j0 = 0; j0 < k; j0 += 64) {
        const int32_t vj = j0 + lane < k ? index[t * k + j0 + lane] : -1;
        const float pj = j0 + lane < k ? rows.pt[t * k + j0 + lane] : 0.f;
        for (int j = 0; j < min(64, k - j0); ++j)
          if (__builtin_amdgcn_readlane(vj, j) == v)
            P += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(pj), j));
      }
      if (!target_ok(v, V)) continue;
      const float g = v == rc ? eref * (1.f - P) - P * rest : exp2f((rows.zt[t * k + me] - u) * c) - P * S;
      if (v == rc)
        first_target(g);
      else
        *e(v) = f32_to_bf16(g);
      rows.zt[t * k + me] = g;  // for k_head_put
    }
  }
  if (Xs)  // rows of X times the row factor's power of two, exactly (k_head_scale gives E the rest of the factor)
    for (int64_t at0 = 8 * lane; at0 < K; at0 += 512 * 4) {
      u32x4_t v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = *reinterpret_cast<const u32x4_t *>(X + t * K + (at0 + 512 * q < K ? at0 + 512 * q : 0));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
          v[q][w] = pack_bf16x2(ldexpf(bf16_lo_to_f32(v[q][w]), ex), ldexpf(bf16_hi_to_f32(v[q][w]), ex));
        if (at0 + 512 * q < K) *reinterpret_cast<u32x4_t *>(Xs + i * K + at0 + 512 * q) = v[q];
      }
    }
}

// E's rows times the fraction (in [1/2, 1)) of their factors, for dW, whose reduction runs over the rows, so that no
// factor can wait for the product's epilogue.  (Rounding X times the factor instead would round every term of a row of
// dW twice; here the first target's entry, which outweighs the others, is rounded once, from its value with the
// remainder, and k_head_put does the same for a teacher's other targets.  dW's error against 64 bits falls from 2.9e-3 to
// 2.3e-3 of its norm.)  Bound by E's read and write: 1843 x 32000 40 us, 5.9 TB/s.  A thread takes eight columns of a row
// in each of kScaleBlocks blocks.
constexpr int kScaleBlocks = 8;
__global__ __launch_bounds__(256) void k_head_scale(HeadRows rows, int64_t row0, int64_t tb,
                                                    const float4 *__restrict__ scale, bf16_t *__restrict__ E,
                                                    int64_t lde, int64_t te) {
  int64_t n = *rows.n - row0;
  n = n < tb ? n : tb;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, i = at >> 2;
  if (i >= n) return;
  const float4 f = scale[i];
  const int rc = __float_as_int(f.w), col = (int)(at & 3) * 8;
  const int64_t b0 = (int64_t)blockIdx.y * kScaleBlocks, blocks = lde / 32;
#pragma unroll
  for (int b = 0; b < kScaleBlocks; ++b) {
    if (b0 + b >= blocks) break;
    u32x4_t *const p = reinterpret_cast<u32x4_t *>(E + ((b0 + b) * te + i) * 32 + col);
    const u32x4_t v = *p;
    float x[8];
#pragma unroll
    for (int w = 0; w < 4; ++w) x[2 * w] = bf16_lo_to_f32(v[w]), x[2 * w + 1] = bf16_hi_to_f32(v[w]);
    const int mine = rc - (int)(b0 + b) * 32 - col;
#pragma unroll
    for (int w = 0; w < 8; ++w) x[w] = (mine == w ? x[w] + f.y : x[w]) * f.z;
    *p = u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  }
}

// The targets' entries once more after k_head_scale, rounded once from what k_head_combine kept of them.
__global__ __launch_bounds__(256) void k_head_put(HeadRows rows, int64_t row0, int64_t tb, int64_t V,
                                                  const int32_t *__restrict__ index, int k,
                                                  const float4 *__restrict__ scale, bf16_t *__restrict__ E, int64_t te) {
  int64_t n = *rows.n - row0;
  n = n < tb ? n : tb;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, i = at / k;
  if (i >= n) return;
  const int64_t e = (int64_t)rows.list[row0 + i] * k + (at - i * k);
  const int64_t v = index[e];
  if (target_ok(v, V)) E[(v / 32 * te + i) * 32 + v % 32] = f32_to_bf16(rows.zt[e] * scale[i].z);
}

// dX rows of the block from the ranges' partial sums part[range][row][K], added in range order, and the first target's
// remainder, N columns a thread, D ranges in flight.  Bound by the sums' read: 1838 x 4096 in two ranges 19 us (with four
// columns a thread 24).  Few rows come in many ranges and have few threads: 17 x 2048 in 32 ranges 5.1 us with four
// columns and 16 ranges in flight, 6.7 with eight and four.
template <int N, int D>
__global__ __launch_bounds__(256) void k_head_reduce(HeadRows rows, int64_t row0, int64_t tb,
                                                     const float *__restrict__ part, const bf16_t *__restrict__ W,
                                                     int64_t K, const float4 *__restrict__ scale,
                                                     bf16_t *__restrict__ dX) {
  int64_t n = *rows.n - row0;
  n = n < tb ? n : tb;
  if (n <= 0) return;
  const int64_t per = K / N, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= n * per) return;
  const int64_t i = at / per, col = (at % per) * N;
  const int whole = rows.ranges[2];
  const bool second = i >= whole;
  const int ranges = rows.ranges[second];
  if (ranges == 1) return;  // the product wrote dX itself
  const float *p = part + (second ? head_first_sums(whole, rows.ranges[0], K) : 0);
  const int64_t count = second ? n - whole : whole;
  float v[N];
  add_ranges<D, D == 16>(p + (second ? i - whole : i) * K + col, count * K, ranges, v);
  const float4 f = scale[i];
  const int64_t t = rows.list[row0 + i];
  typedef uint32_t word_t __attribute__((ext_vector_type(N / 2)));
  const word_t wv = *reinterpret_cast<const word_t *>(W + rows.refcol[t] * K + col);
  word_t o;
#pragma unroll
  for (int w = 0; w < N / 2; ++w)
    o[w] = pack_bf16x2(fmaf(f.y, bf16_lo_to_f32(wv[w]), v[2 * w]) * f.x,
                       fmaf(f.y, bf16_hi_to_f32(wv[w]), v[2 * w + 1]) * f.x);
  *reinterpret_cast<word_t *>(dX + t * K + col) = o;
}

// dW from the ranges' partial sums [range][V][K], in range order.  Bound by their read: 2000 x 504 in eight ranges 6 us.
__global__ __launch_bounds__(256) void k_head_dw_reduce(HeadRows rows, int64_t tb, const float *__restrict__ part,
                                                        int ranges, int64_t count, bf16_t *__restrict__ dW) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= count) return;
  const int n = min(*rows.n, (int)tb), per = head_dw_steps(n, ranges);
  float v[8];
  add_ranges<4, false>(part + at, count, (max((n + 127) / 128, 1) + per - 1) / per, v);
  *reinterpret_cast<u32x4_t *>(dW + at) = u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

}  // namespace

hipError_t launch_head_prep(const bf16_t *X, int64_t T, const bf16_t *W, int64_t V, int64_t K, const int64_t *labels,
                            const int32_t *index, const float *logit, int k, float tau, int32_t *n, int32_t *list,
                            int32_t *ranges, const HeadBlocks &blocks, const HeadRows &rows, float *loss, bf16_t *dX,
                            bf16_t *Xt, int64_t ldx, hipStream_t s) {
  const int64_t wgs = (T + kPrepThreads / 64 - 1) / (kPrepThreads / 64);
  const int tc = head_tile_cols(blocks.tile_rows), ntile = (int)((V + tc - 1) / tc);
  const bool sorts = rows.target && head_few_targets(T, k, blocks.tile_rows);
  launch(k_head_prep, dim3((unsigned)(1 + wgs)), dim3(kPrepThreads), sorts ? (uint32_t)ntile * 4 : 0u, s, X, T, W, V, K,
         labels, index, logit, k, tau, n, list, ranges, blocks, rows, tc, ntile, loss, dX, Xt, ldx);
  return hipGetLastError();
}

hipError_t launch_head_list(const HeadRows &rows, int64_t T, int64_t K, int32_t *n, int32_t *list, int32_t *ranges,
                            const HeadBlocks &blocks, hipStream_t s) {
  launch(k_head_list, dim3(1), dim3(kListThreads), 0, s, T, K, (const int32_t *)rows.refcol, n, list, ranges, blocks);
  return hipGetLastError();
}

hipError_t launch_head_bucket(const HeadRows &rows, int64_t row0, int64_t tb, const int32_t *index, int k, int64_t V,
                              hipStream_t s) {
  const int tr = rows.tile_rows, tc = head_tile_cols(tr);
  const int64_t ntile = (V + tc - 1) / tc;
  launch(k_head_bucket, dim3((unsigned)((tb + tr - 1) / tr)), dim3(kBucketThreads), (uint32_t)ntile * 4, s, rows, row0,
         tb, tc, (int)ntile, index, k, V);
  return hipGetLastError();
}

hipError_t launch_head_soft(const HeadRows &rows, int64_t row0, int64_t tb, const float *part, int ranges, int64_t V,
                            float c, float2 *stat, int64_t ntile, const int32_t *index, int k, bf16_t *E, int64_t lde,
                            int64_t te, hipStream_t s) {
  launch(k_head_soft, dim3((unsigned)tb, (unsigned)((lde + 2047) / 2048)), dim3(256), 0, s, rows, row0, tb, part, ranges,
         V, c, stat, ntile, index, k, E, lde, te);
  return hipGetLastError();
}

hipError_t launch_head_combine(const HeadRows &rows, int64_t row0, int64_t tb, const float2 *stat, int64_t ntile,
                               int64_t V, const int64_t *labels, const int32_t *index, int k, float tau,
                               const float *weight, float *loss, float4 *scale, bf16_t *E, int64_t lde, int64_t te,
                               const bf16_t *X, int64_t K, bf16_t *Xs, hipStream_t s) {
  const int64_t grid_rows = Xs ? (tb > 0 ? (tb + 127) / 128 * 128 : 128) : tb;
  launch(k_head_combine, dim3((unsigned)((grid_rows + 3) / 4)), dim3(256), 0, s, rows, row0, tb,
         stat, ntile, V, labels, index, k, tau, weight, loss, scale, E, lde, te, X, K, Xs);
  return hipGetLastError();
}

hipError_t launch_head_reduce(const HeadRows &rows, int64_t row0, int64_t tb, const float *part, const bf16_t *W,
                              int64_t K, const float4 *scale, bf16_t *dX, hipStream_t s) {
  const bool few = rows.tile_rows == 64;
  const int64_t threads = tb * (K / (few ? 4 : 8));
  launch(few ? k_head_reduce<4, 16> : k_head_reduce<8, 4>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, rows,
         row0, tb, part, W, K, scale, dX);
  return hipGetLastError();
}

hipError_t launch_head_dw_reduce(const HeadRows &rows, int64_t tb, const float *sums, int ranges, int64_t V, int64_t K,
                                 bf16_t *dW, hipStream_t s) {
  launch(k_head_dw_reduce, dim3((unsigned)((V * K / 8 + 255) / 256)), dim3(256), 0, s, rows, tb, sums, ranges, V * K, dW);
  return hipGetLastError();
}

hipError_t launch_head_put(const HeadRows &rows, int64_t row0, int64_t tb, int64_t V, const int32_t *index, int k,
                           const float4 *scale, bf16_t *E, int64_t te, hipStream_t s) {
  launch(k_head_put, dim3((unsigned)((tb * k + 255) / 256)), dim3(256), 0, s, rows, row0, tb, V, index, k, scale, E, te);
  return hipGetLastError();
}

hipError_t launch_head_scale(const HeadRows &rows, int64_t row0, int64_t tb, const float4 *scale, bf16_t *E, int64_t lde,
                             int64_t te, hipStream_t s) {
  const int64_t blocks = (lde / 32 + kScaleBlocks - 1) / kScaleBlocks;
  launch(k_head_scale, dim3((unsigned)((tb * 4 + 255) / 256), (unsigned)blocks), dim3(256), 0, s, rows, row0, tb, scale, E,
         lde, te);
  return hipGetLastError();
}

}  // namespace qlora
