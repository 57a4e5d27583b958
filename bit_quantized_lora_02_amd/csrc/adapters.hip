// adapters.hip -- low-rank adapters of many requests beside a shared projection, each token with an adapter of its own.
//
//   u_t  = X_t A_a^T,              Y_t  = bf16(base_t + s_a u_t B_a^T)        a = index[t]
//   du_t = s_a dY_t B_a,           dX_t = bf16(base_t + du_t A_a)
//   dA_a = sum_t du_t^T X_t,       dB_a = s_a sum_t dY_t^T u_t               over the tokens of adapter a
//
// ("QLoRA: fine-tuning a large model on one GPU" (learn.pranaymahendrakar.com), Researcher level, "LoRA, stated once" and
// "The variants worth knowing": one base model in memory, requests for different adapters batched together.)
// The floor is the traffic of X, Y and the adapters in use: about r operations per byte, so that the products, at a library
// product's rate, take a quarter of its time at rank 64 and less below (backward of 8000 tokens, 4096 x 4096: 12 of 53 us; at
// rank 128 24 of 58).  So each product streams its long operand once, and the rank-wide results u and du stay in binary32:
// where one of them is an operand it enters as two bf16 parts (16 bits of it).  That is a second MFMA (the products above take
// 21 and 42 us with it) and leaves the outputs with the one rounding of their type: they are as far from the 64-bit values as
// with u whole (1.66e-3 of their norm), and from those outputs 1.1e-4 of it or less, entries that round the other way.
//   1. k_adapt_plan    groups the tokens by adapter (stably), a workgroup for 8192 of them (more, which k_adapt_count counts
//                      before); other workgroups transpose the pools for the backward.  Up to kAdaptSmall tokens in the
//                      forward, the next kernels find their tokens themselves.
//   2. k_adapt_shrink  u or du: 16 or 32 tokens of one adapter against its r rows, the long axis over 8 waves (and ranges
//                      of it over workgroups where there are few tokens).
//   3. k_adapt_expand  base + u B^T (or du A): 16 or 32 tokens of one adapter, 128 columns at a time.
//   4. k_adapt_grads   dA and dB: a piece of an adapter's tokens, 64 columns; transposed operands through LDS.
//   5. k_adapt_reduce  sums of the pieces, in order.
// No kernel writes a value in more than one place or adds atomically: results repeat bit by bit.
#include "step.h"
#include "step_device.h"

namespace qlora {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// 16x16x32: lane l holds A[m = l%16][k = 8(l/16)..+7], B[k = 8(l/16)..+7][n = l%16], C[m = 4(l/16)+i][n = l%16].
__device__ __forceinline__ f32x4_t mfma16(const u32x4_t &a, const u32x4_t &b, const f32x4_t &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0,
                                                 0);
}

__device__ __forceinline__ int scan_dpp(int x) {  // inclusive sums over the wave's lanes
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, true);
  return x;
}

// Group of a token (n_pool: none).
__device__ __forceinline__ int group_of(const AdaptRows &a, int64_t t) {
  const int k = a.index[t];
  return (uint32_t)k < (uint32_t)a.n_pool ? k : a.n_pool;
}
__device__ __forceinline__ int rank_of(const AdaptRows &a, int group) {
  if (group >= a.n_pool) return 0;
  if (!a.rank) return a.r;
  const int k = a.rank[group];
  return k < 0 ? 0 : k > a.r ? a.r : k;
}

// A wave's stores to its own part of LDS, then its other lanes' loads from it (or the other way round): the LDS serves a
// wave in order, so this only keeps the compiler to it.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Lanes whose number is this lane's, by a vote on each of its bits.
__device__ __forceinline__ uint64_t same_lanes(int number, int bits) {
  uint64_t m = ~(uint64_t)0;
  for (int b = 0; b < bits; ++b) {
    const bool one = (number >> b) & 1;
    const uint64_t vote = __ballot(one);
    m &= one ? vote : ~vote;
  }
  return m;
}

// At most M tokens of one group: places p0 .. p0 + n - 1 of the order.  Of a group that is cut into several tiles, `slot`
// numbers them over all such groups (-1: the group's only tile).
struct Tile {
  int group, p0, n, slot;
};
// The id-th tile of the groups in order (wave-wide, the same in every lane); false: there are fewer.  POOL: of the
// adapters' groups alone, and one without tokens has a tile too.
template <bool POOL>
__device__ __forceinline__ bool find_tile(const AdaptRows &a, int M, int id, Tile *out) {
  const int lane = threadIdx.x & 63;
  int before = 0, slots = 0;
  for (int k0 = 0; k0 <= a.n_pool; k0 += 64) {
    const int k = k0 + lane;
    int lo = 0, hi = 0;
    const bool there = POOL ? k < a.n_pool : k <= a.n_pool;
    if (there) lo = a.start[k], hi = a.start[k + 1];
    const int tiles = POOL && there && hi == lo ? 1 : (hi - lo + M - 1) / M, several = tiles > 1 ? tiles : 0;
    const int sum = scan_dpp(tiles), sum2 = scan_dpp(several);
    const int all = __builtin_amdgcn_readlane(sum, 63);
    if (id < before + all) {
      const int l = __builtin_ctzll(__ballot(before + sum > id));
      const int j = id - (before + __builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(tiles, l));
      const int end = __builtin_amdgcn_readlane(hi, l), n_tiles = __builtin_amdgcn_readlane(tiles, l);
      out->group = k0 + l;
      out->p0 = __builtin_amdgcn_readlane(lo, l) + j * M;
      out->n = end - out->p0 < M ? end - out->p0 : M;
      out->slot = n_tiles > 1 ? slots + __builtin_amdgcn_readlane(sum2, l) - n_tiles + j : -1;
      return true;
    }
    before += all;
    slots += __builtin_amdgcn_readlane(sum2, 63);
  }
  return false;
}

// The id-th tile of M tokens and this lane's token in it, place lane % M (behind the tile's end: its first token).
// Without a plan (T <= 64) the groups come in the order of their first tokens.
template <int M>
__device__ __forceinline__ bool find_tokens(const AdaptRows &a, int id, Tile *tile, int tokens[(M + 15) / 16]) {
  const int lane = threadIdx.x & 63;
  if (a.start) {
    if (!find_tile<false>(a, M, id, tile)) return false;
#pragma unroll
    for (int m = 0; m < (M + 15) / 16; ++m) {
      const int p = m * 16 + (lane & 15);
      tokens[m] = a.order[tile->p0 + (p < tile->n ? p : 0)];
    }
    return true;
  }
  // (the lanes of a group by a vote per bit of its number; its first lane counts its tiles)
  const int groups = a.n_pool + 1, group = lane < a.T ? group_of(a, lane) : groups;
  const uint64_t same = same_lanes(group, 32 - __builtin_clz(groups)), before = ((uint64_t)1 << lane) - 1;
  const int count = __popcll(same);
  const int tiles = lane < a.T && (same & before) == 0 ? (count + M - 1) / M : 0, sum = scan_dpp(tiles);
  const uint64_t at = __ballot(sum > id);
  if (at == 0) return false;
  const int lead = __builtin_ctzll(at), n = __builtin_amdgcn_readlane(count, lead);
  const int j = id - (__builtin_amdgcn_readlane(sum, lead) - __builtin_amdgcn_readlane(tiles, lead));
  tile->group = __builtin_amdgcn_readlane(group, lead);
  tile->p0 = j * M;
  tile->n = n - j * M < M ? n - j * M : M;
  tile->slot = -1;
  // the group's lanes go to the front, in order, and each lane takes its token from there
  const bool mine = group == tile->group;
  const uint64_t all = __ballot(mine);
  const int to = mine ? __popcll(all & before) : n + __popcll(~all & before);
  const int sorted = __builtin_amdgcn_ds_permute(to * 4, lane);
#pragma unroll
  for (int m = 0; m < (M + 15) / 16; ++m) {
    const int p = m * 16 + (lane & 15);
    tokens[m] = __builtin_amdgcn_ds_bpermute((tile->p0 + (p < tile->n ? p : 0)) * 4, sorted);
  }
  return true;
}

// u as two bf16 parts, hi + lo (16 bits of it).  The high part stays in bf16's range, so that an infinite u is a finite part
// and an infinite one, not two infinities of different signs.
__device__ __forceinline__ void split8(const float u[8], u32x4_t *hi, u32x4_t *lo) {
  constexpr float kMost = 0x1.fep127f;  // the largest bf16
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = __builtin_amdgcn_fmed3f(u[i], -kMost, kMost);
  const u32x4_t h = pack8(rest);
  unpack8(h, rest);
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = u[i] - rest[i];
  *hi = h;
  *lo = pack8(rest);
}

// Zero for the columns j0 .. j0 + 7 of an adapter at and past its rank (they may hold anything).
__device__ __forceinline__ u32x4_t below_rank(u32x4_t v, int left) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t keep = (left > 2 * w ? 0xffffu : 0u) | (left > 2 * w + 1 ? 0xffff0000u : 0u);
    v[w] &= keep;
  }
  return v;
}

// ----------------------------------------------------------------------- plan
constexpr int kPlanWaves = 16;
struct PlanShared {
  int at[kPlanWaves][1024];  // tokens of a wave's share in each group, then where the next of them goes
  int wave[kPlanWaves];
};
// A chunk of 8192 tokens is shared out to 16 waves in order.  A lane finds the lanes with its own group by a vote per bit of
// the group's number; the first of them adds their count to the wave's, and a lane's place is the group's start, plus the
// counts of earlier chunks, waves and steps, plus the equal lanes before it: the order of the batch is kept.  Of several
// chunks a first launch writes the counts (COUNT), and each one adds up what it needs of them (65536 tokens 16 us for both,
// in one workgroup 85).
constexpr int kPlanSteps = 8;  // of 64 tokens, whose groups a wave holds at once
static_assert(kPlanWaves * 64 * kPlanSteps == kAdaptChunk, "a wave holds its share of a chunk");
template <bool COUNT>
__device__ __forceinline__ void plan_tokens(const AdaptRows &a, int chunk, PlanShared &sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), groups = a.n_pool + 1;
  const int bits = 32 - __builtin_clz(groups);
  const int64_t c0 = chunk * kAdaptChunk, c1 = c0 + kAdaptChunk < a.T ? c0 + kAdaptChunk : a.T;
  const int64_t per = ((c1 - c0 + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64, first = c0 + wave * per;
  const int64_t end = first + per < c1 ? first + per : c1;
  int group[kPlanSteps];
  uint64_t same[kPlanSteps];
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i) {
    const int64_t t = first + i * 64 + lane;
    group[i] = t < end ? group_of(a, t) : groups;  // (no token: a group of its own)
  }
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i) same[i] = same_lanes(group[i], bits);
  const uint64_t before = ((uint64_t)1 << lane) - 1;
  if (tid < groups)
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) sh.at[w][tid] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i)
    if (group[i] < groups && (same[i] & before) == 0) atomicAdd(&sh.at[wave][group[i]], __popcll(same[i]));
  __syncthreads();
  int n = 0;  // thread k: tokens of group k
  if (tid < groups)
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) n += sh.at[w][tid];
  if (COUNT) {
    if (tid < groups) a.counts[(int64_t)chunk * groups + tid] = n;
    return;
  }
  int earlier = 0;  // those in earlier chunks
  if (a.counts && tid < groups) {
    const int chunks = (int)adapt_chunks(a.T);
    n = 0;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) {
      const int k = a.counts[(int64_t)c * groups + tid];
      earlier += c < chunk ? k : 0;
      n += k;
    }
  }
  const int sum = scan_dpp(n);
  if (lane == 63) sh.wave[wave] = sum;
  __syncthreads();
  int at = sum - n;
  for (int w = 0; w < wave; ++w) at += sh.wave[w];
  if (tid < groups) {
    if (chunk == 0) {
      a.start[tid] = at;
      if (tid == a.n_pool) a.start[groups] = at + n;
    }
    at += earlier;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = sh.at[w][tid];
      sh.at[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanSteps; ++i) {
    if (group[i] < groups) {
      int *const at_ = &sh.at[wave][group[i]];
      const int base = *at_;
      a.order[base + __popcll(same[i] & before)] = (int32_t)(first + i * 64 + lane);
      wave_order();
      if ((same[i] & before) == 0) *at_ = base + __popcll(same[i]);
    }
    wave_order();
  }
}

// A workgroup turns all r ranks of 8 (1024 / r) rows or columns, a chunk of 16 bytes per thread: what it reads or writes is
// one piece of memory (with the plan, four of rank 72, 12600 and 13256 long 8.7 us, in tiles of 64 x 128 14.7; 16 of rank
// 32, 4096 and 4096 long 6.1 and 9.7).
// In LDS eight rows are followed by one word, so that a wave's reads down a column meet different banks.
struct TurnShared {
  uint32_t tile[4096 + 128];
};
__device__ __forceinline__ void turn_pool(const AdaptTurn &t, uint32_t id, TurnShared &sh) {
  const uint32_t pool = id / t.blocks, rest = id - pool * t.blocks;
  const int64_t r0 = t.rows == t.tile_rows ? 0 : (int64_t)rest * t.tile_rows;
  const int64_t c0 = t.rows == t.tile_rows ? (int64_t)rest * t.tile_cols : 0;
  const bf16_t *from = t.from + pool * t.rows * t.cols;
  bf16_t *to = t.to + pool * t.rows * t.cols;
  const uint32_t tid = threadIdx.x, across = t.tile_cols / 8, down = t.tile_rows / 8;  // (all sizes are multiples of 8)
  const uint32_t ld = t.tile_cols / 2;  // words of a row
  {
    const uint32_t row = tid / across, col = (tid - row * across) * 8;
    if (row < (uint32_t)t.tile_rows && r0 + row < t.rows && c0 + col < t.cols) {
      const u32x4_t v = load16(from + (r0 + row) * t.cols + c0 + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) sh.tile[row * ld + (row >> 3) + col / 2 + i] = v[i];
    }
  }
  __syncthreads();
  const uint32_t col = tid / down, row = (tid - col * down) * 8;
  if (col < (uint32_t)t.tile_cols && c0 + col < t.cols && r0 + row < t.rows) {
    const bf16_t *const at = reinterpret_cast<const bf16_t *>(&sh.tile[row * ld + (row >> 3)]) + col;
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = at[4 * i * ld] | (uint32_t)at[(4 * i + 2) * ld] << 16;
    store16(to + (c0 + col) * t.rows + r0 + row, v);
  }
}

// The first workgroups group the tokens, a chunk each; the others transpose.
__global__ __launch_bounds__(1024) void k_adapt_plan(AdaptRows a, int chunks, AdaptTurn t0, AdaptTurn t1, uint32_t blocks0,
                                                     uint32_t blocks) {
  __shared__ __attribute__((aligned(16))) char shared[sizeof(PlanShared)];
  static_assert(sizeof(TurnShared) <= sizeof(PlanShared), "one piece of LDS for both");
  if ((int)blockIdx.x < chunks) {
    plan_tokens<false>(a, blockIdx.x, *reinterpret_cast<PlanShared *>(shared));
    return;
  }
  for (uint32_t id = blockIdx.x - chunks; id < blocks; id += gridDim.x - chunks) {
    turn_pool(id < blocks0 ? t0 : t1, id < blocks0 ? id : id - blocks0, *reinterpret_cast<TurnShared *>(shared));
    __syncthreads();
  }
}
__global__ __launch_bounds__(1024) void k_adapt_count(AdaptRows a) {
  __shared__ PlanShared shared;
  plan_tokens<true>(a, blockIdx.x, shared);
}

// A 16-byte chunk of a row of 64 values in LDS: the eight chunks of rows in turn, so that the 16 rows that an MFMA operand
// reads at one place begin in different banks.
__device__ __forceinline__ int chunk_at(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// --------------------------------------------------------------------- shrink
// RT: rank tiles of 16, MT: token tiles of 16.  Eight waves take 64-value steps of the long axis in turn.  A step's rows
// come in whole lines (eight lanes each) and go through a part of LDS that is the wave's own: no barriers.  Straight into
// the MFMA's layout, where neighbouring lanes are neighbouring rows, each lane is a cache access of its own, which alone
// took 15 of 20 us (4096 tokens x 4096, ranks to 64; now 12, 2.8 TB/s of X beside the adapters' rows from the L2).  What
// stands in a row that is none (past the rank) stays in that row's sums, which are not stored.  (MT = 2 at these ranks:
// 12.4 -> 16.4 us.)
constexpr int kShrinkWaves = 8;
template <int RT, int MT>
__global__ __launch_bounds__(64 * kShrinkWaves, RT <= 4 ? 4 : MT == 1 ? 3 : 2) void k_adapt_shrink(
    AdaptRows a, const bf16_t *__restrict__ P, int64_t K, const bf16_t *__restrict__ Q, bool scaled, int ranges,
    float *__restrict__ U) {
  constexpr int LD = RT * 16 + 4, PART = RT < 2 ? RT : 2;  // rank tiles that are in LDS at once
  constexpr int kOwn = 2048 * (MT + PART), kAll = kShrinkWaves * kOwn, kSums = kShrinkWaves * 16 * LD * 4;
  __shared__ __attribute__((aligned(128))) char shared[kAll > kSums ? kAll : kSums];
  __shared__ int s_token[16 * MT];
  float(*const s_sum)[16][LD] = reinterpret_cast<float(*)[16][LD]>(shared);
  const int id = blockIdx.x / ranges, range = blockIdx.x - id * ranges;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l = lane & 15;
  Tile tile;
  int token[MT];
  if (!find_tokens<16 * MT>(a, id, &tile, token)) return;
  const int rank = rank_of(a, tile.group);
  if (wave == 0 && lane < 16)
#pragma unroll
    for (int m = 0; m < MT; ++m) s_token[16 * m + lane] = token[m];
  f32x4_t acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (rank > 0) {
    char *const own = shared + wave * kOwn;
    const int row0 = lane >> 3, chunk = lane & 7;  // of this lane's loads: rows row0 and row0 + 8 of 16
    const bf16_t *p[2 * MT];
    bool there[2 * MT];
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) {
      there[h] = row0 + 8 * h < tile.n;
      p[h] = P + (int64_t)__builtin_amdgcn_ds_bpermute((row0 + 8 * (h & 1)) * 4, token[h >> 1]) * K + chunk * 8;
    }
    const char *q = (const char *)(Q + (int64_t)tile.group * a.r * K);
    uint32_t row[RT][2];  // bytes from the adapter's first (r K <= 2^29)
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = j * 16 + row0 + 8 * h;
        row[j][h] = (uint32_t)(((at < rank ? at : 0) * K + chunk * 8) * 2);
      }
    const int64_t steps = (K + 63) / 64, per = (steps + ranges - 1) / ranges;
    const int64_t first = range * per, end = first + per < steps ? first + per : steps;
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    u32x4_t pv[2 * MT], qv[RT][2];
    auto load = [&](int64_t k) {
      const bool in = k + chunk * 8 < K;
#pragma unroll
      for (int h = 0; h < 2 * MT; ++h) pv[h] = in && there[h] ? load16(p[h] + k) : zero;
      if (k + 64 <= K) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) qv[j][h] = *reinterpret_cast<const u32x4_t *>(q + (row[j][h] + (uint32_t)k * 2));
      } else {  // the rows' end
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            qv[j][h] = in ? *reinterpret_cast<const u32x4_t *>(q + (row[j][h] + (uint32_t)k * 2)) : zero;
      }
    };
    // Each tile begins at a step of its own: rows a power of two apart would otherwise meet in few memory channels.
    const int n = (int)(end - first);
    int at = n > 0 ? (int)((uint32_t)(id * 8 + wave) % (uint32_t)n) : 0;
    auto next = [&] {
      at += kShrinkWaves;
      if (at >= n) at = at - n < n ? at - n : (int)((uint32_t)at % (uint32_t)n);
    };
    if (wave < n) load((first + at) * 64);
    for (int i = wave; i < n; i += kShrinkWaves) {
      u32x4_t pf[MT][2];
#pragma unroll
      for (int h = 0; h < 2 * MT; ++h) *reinterpret_cast<u32x4_t *>(own + chunk_at(row0 + 8 * h, chunk)) = pv[h];
#pragma unroll
      for (int j0 = 0; j0 < RT; j0 += PART) {
#pragma unroll
        for (int j = 0; j < PART; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<u32x4_t *>(own + 2048 * (MT + j) + chunk_at(row0 + 8 * h, chunk)) = qv[j0 + j][h];
        if (j0 + PART == RT) {  // (all of this step is on its way)
          next();
          if (i + kShrinkWaves < n) load((first + at) * 64);
        }
        wave_order();
        if (j0 == 0)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              pf[m][h] = *reinterpret_cast<const u32x4_t *>(own + 2048 * m + chunk_at(l, 4 * h + g));
#pragma unroll
        for (int j = 0; j < PART; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4_t qf = *reinterpret_cast<const u32x4_t *>(own + 2048 * (MT + j) + chunk_at(l, 4 * h + g));
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m][j0 + j] = mfma16(qf, pf[m][h], acc[m][j0 + j]);
          }
        wave_order();
      }
    }
  }
  const float scale = scaled && tile.group < a.n_pool ? a.scale[tile.group] : 1.f;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < RT; ++j) *reinterpret_cast<f32x4_t *>(&s_sum[wave][l][j * 16 + 4 * g]) = acc[m][j];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * RT * 16; e += 64 * kShrinkWaves) {
      const int n = e / (RT * 16), j = e % (RT * 16);
      if (16 * m + n >= tile.n || j >= a.r) continue;
      float sum = 0.f;
      if (j < rank) {
#pragma unroll
        for (int w = 0; w < kShrinkWaves; ++w) sum += s_sum[w][n][j];
        sum *= scale;
      }
      U[((int64_t)range * a.T + s_token[16 * m + n]) * a.r + j] = sum;
    }
  }
}

// Columns j0 .. j0 + 7 of a token's u: the ranges' sums, times the scale, zero at and past the rank.
__device__ __forceinline__ void load_u(const AdaptRows &a, const float *__restrict__ U, int ranges, int64_t token, int j0,
                                       int rank, float u[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = 0.f;
  if (j0 >= rank) return;
  const float *p = U + token * a.r + j0;
  const int64_t step = a.T * a.r;
  for (int q = 0; q < ranges; q += 4) {  // four ranges in flight; what is behind the last adds nothing
    float4 x[4], y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q + e < ranges) {
        x[e] = reinterpret_cast<const float4 *>(p + (q + e) * step)[0];
        y[e] = reinterpret_cast<const float4 *>(p + (q + e) * step)[1];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[0] += x[e].x, u[1] += x[e].y, u[2] += x[e].z, u[3] += x[e].w;
      u[4] += y[e].x, u[5] += y[e].y, u[6] += y[e].z, u[7] += y[e].w;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = j0 + i < rank ? u[i] : 0.f;
}

// --------------------------------------------------------------------- expand
// MT: tiles of 16 tokens.  KS: 32-wide steps over the rank, each an MFMA with u's high part and one with its low part;
// KS = 0 (rank up to 16): both parts side by side in one.  A wave takes 32 rows of Q at a time, which lie together in
// memory, through its own part of LDS (see k_adapt_shrink), and the products of the four waves go through LDS, so that base
// and output are read and written 256 bytes of a row at a time: from the MFMA's layout (64 bytes of 16 tokens each)
// a copy alone reached 3.9 to 4.9 TB/s, in such pieces 5.8.
constexpr int kExpandCols = 128;
// ONCE: the base goes past the caches.  LINES: output and base in whole lines of memory where rows do not begin with one: a
// row goes `back` columns behind the products, to where a line begins, and what is left of a step's products waits in
// registers for the next one (4096 tokens x 14344, rank 64 66 us, else 89; x 14336 56).
struct ExpandArgs {
  const float *U;
  int ranges;
  const bf16_t *Q;
  int64_t N;
  bool scaled;
  int64_t per;  // columns of a block, a multiple of 128
  int blocks;
  const bf16_t *base;
  bf16_t *out;
  float *U_out;
};
template <int KS, int MT>
struct ExpandShared {
  static constexpr int CP = KS ? KS * 4 : 2, TOKENS = 16 * MT;  // CP: 16-byte chunks of a row of the adapter
  static constexpr int kOut = TOKENS * (kExpandCols + 4) * 4, kParts = TOKENS * CP * 32;
  char q[4][32 * CP * 16];
  char mem[kOut > kParts ? kOut : kParts];
  int token[TOKENS];
};
template <int KS, int MT, bool ONCE, bool LINES>
__device__ __forceinline__ void expand_tile(const AdaptRows &a, const ExpandArgs &x, int at_block, char *shared) {
  using S = ExpandShared<KS, MT>;
  constexpr int CP = S::CP, KQ = KS ? KS : 1, TOKENS = S::TOKENS;
  const float *const U = x.U;
  const int64_t N = x.N;
  const bf16_t *const base = x.base;
  bf16_t *const out = x.out;
  S &sh = *reinterpret_cast<S *>(shared);
  char *const s_mem = sh.mem;
  int *const s_token = sh.token;
  float(*const s_out)[kExpandCols + 4] = reinterpret_cast<float(*)[kExpandCols + 4]>(s_mem);
  const int id = at_block / x.blocks, block = at_block - id * x.blocks;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, l = lane & 15;
  // chunk of a row of CP chunks: rows in turn, as chunk_at
  auto swizzled = [](int row, int chunk) {
    return (row * CP + (CP == 2 ? chunk : chunk ^ (CP == 4 ? (row >> 2) & 3 : row & 7))) * 16;
  };
  Tile tile;
  int token[MT];
  if (!find_tokens<TOKENS>(a, id, &tile, token)) return;
  const int rank = rank_of(a, tile.group);
  if (rank == 0 && base == out && !x.U_out) return;
  if (wave == 0 && g == 0)
#pragma unroll
    for (int m = 0; m < MT; ++m) s_token[m * 16 + l] = token[m];
  __syncthreads();
  const int64_t first = block * x.per, end = first + x.per < N ? first + x.per : N;
  // rows as they lie in memory: a thread's 8 columns of every 16th token; its chunks of the wave's 32 rows of Q.  The first
  // step's are on their way before u is, and each next step's before the present one is stored.
  const int row0 = tid >> 4, col0 = (tid & 15) * 8;
  const int64_t stop = LINES ? end + kExpandCols : end;
  int64_t at[MT];
  int back[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = (int64_t)s_token[row0 + 16 * i] * N;
    back[i] = LINES ? (int)((uintptr_t)(out + row) >> 4 & 7) * 8 : 0;
    at[i] = row + col0 - back[i];
  }
  auto mine = [&](int i, int64_t n0) {
    const int64_t n = n0 + col0 - back[i];
    return row0 + 16 * i < tile.n && (!LINES || n >= first) && n < end;
  };
  const char *const q = (const char *)(x.Q + (int64_t)(rank ? tile.group : 0) * N * a.r);
  char *const own = sh.q[wave];
  u32x4_t bv[MT], qv[CP / 2];
  auto load = [&](int64_t n0) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      bv[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (base && mine(i, n0))
        bv[i] = ONCE ? load16_once(base + at[i] + n0) : load16(base + at[i] + n0);
    }
    if (rank && n0 < end)
#pragma unroll
      for (int i = 0; i < CP / 2; ++i) {  // (behind the last row: any row, whose products are not stored)
        const int r = i * (64 / CP) + lane / CP, c = lane % CP;
        const int64_t n = n0 + wave * 32 + r, row = n < N ? n : N - 1;
        qv[i] = *reinterpret_cast<const u32x4_t *>(q + ((uint32_t)row * (uint32_t)a.r + (c * 8 < a.r ? c * 8 : 0)) * 2u);
      }
  };
  load(first);
  const float scale = x.scaled && tile.group < a.n_pool ? a.scale[tile.group] : 1.f;
  // u of the tile's tokens: the ranges' sums, to x.U_out, and times the scale in two parts to LDS
  for (int e = tid; e < TOKENS * CP; e += 256) {
    const int n = e / CP, c = e % CP;
    float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n < tile.n) load_u(a, U, x.ranges, s_token[n], c * 8, rank, u);
    if (x.U_out && block == 0 && n < tile.n && c * 8 < a.r) {
      float4 *to = reinterpret_cast<float4 *>(x.U_out + (int64_t)s_token[n] * a.r + c * 8);
      to[0] = make_float4(u[0], u[1], u[2], u[3]);
      to[1] = make_float4(u[4], u[5], u[6], u[7]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = c * 8 + i < rank ? u[i] * scale : 0.f;  // (an infinite scale times no column)
    u32x4_t h, o;
    split8(u, &h, &o);
    *reinterpret_cast<u32x4_t *>(s_mem + swizzled(n, c)) = h;
    *reinterpret_cast<u32x4_t *>(s_mem + TOKENS * CP * 16 + swizzled(n, c)) = o;
  }
  __syncthreads();
  u32x4_t hi[MT][KQ], lo[MT][KQ];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int k = 0; k < KQ; ++k) {
      const char *from = s_mem + swizzled(m * 16 + l, KS ? k * 4 + g : g & 1);
      if (KS) {
        hi[m][k] = *reinterpret_cast<const u32x4_t *>(from);
        lo[m][k] = *reinterpret_cast<const u32x4_t *>(from + TOKENS * CP * 16);
      } else {
        hi[m][k] = *reinterpret_cast<const u32x4_t *>(from + (g < 2 ? 0 : TOKENS * CP * 16));
      }
    }
  __syncthreads();
  const bool full = rank == CP * 8;
  f32x4_t left[MT][2] = {};
  for (int64_t n0 = first; n0 < stop; n0 += kExpandCols) {
    u32x4_t now[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) now[i] = bv[i];
    const bool products = rank && (!LINES || n0 < end);
    if (products)
#pragma unroll
      for (int i = 0; i < CP / 2; ++i) {
        const int r = i * (64 / CP) + lane / CP, c = lane % CP;
        *reinterpret_cast<u32x4_t *>(own + swizzled(r, c)) = full ? qv[i] : below_rank(qv[i], rank - c * 8);
      }
    if (n0 + kExpandCols < stop) load(n0 + kExpandCols);
    if (products) {
      wave_order();
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        u32x4_t qf[KQ];
#pragma unroll
        for (int k = 0; k < KQ; ++k)
          qf[k] = *reinterpret_cast<const u32x4_t *>(own + swizzled(p * 16 + l, KS ? k * 4 + g : g & 1));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KQ; ++k) {
            acc = mfma16(qf[k], hi[m][k], acc);
            if (KS) acc = mfma16(qf[k], lo[m][k], acc);
          }
          *reinterpret_cast<f32x4_t *>(&s_out[m * 16 + l][wave * 32 + 16 * p + 4 * g]) = acc;
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const f32x4_t *d = reinterpret_cast<const f32x4_t *>(&s_out[row0 + 16 * i][(col0 - back[i]) & (kExpandCols - 1)]);
      f32x4_t d0, d1;
      if (LINES) {
        const f32x4_t v0 = d[0], v1 = d[1];  // (behind the last step nothing new, which nothing takes)
        d0 = col0 < back[i] ? left[i][0] : v0, d1 = col0 < back[i] ? left[i][1] : v1;
        left[i][0] = v0, left[i][1] = v1;
      }
      if (mine(i, n0)) {
        if (rank) {
          if (!LINES) d0 = d[0], d1 = d[1];
          float y[8];
          unpack8(now[i], y);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] += d0[e], y[4 + e] += d1[e];
          now[i] = pack8(y);
        }
        store16_once(out + at[i] + n0, now[i]);
      }
    }
    if (products) __syncthreads();
  }
}

template <int KS, int MT, bool ONCE, bool LINES>
__global__ __launch_bounds__(256, KS * MT <= 4 ? 4 : 2) void k_adapt_expand(AdaptRows a, ExpandArgs x) {
  __shared__ __attribute__((aligned(128))) char shared[sizeof(ExpandShared<KS, MT>)];
  expand_tile<KS, MT, ONCE, LINES>(a, x, blockIdx.x, shared);
}

// ---------------------------------------------------------------------- grads
// One piece of an adapter's tokens, CW columns of the long operand.  Each of four waves takes 32 tokens in turn: their
// rows go to its own part of LDS as they are and are read back transposed (ds_read_b64_tr_b16: lane i of 16 gets element
// i % 4 of the 8 bytes that lanes 4 m + i / 4 address, m = 0 .. 3), the rank-wide operand likewise in two bf16 parts; the
// next 32 tokens' rows are on their way meanwhile, and there are no barriers.  At the end the waves' sums are added in LDS
// ((0 + 2) + (1 + 3)).
__device__ __forceinline__ u32x4_t turned(const bf16_t *base, int ld, int row, int col) {
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t *)(base + row * ld + col));
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t *)(base + (row + 4) * ld + col));
  const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
  return u32x4_t{l2.x, l2.y, h2.x, h2.y};
}

// Columns of a workgroup (128 take more registers for the sums: rank 64 23 us, else 17; rank 16 9.4, else 8.8).
constexpr int kGradCols = 64;
template <int RT>
struct GradShape {
  static constexpr int CW = kGradCols, LX = CW + 16, LV = RT * 16 + (RT > 1 ? 16 : 0);
  static constexpr int kOwn = 32 * (LX + 2 * LV) * 2;                                // bytes of a wave
  static constexpr int LD_A = CW + 4, LD_B = RT * 16 + 4;                            // rows of the sums of dA, dB
  static constexpr int kSums = (RT * 16 * LD_A > CW * LD_B ? RT * 16 * LD_A : CW * LD_B) * 4;  // bytes, of one wave
  static constexpr int kAll = 4 * kOwn > 2 * kSums ? 4 * kOwn : 2 * kSums;
};

// BY_J: the output is [n][r] (dB), else [r][n] (dA).  The ranks from jb on, 16 RT of them.
template <int RT, bool BY_J>
__device__ __forceinline__ void grad_piece(const AdaptRows &a, const Tile &tile, int rank, int jb,
                                           const float *__restrict__ V, int ranges, float scale,
                                           const bf16_t *__restrict__ X, int64_t N, int64_t c0, float *__restrict__ part,
                                           bf16_t *__restrict__ grad, char *shared) {
  using S = GradShape<RT>;
  constexpr int CW = S::CW, LX = S::LX, LV = S::LV, XL = CW / 16, PT = CW / 16;  // XL: 16-byte loads of X per lane
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, l = lane & 15;
  bf16_t *const s_x = reinterpret_cast<bf16_t *>(shared + wave * S::kOwn), *const s_hi = s_x + 32 * LX,
                *const s_lo = s_hi + 32 * LV;
  f32x4_t acc[PT][RT];
#pragma unroll
  for (int p = 0; p < PT; ++p)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[p][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int XC = CW / 8;  // 16-byte chunks of a row of X
  const int xrow = lane / XC, xcol = lane % XC * 8;
  const int64_t col = c0 + xcol < N ? c0 + xcol : N - 8;  // (behind the row's end: any, whose products are not stored)
  // lane i: the token at place t + i % 32; behind the end the last one again, whose row of X then counts as zero
  auto tokens_of = [&](int t) {
    const int p = t + (lane & 31);
    return a.order[tile.p0 + (p < tile.n ? p : tile.n - 1)];
  };
  u32x4_t x[XL];
  float4 v[RT][2];
  const int64_t step = a.T * a.r / 4;  // from range to range
  auto load = [&](int tokens) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int64_t t = __builtin_amdgcn_ds_bpermute((xrow + i * (64 / XC)) * 4, tokens);
      x[i] = load16(X + t * N + col);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int e = lane + 64 * i, row = e / (RT * 2), j0 = e % (RT * 2) * 8;
      const int64_t t = __builtin_amdgcn_ds_bpermute(row * 4, tokens);
      const float4 *from = reinterpret_cast<const float4 *>(V + t * a.r + (jb + j0 < a.r ? jb + j0 : 0));
      v[i][0] = from[0];
      v[i][1] = from[1];
      for (int q = 1; q < ranges; ++q) {  // (few tokens only: otherwise the ranges have been added)
        const float4 y = from[q * step], z = from[q * step + 1];
        v[i][0].x += y.x, v[i][0].y += y.y, v[i][0].z += y.z, v[i][0].w += y.w;
        v[i][1].x += z.x, v[i][1].y += z.y, v[i][1].z += z.z, v[i][1].w += z.w;
      }
    }
  };
  int tokens = 0;
  if (wave * 32 < tile.n) {
    load(tokens_of(wave * 32));
    tokens = tokens_of(wave * 32 + 128);
  }
  for (int t0 = wave * 32; t0 < tile.n; t0 += 128) {
    const int left = tile.n - t0;
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int row = xrow + i * (64 / XC);
      *reinterpret_cast<u32x4_t *>(s_x + row * LX + xcol) = row < left ? x[i] : u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int e = lane + 64 * i, row = e / (RT * 2), j0 = e % (RT * 2) * 8;
      const float4 p = v[i][0], q = v[i][1];
      const float u[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
      u32x4_t hi, lo;
      split8(u, &hi, &lo);
      if (left < 32 && row >= left) hi = lo = u32x4_t{0u, 0u, 0u, 0u};  // (an infinite u times that zero row of X)
      *reinterpret_cast<u32x4_t *>(s_hi + row * LV + j0) = hi;
      *reinterpret_cast<u32x4_t *>(s_lo + row * LV + j0) = lo;
    }
    if (left > 128) {
      load(tokens);
      tokens = tokens_of(t0 + 256);
    }
    wave_order();
    const int row = 8 * g + (l >> 2), at = 4 * (l & 3);
    u32x4_t xv[PT];
#pragma unroll
    for (int p = 0; p < PT; ++p) xv[p] = turned(s_x, LX, row, 16 * p + at);
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const u32x4_t hi = turned(s_hi, LV, row, 16 * j + at), lo = turned(s_lo, LV, row, 16 * j + at);
#pragma unroll
      for (int p = 0; p < PT; ++p) {
        if (BY_J) {
          acc[p][j] = mfma16(hi, xv[p], acc[p][j]);
          acc[p][j] = mfma16(lo, xv[p], acc[p][j]);
        } else {
          acc[p][j] = mfma16(xv[p], hi, acc[p][j]);
          acc[p][j] = mfma16(xv[p], lo, acc[p][j]);
        }
      }
    }
    wave_order();
  }
  // the sums of two waves at a time, in the output's layout: [rank][column] or [column][rank]
  constexpr int LD = BY_J ? S::LD_B : S::LD_A;
  float *const s_sum = reinterpret_cast<float *>(shared + (wave & 1) * S::kSums);
  auto each = [&](auto &&f) {
#pragma unroll
    for (int p = 0; p < PT; ++p)
#pragma unroll
      for (int j = 0; j < RT; ++j)
        f(acc[p][j], reinterpret_cast<f32x4_t *>(BY_J ? s_sum + (16 * p + l) * LD + 16 * j + 4 * g
                                                      : s_sum + (16 * j + l) * LD + 16 * p + 4 * g));
  };
  __syncthreads();
  if (wave >= 2) each([](f32x4_t &v_, f32x4_t *at) { *at = v_; });
  __syncthreads();
  if (wave < 2) each([](f32x4_t &v_, f32x4_t *at) { *at = v_ + *at; });
  __syncthreads();
  const int64_t size = (int64_t)a.r * N;
  constexpr int ROW = BY_J ? RT * 16 : CW, ROWS = BY_J ? CW : RT * 16;
  for (int e = tid; e < ROWS * (ROW / 8); e += 256) {
    const int row = e / (ROW / 8), c = e % (ROW / 8) * 8;
    const int64_t n = c0 + (BY_J ? row : c);
    const int j = jb + (BY_J ? c : row);
    if (n >= N || j >= a.r) continue;
    const f32x4_t *p = reinterpret_cast<const f32x4_t *>(reinterpret_cast<const float *>(shared) + row * LD + c);
    const f32x4_t *q = reinterpret_cast<const f32x4_t *>(reinterpret_cast<const float *>(shared + S::kSums) + row * LD + c);
    f32x4_t v0 = p[0] + q[0], v1 = p[1] + q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // (past the rank: zero, whatever u holds there)
      v0[i] = j + (BY_J ? i : 0) < rank ? v0[i] * scale : 0.f;
      v1[i] = j + (BY_J ? 4 + i : 0) < rank ? v1[i] * scale : 0.f;
    }
    const int64_t to = BY_J ? n * a.r + j : j * N + n;
    if (tile.slot >= 0) {
      f32x4_t *out = reinterpret_cast<f32x4_t *>(part + tile.slot * size + to);
      out[0] = v0;
      out[1] = v1;
    } else {
      store16(grad + tile.group * size + to, u32x4_t{pack_bf16x2(v0[0], v0[1]), pack_bf16x2(v0[2], v0[3]),
                                                     pack_bf16x2(v1[0], v1[1]), pack_bf16x2(v1[2], v1[3])});
    }
  }
}

// A workgroup takes at most 64 ranks, an equal part of them, as their sums then leave room for others (8000 tokens, 4096 x
// 4096, rank 128: with all of them in one, and one workgroup per CU, 95 us; so 78).
struct GradArgs {
  AdaptGrads g;
  int piece, parts, blocks_a, columns, blocks;  // columns: blocks of 64, of X first; blocks: of a piece, in all
};
template <int RT>
__device__ __forceinline__ void grads_tile(const AdaptRows &a, const GradArgs &q, int at_block, char *shared) {
  const int id = at_block / q.blocks, rest = at_block - id * q.blocks;
  // (the parts of a block of columns come eight workgroups apart, on one XCD: the columns are then in its L2)
  const int eights = rest / (8 * q.parts), in = rest - eights * 8 * q.parts;
  const int block = q.parts == 1 ? rest : eights * 8 + (in & 7), jb = q.parts == 1 ? 0 : (in >> 3) * 16 * RT;
  if (block >= q.columns) return;
  Tile tile;
  if (!find_tile<true>(a, q.piece, id, &tile)) return;
  const int rank = tile.n > 0 ? rank_of(a, tile.group) : 0;  // (without tokens: zeros, whatever the scale holds)
  const AdaptGrads &g = q.g;
  if (block < q.blocks_a)
    grad_piece<RT, false>(a, tile, rank, jb, g.dU, g.dU_ranges, 1.f, g.X, g.n_in, (int64_t)block * kGradCols, g.part_a, g.dA,
                          shared);
  else
    grad_piece<RT, true>(a, tile, rank, jb, g.U, 1, a.scale[tile.group], g.dY, g.n_out,
                         (int64_t)(block - q.blocks_a) * kGradCols, g.part_b, g.dB, shared);
}
template <int RT>
__global__ __launch_bounds__(256) void k_adapt_grads(AdaptRows a, GradArgs q) {
  __shared__ __attribute__((aligned(128))) char shared[GradShape<RT>::kAll];
  grads_tile<RT>(a, q, blockIdx.x, shared);
}

// Few tokens, whose kernels' time is mostly their start: dX and the gradients of the pools in one.
template <int KS, int RT>
__global__ __launch_bounds__(256) void k_adapt_back(AdaptRows a, ExpandArgs x, GradArgs q, int expand_blocks) {
  constexpr int kExpand = sizeof(ExpandShared<KS, 1>), kGrads = GradShape<RT>::kAll;
  __shared__ __attribute__((aligned(128))) char shared[kExpand > kGrads ? kExpand : kGrads];
  if ((int)blockIdx.x < expand_blocks) expand_tile<KS, 1, false, false>(a, x, blockIdx.x, shared);
  else grads_tile<RT>(a, q, blockIdx.x - expand_blocks, shared);
}

// A group's gradient from the sums of its pieces, in order, 8 values per thread.  What has one piece is written already.
__global__ __launch_bounds__(256) void k_adapt_reduce(AdaptRows a, AdaptGrads g, int piece, int64_t blocks_a) {
  const int group = blockIdx.y, lane = threadIdx.x & 63;
  const int n = a.start[group + 1] - a.start[group], pieces = (n + piece - 1) / piece;
  if (pieces <= 1) return;
  int slot = 0;  // pieces of earlier groups of several
  for (int k0 = 0; k0 < group; k0 += 64) {
    int c = 0;
    if (k0 + lane < group) c = (a.start[k0 + lane + 1] - a.start[k0 + lane] + piece - 1) / piece;
    slot += __builtin_amdgcn_readlane(scan_dpp(c > 1 ? c : 0), 63);
  }
  const bool of_a = blockIdx.x < blocks_a;
  const int64_t size = (int64_t)a.r * (of_a ? g.n_in : g.n_out);
  const int64_t e = ((blockIdx.x - (of_a ? 0 : blocks_a)) * 256 + threadIdx.x) * 8;
  if (e >= size) return;
  const float *p = (of_a ? g.part_a : g.part_b) + slot * size + e;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int q = 0; q < pieces; ++q) {
    const float4 *const at = reinterpret_cast<const float4 *>(p + q * size);
    const float4 x = at[0], y = at[1];
    sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w, sum[4] += y.x, sum[5] += y.y, sum[6] += y.z, sum[7] += y.w;
  }
  store16((of_a ? g.dA : g.dB) + group * size + e, pack8(sum));
}

// Tiles of M tokens, at most: groups do not share one.
int64_t most_tiles(const AdaptRows &a, int M) {
  const int64_t groups = a.n_pool + 1 < a.T ? a.n_pool + 1 : a.T;
  return a.T / M + groups;
}

}  // namespace

hipError_t launch_adapt_plan(const AdaptRows &a, AdaptTurn t0, AdaptTurn t1, hipStream_t s) {
  // (at most 2^27 / 64 + 1000 workgroups for a pool)
  const int side = 1024 / a.r * 8;
  t0.tile_rows = t1.tile_cols = a.r;
  t0.tile_cols = t1.tile_rows = side;
  t0.blocks = (uint32_t)((t0.cols + side - 1) / side), t1.blocks = (uint32_t)((t1.rows + side - 1) / side);
  const uint32_t b0 = t0.to ? a.n_pool * t0.blocks : 0, blocks = b0 + (t1.to ? a.n_pool * t1.blocks : 0);
  // (the largest pools have more blocks than a launch may have threads)
  const int64_t chunks = a.T > 0 ? adapt_chunks(a.T) : 1;
  const dim3 grid((uint32_t)chunks + (blocks < 8192 ? blocks : 8192));
  launch(k_adapt_plan, grid, dim3(1024), 0, s, a, (int)chunks, t0, t1, b0, blocks);
  return hipGetLastError();
}

hipError_t launch_adapt_count(const AdaptRows &a, hipStream_t s) {
  launch(k_adapt_count, dim3((uint32_t)adapt_chunks(a.T)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

// Tiles of 32 tokens, which read the adapter half as often: above rank 64, where a CU holds one workgroup either way, and
// where there are tiles enough (8000 x 4096, rank 128 44.4 -> 29.5 us; 300 x 4096, rank 72 6.0 -> 7.2).
static bool shrink_wide(int64_t T, int r) { return r > 64 && T >= 2048; }

// Enough workgroups for the GPU, but no more partial sums than that takes, which the next product adds for each of its
// blocks of columns (4096 x 4096: 1200 tokens, rank 64 22.7 us with three ranges, 25.5 with nine; 2048 29.3 with
// two, 32.6 with five; 4096 42.9 with two, 44.2 with one).  Above rank 64 a CU holds one workgroup of the shrinking product,
// and a second round of them costs as much as the first (4000 tokens, rank 128 49 us with one range, 61 with two).
int adapt_ranges(int64_t T, int n_pool, int r, int64_t K) {
  const int m = shrink_wide(T, r) ? 32 : 16;
  const int64_t tiles = (T + m - 1) / m + (n_pool < T ? n_pool : T) / 2, most = (K + 511) / 512;
  int64_t n = tiles < 1 ? 1 : (r > 32 ? 256 : 512) / tiles;
  if (n < 2 && r <= 64 && tiles <= 384) n = 2;
  n = n < 1 ? 1 : n > 8 ? 8 : n;
  return (int)(n < most ? n : most);
}

hipError_t launch_adapt_shrink(const AdaptRows &a, const bf16_t *P, int64_t K, const bf16_t *Q, bool scaled, int ranges,
                               float *U, hipStream_t s) {
  const bool wide = shrink_wide(a.T, a.r);
  const dim3 grid((uint32_t)(most_tiles(a, wide ? 32 : 16) * ranges)), block(64 * kShrinkWaves);
#define SHRINK(RT_, MT_) launch(k_adapt_shrink<RT_, MT_>, grid, block, 0, s, a, P, K, Q, scaled, ranges, U)
  if (a.r <= 16) SHRINK(1, 1);
  else if (a.r <= 32) SHRINK(2, 1);
  else if (a.r <= 64) SHRINK(4, 1);
  else if (a.r <= 96 && wide) SHRINK(6, 2);
  else if (a.r <= 96) SHRINK(6, 1);
  else if (wide) SHRINK(8, 2);
  else SHRINK(8, 1);
#undef SHRINK
  return hipGetLastError();
}

namespace {
// The expanding product's arguments and workgroups.
ExpandArgs expand_args(const AdaptRows &a, bool wide, const float *U, int ranges, const bf16_t *Q, int64_t N, bool scaled,
                       const bf16_t *base, bf16_t *out, float *U_out, int64_t *grid) {
  const int64_t tiles = most_tiles(a, wide ? 32 : 16), cols = (N + kExpandCols - 1) / kExpandCols;
  // Column blocks, so many that the workgroups which the GPU holds at once (`slots`) are used up in whole rounds, and each
  // has several steps to share its lookups and u, which cost about one: of the numbers of rounds the one that takes least
  // (4096 x 4096: 8000 tokens, rank 64 32.3 us so, 37.8 with 16 blocks in all cases; 3000 x 6000, rank 96 26.5 us, with 8
  // blocks 32).  Adapters past the L2s take a multiple of 8 blocks, so that a block's rows of Q stay in the L2 of one XCD
  // (workgroups go round the eight: 4096 x 14336, 8 of rank 64 62 us, else 67); above rank 64 that is no gain (2000 x
  // 9000, 5 of rank 128 33 us, else 29.5).
  const int64_t slots = a.r > 64 ? (wide ? 512 : 768) : a.r > 32 && wide ? 1024 : 1280;
  const int64_t adapters = a.n_pool < a.T ? a.n_pool : a.T, likely = a.T / (wide ? 32 : 16) + adapters / 2 + 1;
  const bool eights = a.r <= 64 && adapters * N * a.r * 2 > (int64_t)8 << 20;
  int64_t least = INT64_MAX, per = 1;
  for (int k = 1; k <= 6; ++k) {
    int64_t b = eights ? 8 * k : k * slots / likely;
    if (b < 1) b = 1;
    const int64_t steps = (cols + b - 1) / b, rounds = (b * likely + slots - 1) / slots;
    if (rounds * (steps + 1) < least) least = rounds * (steps + 1), per = steps;
  }
  int64_t blocks = (cols + per - 1) / per;
  if (eights && blocks > 8) blocks = (blocks + 7) / 8 * 8;
  *grid = blocks * tiles;
  return ExpandArgs{U, ranges, Q, N, scaled, per * kExpandCols, (int)blocks, base, out, U_out};
}

GradArgs grad_args(const AdaptRows &a, const AdaptGrads &g, int piece, int64_t *grid) {
  const int64_t ba = g.dA ? (g.n_in + kGradCols - 1) / kGradCols : 0, bb = g.dB ? (g.n_out + kGradCols - 1) / kGradCols : 0;
  const int parts = (a.r + 63) / 64;
  const int64_t blocks = parts > 1 ? (ba + bb + 7) / 8 * 8 * parts : ba + bb;
  *grid = blocks * (a.T / piece + a.n_pool);
  return GradArgs{g, piece, parts, (int)ba, (int)(ba + bb), (int)blocks};
}
}  // namespace

hipError_t launch_adapt_expand(const AdaptRows &a, const float *U, int ranges, const bf16_t *Q, int64_t N, bool scaled,
                               const bf16_t *base, bf16_t *out, float *U_out, hipStream_t s) {
  const bool wide = a.T >= 2048;
  int64_t blocks;
  const ExpandArgs x = expand_args(a, wide, U, ranges, Q, N, scaled, base, out, U_out, &blocks);
  // A base that the caches cannot hold beside the rest goes past them (4096 x 14336, 117 MB: the call 79 us, else 84; of
  // 25 MB, just written, 19 us of the kernel, else 14).
  const bool once = a.T * N * 2 > (int64_t)64 << 20;
  // (what the L2s hold is put together there: 5703 x 2704 takes 17.6 us either way, 3001 x 1000 13.4, with LINES 15.0)
  const bool lines = (N % 64 != 0 || ((uintptr_t)out & 127) != 0) && a.T * N * 2 > (int64_t)32 << 20;
  const dim3 grid((uint32_t)blocks), block(256);
#define EXPAND_(KS_, MT_, ONCE_)                                                               \
  do {                                                                                         \
    if (lines) launch(k_adapt_expand<KS_, MT_, ONCE_, true>, grid, block, 0, s, a, x);         \
    else launch(k_adapt_expand<KS_, MT_, ONCE_, false>, grid, block, 0, s, a, x);              \
  } while (0)
#define EXPAND(KS_)                            \
  do {                                         \
    if (wide && once) EXPAND_(KS_, 2, true);   \
    else if (wide) EXPAND_(KS_, 2, false);     \
    else EXPAND_(KS_, 1, false);               \
  } while (0)
  if (a.r <= 16) EXPAND(0);
  else if (a.r <= 32) EXPAND(1);
  else if (a.r <= 64) EXPAND(2);
  else EXPAND(4);
#undef EXPAND
#undef EXPAND_
  return hipGetLastError();
}

int adapt_piece(int64_t T, int64_t n_in, int64_t n_out) {
  if (T <= 512) return 512;  // (one piece: no sums to add)
  const int64_t blocks = (n_in + kGradCols - 1) / kGradCols + (n_out + kGradCols - 1) / kGradCols;
  int piece = 1024;
  while (piece > 128 && T / piece * blocks < 256) piece /= 2;
  return piece;
}

hipError_t launch_adapt_grads(const AdaptRows &a, const AdaptGrads &g, int piece, hipStream_t s) {
  int64_t blocks;
  const GradArgs q = grad_args(a, g, piece, &blocks);
  const dim3 grid((uint32_t)blocks), block(256);
  const int ranks = (a.r + q.parts - 1) / q.parts;  // of a part
  if (ranks <= 16) launch(k_adapt_grads<1>, grid, block, 0, s, a, q);
  else if (ranks <= 32) launch(k_adapt_grads<2>, grid, block, 0, s, a, q);
  else if (ranks <= 48) launch(k_adapt_grads<3>, grid, block, 0, s, a, q);
  else launch(k_adapt_grads<4>, grid, block, 0, s, a, q);
  return hipGetLastError();
}

hipError_t launch_adapt_back(const AdaptRows &a, const AdaptGrads &g, int piece, const bf16_t *Q, const bf16_t *base,
                             bf16_t *dX, hipStream_t s) {
  int64_t eb, gb;
  const ExpandArgs x = expand_args(a, false, g.dU, g.dU_ranges, Q, g.n_in, false, base, dX, nullptr, &eb);
  const GradArgs q = grad_args(a, g, piece, &gb);
  const dim3 grid((uint32_t)(eb + gb)), block(256);
  const int e = (int)eb;
  if (a.r <= 16) launch(k_adapt_back<0, 1>, grid, block, 0, s, a, x, q, e);
  else if (a.r <= 32) launch(k_adapt_back<1, 2>, grid, block, 0, s, a, x, q, e);
  else if (a.r <= 64) launch(k_adapt_back<2, 4>, grid, block, 0, s, a, x, q, e);
  else launch(k_adapt_back<4, 4>, grid, block, 0, s, a, x, q, e);
  return hipGetLastError();
}

hipError_t launch_adapt_reduce(const AdaptRows &a, const AdaptGrads &g, int piece, hipStream_t s) {
  const int64_t ba = g.dA ? (a.r * g.n_in + 2047) / 2048 : 0, bb = g.dB ? (a.r * g.n_out + 2047) / 2048 : 0;
  launch(k_adapt_reduce, dim3((uint32_t)(ba + bb), (uint32_t)a.n_pool), dim3(256), 0, s, a, g, piece, ba);
  return hipGetLastError();
}

}  // namespace qlora
