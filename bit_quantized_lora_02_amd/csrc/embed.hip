// embed.hip -- the embedding beside the 4-bit linears: lookup with scaling, and its gradient by sorted tokens.
//
//   Y[t]  = bf16(scale W[token_t]),  0 where token_t lies outside the vocabulary
//   dW[v] = bf16((dW[v] +) scale sum_{t: token_t = v} dY[t])
//
// The lookup moves 4 bytes per value and computes next to nothing: it is bound by HBM (8192 x 8192 44 us, 5.6 TB/s).
// The gradient reads dY once and writes the whole of dW, nearly all of it zeros (a vocabulary of 128256 x 4096: 1.05 GB
// against 0.13 GB of 16384 rows of dY; 240 us in all, 150 of them the zeros).  Nothing is added atomically: the positions
// are sorted by token, stably, and each row of dW is the sum of its rows of dY in the order of their positions, cut into
// pieces at fixed places, so results repeat bit by bit.
//   1. k_embed_order  ranks the positions against each other; the workgroups that have no positions to rank fill dW with
//                     zeros, which takes longer, so the sort costs no time of its own where dW is large.
//   2. k_embed_merge  (more than kOrderChunk positions) merges the sorted chunks, four at a time.
//   3. k_embed_sum    a wave adds a piece of the sorted list over 512 columns; a row that lies in one piece is written at
//                     once.
//   4. k_embed_join   rows that were cut at the pieces' borders.
// Up to kEmbedFew tokens k_embed_few does all of it.
#include "step.h"
#include "step_device.h"

namespace qlora {
namespace {

constexpr int kWaveCols = 512;  // columns of a row that one wave takes: 16 bytes per lane

__global__ __launch_bounds__(256) void k_embed(const int64_t *__restrict__ tokens, int64_t T, const bf16_t *__restrict__ W,
                                               int64_t V, int64_t D, float scale, bf16_t *__restrict__ Y, int64_t chunks) {
  const int64_t per = D / 8;  // 16-byte chunks of a row
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks; c += (int64_t)gridDim.x * 256) {
    const int64_t t = c / per, d = (c - t * per) * 8;
    const int64_t v = tokens[t];
    u32x4_t o = {0u, 0u, 0u, 0u};
    if ((uint64_t)v < (uint64_t)V) {
      float x[8];
      unpack8(load16(W + v * D + d), x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= scale;
      o = pack8(x);
    }
    store16_once(Y + t * D + d, o);
  }
}

// Ranks 16 positions of a chunk against the whole chunk: the rank of position i is the number of keys below its own plus
// the number of equal ones before it.  16 threads count for each position, a sixteenth of 2048 keys at a time, which all
// read from LDS, two vector instructions per pair (8192 positions: 67 million pairs over the whole GPU, 6 us).
constexpr int kRankItems = 16, kRankParts = 16, kRankKeys = 2048, kRankPart = kRankKeys / kRankParts;
__device__ __forceinline__ void rank_chunk(const int64_t *__restrict__ tokens, int64_t T, int64_t V, int64_t block,
                                           int chunk, int32_t *__restrict__ order, int32_t *__restrict__ key) {
  __shared__ __attribute__((aligned(16))) uint32_t s_key[kRankParts][kRankPart + 4];
  __shared__ uint32_t s_rank[kRankParts][kRankItems];
  const int64_t first = block * kRankItems, base = first & -(int64_t)chunk;  // (a power of two)
  const int n = (int)(T - base < chunk ? T - base : chunk);
  const int tid = threadIdx.x, item = tid % kRankItems, part = tid / kRankItems;
  const int i0 = (int)(first - base), i = i0 + item;
  auto key_of = [&](int at, int64_t v) {  // (behind the end: above every key)
    return at >= n ? 0xffffffffu : (uint64_t)v < (uint64_t)V ? (uint32_t)v : (uint32_t)V;
  };
  int64_t next[kRankKeys / 256];
  auto load = [&](int j0) {
#pragma unroll
    for (int p = 0; p < kRankKeys / 256; ++p) {
      const int at = j0 + p * 256 + tid;
      next[p] = tokens[base + (at < n ? at : n - 1)];
    }
  };
  const int64_t token = tokens[base + (i < n ? i : n - 1)];
  load(0);
  const uint32_t mine = key_of(i, token);
  uint32_t rank = 0;
  for (int j0 = 0; j0 < n; j0 += kRankKeys) {
    if (j0) __syncthreads();
#pragma unroll
    for (int p = 0; p < kRankKeys / 256; ++p)
      s_key[(p * 256 + tid) / kRankPart][tid % kRankPart] = key_of(j0 + p * 256 + tid, next[p]);
    if (j0 + kRankKeys < n) load(j0 + kRankKeys);
    __syncthreads();
    const int lo = j0 + part * kRankPart;
#pragma unroll 1
    for (int j = 0; j < kRankPart; j += kRankItems) {
      const uint32_t *const at = &s_key[part][j];
      if (lo + j == i0) {
#pragma unroll
        for (int e = 0; e < kRankItems; ++e) rank += at[e] < mine + (e < item ? 1u : 0u) ? 1u : 0u;
      } else {
        const uint32_t below = mine + (lo + j < i0 ? 1u : 0u);
#pragma unroll
        for (int e = 0; e < kRankItems; e += 4) {
          const u32x4_t k = *reinterpret_cast<const u32x4_t *>(at + e);
          rank += (k[0] < below ? 1u : 0u) + (k[1] < below ? 1u : 0u) + (k[2] < below ? 1u : 0u) + (k[3] < below ? 1u : 0u);
        }
      }
    }
  }
  s_rank[part][item] = rank;
  __syncthreads();
  if (part == 0 && i < n) {
    uint32_t r = 0;
#pragma unroll
    for (int p = 0; p < kRankParts; ++p) r += s_rank[p][item];
    order[base + r] = (int32_t)(base + i);
    key[base + r] = (int32_t)mine;
  }
}
static_assert(kRankItems * kRankParts == 256 && 256 % kRankPart == 0 && kRankPart % kRankItems == 0, "layout of the keys");

// The rest of the workgroups fill: one store per thread, which reaches 6.8 TB/s (1.05 GB in 154 us; workgroups that stay
// for several stores 4.4 to 6.2, nontemporal stores 4.4).
__global__ __launch_bounds__(256) void k_embed_order(const int64_t *__restrict__ tokens, int64_t T, int64_t V,
                                                     int chunk, int32_t *__restrict__ order, int32_t *__restrict__ key,
                                                     int64_t blocks, bf16_t *__restrict__ fill, int64_t fill_n) {
  if (blockIdx.x < blocks) {
    rank_chunk(tokens, T, V, blockIdx.x, chunk, order, key);
    return;
  }
  const int64_t e = ((int64_t)(blockIdx.x - blocks) * 256 + threadIdx.x) * 8;
  if (e < fill_n) store16(fill + e, u32x4_t{0u, 0u, 0u, 0u});
}

// Merges sorted runs of `run` places (a power of two), four at a time: a place goes behind, in each earlier run of the
// four, the keys not above its own and, in each later one, those below.  The four searches go in step, so that a step waits
// for memory once.
constexpr int kMergeRuns = 4;
__global__ __launch_bounds__(256) void k_embed_merge(int64_t T, int64_t run, const int32_t *__restrict__ order,
                                                     const int32_t *__restrict__ key, int32_t *__restrict__ order_out,
                                                     int32_t *__restrict__ key_out) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= T) return;
  const int64_t own = p / run, first = own / kMergeRuns * kMergeRuns;
  const int k = key[p], position = order[p];
  const int32_t *from[kMergeRuns];
  int n[kMergeRuns], limit[kMergeRuns], below[kMergeRuns];
#pragma unroll
  for (int c = 0; c < kMergeRuns; ++c) {
    const int64_t base = (first + c) * run, left = T - base;
    n[c] = first + c == own || left <= 0 ? 0 : (int)(left < run ? left : run);
    from[c] = key + (n[c] ? base : p);
    limit[c] = first + c < own ? k + 1 : k;
    below[c] = 0;
  }
  for (int step = (int)run; step; step >>= 1)
#pragma unroll
    for (int c = 0; c < kMergeRuns; ++c) {  // (the keys below the limit are the first of the run)
      const int m = below[c] + step;
      if (from[c][m <= n[c] ? m - 1 : 0] < limit[c] && m <= n[c]) below[c] = m;
    }
  int64_t at = first * run + (p - own * run);
#pragma unroll
  for (int c = 0; c < kMergeRuns; ++c) at += below[c];
  order_out[at] = position;
  key_out[at] = k;
}

__device__ __forceinline__ void write_row(bf16_t *__restrict__ at, const float sum[8], float scale, bool add) {
  float o[8];
  if (add) {
    unpack8(load16(at), o);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf(sum[i], scale, o[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = sum[i] * scale;
  }
  store16(at, pack8(o));
}

// One piece of the sorted list, 512 columns.  A row whose positions all lie in the piece is written; the binary32 sum of
// one that began in an earlier piece goes to part[piece][0], of one that begins here and goes on to part[piece][1].  Each
// lane holds an entry of the list, so that the rows' loads wait for nothing else.
constexpr int kPieceMost = 32;
__global__ __launch_bounds__(256) void k_embed_sum(const int32_t *__restrict__ order, const int32_t *__restrict__ key,
                                                   int64_t T, int piece, const bf16_t *__restrict__ dY, int64_t V, int64_t D,
                                                   int64_t slices, int64_t jobs, float scale, bool add,
                                                   bf16_t *__restrict__ dW, float *__restrict__ part) {
  constexpr int N = 8;  // rows in flight
  const int64_t job = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (job >= jobs) return;
  const int lane = threadIdx.x & 63;
  const int64_t c = job / slices, d = (job - c * slices) * kWaveCols + lane * 8;
  const int64_t p0 = c * piece;
  const int n = (int)(T - p0 < piece ? T - p0 : piece);
  // lane i: the key at place p0 - 1 + i, up to the one behind the piece (none: -1), and the position at p0 + i
  const int64_t p = p0 - 1 + lane;
  const int k = lane <= n + 1 && p >= 0 && p < T ? key[p] : -1;
  const int row = lane < n ? order[p0 + lane] : 0;
  const int first = __builtin_amdgcn_readlane(k, 1);
  if (first >= V) return;  // what names no row comes last
  const int count = __popcll(__ballot(lane >= 1 && lane <= n && k < V));
  const bool in = d < D;
  const bf16_t *const from = dY + (in ? d : 0);
  bool head = __builtin_amdgcn_readlane(k, 0) == first;
  int cur = first;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto flush = [&](bool goes_on) {
    if (!in) return;
    if (!head && !goes_on) {
      write_row(dW + (int64_t)cur * D + d, sum, scale, add);
    } else {
      float *at = part + ((c * 2 + (head ? 0 : 1)) * D + d);
      *reinterpret_cast<float4 *>(at) = make_float4(sum[0], sum[1], sum[2], sum[3]);
      *reinterpret_cast<float4 *>(at + 4) = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
  };
  u32x4_t now[N], next[N];
  auto load = [&](u32x4_t(&to)[N], int e0) {  // (behind the last entry: its row again, not added)
#pragma unroll
    for (int e = 0; e < N; ++e)
      to[e] = load16(from + (int64_t)__builtin_amdgcn_readlane(row, e0 + e < count ? e0 + e : count - 1) * D);
  };
  auto take = [&](const u32x4_t(&rows)[N], int e0) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (e0 + e >= count) break;
      const int at = __builtin_amdgcn_readlane(k, e0 + e + 1);
      if (at != cur) {
        flush(false);
        cur = at;
        head = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
      }
      float x[8];
      unpack8(rows[e], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += x[i];
    }
  };
  load(now, 0);
  for (int e0 = 0; e0 < count; e0 += 2 * N) {
    if (e0 + N < count) load(next, e0 + N);
    take(now, e0);
    if (e0 + N >= count) break;
    if (e0 + 2 * N < count) load(now, e0 + 2 * N);
    take(next, e0 + N);
  }
  flush(count == n && __builtin_amdgcn_readlane(k, n + 1) == cur);
}

// The row that begins in a piece and goes on: its sums of the pieces, added in order (four waves a quarter of them each,
// then the quarters).
__global__ __launch_bounds__(256) void k_embed_join(const int32_t *__restrict__ key, int64_t T, int piece, int64_t V,
                                                    int64_t D, int64_t slices, float scale, bool add,
                                                    bf16_t *__restrict__ dW, const float *__restrict__ part) {
  __shared__ float s_sum[3][64][9];
  const int64_t c = blockIdx.x / slices;
  const int64_t p0 = c * piece, p1 = p0 + piece;
  if (p1 >= T) return;
  const int cur = key[p1 - 1];
  if (cur >= V || key[p1] != cur) return;              // its last row ends in it
  if (p0 > 0 && key[p0] == cur && key[p0 - 1] == cur) return;  // begins in an earlier piece
  int64_t lo = p1, hi = T;                             // the first place behind the row
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (key[mid] <= cur) lo = mid + 1;
    else hi = mid;
  }
  const int64_t last = (lo - 1) / piece, n = last - c;  // pieces that continue it
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t d = (blockIdx.x - c * slices) * kWaveCols + lane * 8;
  const bool in = d < D;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int64_t per = (n + 3) / 4, a = c + 1 + wave * per, b = a + per < last + 1 ? a + per : last + 1;
  if (in) {
    if (wave == 0) {
      const float4 *at = reinterpret_cast<const float4 *>(part + (c * 2 + 1) * D + d);
      const float4 x = at[0], y = at[1];
      sum[0] = x.x, sum[1] = x.y, sum[2] = x.z, sum[3] = x.w, sum[4] = y.x, sum[5] = y.y, sum[6] = y.z, sum[7] = y.w;
    }
#pragma unroll 8
    for (int64_t q = a; q < b; ++q) {
      const float4 *at = reinterpret_cast<const float4 *>(part + q * 2 * D + d);
      const float4 x = at[0], y = at[1];
      sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w;
      sum[4] += y.x, sum[5] += y.y, sum[6] += y.z, sum[7] += y.w;
    }
  }
  if (wave > 0)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sum[wave - 1][lane][i] = sum[i];
  __syncthreads();
  if (wave == 0 && in) {
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += s_sum[w][lane][i];
    write_row(dW + (int64_t)cur * D + d, sum, scale, add);
  }
}

// Few tokens, one launch: each lane of a wave holds L of them, 64 apart.  A thread fills 8 columns with zeros, as above, or
// adds them up where a token names their row; with ADD a workgroup takes 2048 columns of the row of token blockIdx.x /
// slices, unless an earlier token names it too.  (16 tokens of 50000 x 1024 16.3 us, with the sort 20.6; 128 of 1000 x
// 1024 8 and 13.  256 tokens that are all the same would take 26, with the sort 14: they are added eight at a time.)
template <int L, bool ADD>
__global__ __launch_bounds__(256) void k_embed_few(const int64_t *__restrict__ tokens, int T, const bf16_t *__restrict__ dY,
                                                   int64_t V, int64_t D, float scale, bf16_t *__restrict__ dW,
                                                   uint32_t slices) {
  const int lane = threadIdx.x & 63;
  int64_t v[L];
  int key[L];
#pragma unroll
  for (int l = 0; l < L; ++l) v[l] = tokens[l * 64 + lane < T ? l * 64 + lane : T - 1];
#pragma unroll
  for (int l = 0; l < L; ++l) key[l] = l * 64 + lane < T && (uint64_t)v[l] < (uint64_t)V ? (int)v[l] : -1;
  const uint32_t per = (uint32_t)(D / 8), chunks = per * (uint32_t)V;  // (at most 2^31)
  int row, first, last;  // of this thread; of the workgroup
  uint32_t c;            // 16-byte chunk of the row
  bool in;               // (behind the end a thread stays, whose lane holds a token)
  if (ADD) {
    const int t = blockIdx.x / slices;
    row = -1;
#pragma unroll
    for (int l = 0; l < L; ++l)
      if (t >> 6 == l) row = __builtin_amdgcn_readlane(key[l], t & 63);
    first = last = row;
    c = (blockIdx.x - t * slices) * 256 + threadIdx.x;
    if (row < 0) return;
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const uint64_t same = __ballot(key[l] == row);
      if (l < t >> 6 ? same != 0 : l == t >> 6 && (same & (((uint64_t)1 << (t & 63)) - 1)) != 0) return;
    }
    in = c < per;
  } else {
    const uint32_t c0 = blockIdx.x * 256u, c1 = chunks - c0 > 255 ? c0 + 255 : chunks - 1;
    first = (int)(c0 / per), last = (int)(c1 / per);
    in = threadIdx.x <= c1 - c0;
    c = in ? c0 + threadIdx.x : c1;
    row = (int)(c / per);
    c -= (uint32_t)row * per;
  }
  if (!in) c = 0;
  bf16_t *const to = dW + ((int64_t)row * D + c * 8);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  uint64_t named[L], any = 0;
#pragma unroll
  for (int l = 0; l < L; ++l) any |= named[l] = __ballot(key[l] >= first && key[l] <= last);
  if (!ADD && any == 0) {
    if (in) store16(to, u32x4_t{0u, 0u, 0u, 0u});
    return;
  }
  constexpr int N = 8;  // rows in flight
  bool mine = ADD;      // a token names this thread's row
#pragma unroll
  for (int l = 0; l < L; ++l)
    for (uint64_t left = named[l]; left;) {
      u32x4_t x[N];
      int of[N], t = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {  // (behind the last: its row again, not added)
        if (left) t = __builtin_ctzll(left);
        of[i] = left ? __builtin_amdgcn_readlane(key[l], t) : -1;
        x[i] = load16(dY + (int64_t)(l * 64 + t) * D + c * 8);
        left &= left - 1;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float y[8];
        unpack8(x[i], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = of[i] == row ? sum[e] + y[e] : sum[e];
        mine |= of[i] == row;
      }
    }
  if (in) write_row(to, sum, mine ? scale : 0.f, ADD);
}

int64_t slices_of(int64_t D) { return (D + kWaveCols - 1) / kWaveCols; }

}  // namespace

hipError_t launch_embed(const int64_t *tokens, int64_t T, const bf16_t *W, int64_t V, int64_t D, float scale, bf16_t *Y,
                        hipStream_t s) {
  const int64_t chunks = T * (D / 8), blocks = (chunks + 255) / 256;
  launch(k_embed, dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, tokens, T, W, V, D, scale, Y, chunks);
  return hipGetLastError();
}

// (enough pieces to fill the GPU)
int embed_piece(int64_t T) { return T <= 2048 ? 8 : T <= 8192 ? 16 : kPieceMost; }

hipError_t launch_embed_few(const int64_t *tokens, int64_t T, const bf16_t *dY, int64_t V, int64_t D, float scale, bool add,
                            bf16_t *dW, hipStream_t s) {
  const int64_t slices = (D + 2047) / 2048, blocks = add ? T * slices : (V * (D / 8) + 255) / 256;
#define FEW(L_)                                                                                                       \
  do {                                                                                                                \
    if (add) launch(k_embed_few<L_, true>, grid, block, 0, s, tokens, (int)T, dY, V, D, scale, dW, (uint32_t)slices); \
    else launch(k_embed_few<L_, false>, grid, block, 0, s, tokens, (int)T, dY, V, D, scale, dW, (uint32_t)slices);    \
  } while (0)
  const dim3 grid((uint32_t)blocks), block(256);
  if (T <= 64) FEW(1);
  else FEW(2);
#undef FEW
  return hipGetLastError();
}

// Positions that are ranked against each other: ranking costs T x chunk, and up to four chunks take one pass of the merge
// (131072 positions: ranked in 87 us 8192 at a time, in 29 us 2048 at a time with one pass more, which takes 7).
static int64_t order_chunk(int64_t T) {
  const int64_t c = T <= kOrderChunk || T > 2 * kOrderChunk ? kOrderChunk : kOrderChunk / 2;
  return T <= kMergeRuns * c ? c : kOrderChunk / 4;
}
int embed_passes(int64_t T) {
  int n = 0;
  for (int64_t run = order_chunk(T); run < T; run *= kMergeRuns) ++n;
  return n;
}

// (each pass goes from one pair of lists to the other, the last one to order and key)
hipError_t launch_embed_order(const int64_t *tokens, int64_t T, int64_t V, const Order &o, bf16_t *fill, int64_t fill_n,
                              hipStream_t s) {
  const int64_t blocks = (T + kRankItems - 1) / kRankItems, fills = (fill_n + 2047) / 2048;
  const bool second = embed_passes(T) & 1;
  launch(k_embed_order, dim3((uint32_t)(blocks + fills)), dim3(256), 0, s, tokens, T, V, (int)order_chunk(T),
         second ? o.order2 : o.order, second ? o.key2 : o.key, blocks, fill, fill_n);
  return hipGetLastError();
}

hipError_t launch_embed_merge(int64_t T, int pass, const Order &o, hipStream_t s) {
  int64_t run = order_chunk(T);
  for (int i = 0; i < pass; ++i) run *= kMergeRuns;
  const bool second = (embed_passes(T) - pass) & 1;
  launch(k_embed_merge, dim3((uint32_t)((T + 255) / 256)), dim3(256), 0, s, T, run,
         (const int32_t *)(second ? o.order2 : o.order), (const int32_t *)(second ? o.key2 : o.key),
         second ? o.order : o.order2, second ? o.key : o.key2);
  return hipGetLastError();
}

hipError_t launch_embed_sum(const Order &o, int64_t T, const bf16_t *dY, int64_t V, int64_t D, float scale, bool add,
                            bf16_t *dW, float *part, hipStream_t s) {
  const int piece = embed_piece(T);
  const int64_t slices = slices_of(D), jobs = (T + piece - 1) / piece * slices;
  launch(k_embed_sum, dim3((uint32_t)((jobs + 3) / 4)), dim3(256), 0, s, (const int32_t *)o.order, (const int32_t *)o.key, T,
         piece, dY, V, D, slices, jobs, scale, add, dW, part);
  return hipGetLastError();
}

hipError_t launch_embed_join(const Order &o, int64_t T, int64_t V, int64_t D, float scale, bool add, bf16_t *dW,
                             const float *part, hipStream_t s) {
  const int piece = embed_piece(T);
  const int64_t slices = slices_of(D), pieces = (T + piece - 1) / piece;
  launch(k_embed_join, dim3((uint32_t)(pieces * slices)), dim3(256), 0, s, (const int32_t *)o.key, T, piece, V, D, slices,
         scale, add, dW, part);
  return hipGetLastError();
}

}  // namespace qlora
