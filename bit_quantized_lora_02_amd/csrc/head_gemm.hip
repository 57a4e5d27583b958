// head_gemm.hip -- the three products of the output layer's losses on bf16 MFMAs:
//
//   logits   z = X W^T       per tile: softmax statistics, and E = exp2((z - u) c) in bf16 (never z itself)
//   dX       dX = f o (E W)  reduction over the vocabulary, f the rows' factors
//   dW       dW = E^T (f o X)  reduction over the rows
//
// (E with its targets' entries put in by k_head_combine; see head_loss.hip for the mathematics.)
//
// One kernel body serves all three: C[n][m] = sum_r A(m, r) B(n, r), the operands read from global memory either
// along the reduction ("rows": [m][r]) or across it ("transposed": [r][m]).  A workgroup of 4 or 8 waves computes a
// 256 x BN tile with v_mfma_f32_32x32x16_bf16; m is the MFMA's row index, so a lane holds four consecutive m of
// one n, which makes the softmax statistics of a row of X (n) a reduction inside the lane.  The reduction runs in
// 32-deep steps over a ring of four LDS tiles that the load unit fills directly (16 bytes per lane, see
// reduce_steps).
//
// LDS tiles: "rows" [row][32] with the 16-byte chunk index XOR-swizzled by (row / 4) % 4; "transposed" [32][cols]
// with the 64-byte groups of a row XOR-swizzled by row % 4 (a transposing read takes four rows at once), both
// conflict-free; the direct copies write lane-consecutive LDS, so the swizzle is applied to the source address.
#include <type_traits>

#include "device.h"
#include "head.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int BK = 32;      // reduction depth of a step
constexpr int STAGES = 4;   // tiles in LDS: one being multiplied, three on their way
constexpr int BM = kHeadTile;

template <int WAVES_M_, int WAVES_N_, int WM_, int WN_>
struct HeadCfg {
  static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WM = WM_, WN = WN_;
  static constexpr int NW = WAVES_M * WAVES_N, NT = 64 * NW;
  static constexpr int BN = WAVES_N * WN * 32;
  static_assert(WAVES_M * WM * 32 == BM, "tiles are 256 wide");
};
using H256 = HeadCfg<2, 4, 4, 2>;  // 128 x 64 per wave
using H128 = HeadCfg<4, 2, 2, 2>;  // 64 x 64 per wave
using H64 = HeadCfg<4, 1, 2, 2>;   // 64 x 64 per wave, two workgroups per CU

__device__ __forceinline__ void fence_sched() { __builtin_amdgcn_sched_barrier(0); }

// How an operand lies in memory (element (i, r): row or column i of the tile's side, reduction index r):
//  LINES:   row-major [i][r].
//  BLOCKS:  32 reduction indices at a time, [r / 32][i][32]: a step's tile is one contiguous piece, where LINES
//           would fetch half of every 128-byte line it touches in one step and the other half in the next.
//  ACROSS:  row-major [r][i].
//  BLOCKS_ACROSS: [i / 32][r][32], what BLOCKS is seen from its other side.
enum { LINES, BLOCKS, ACROSS, BLOCKS_ACROSS };

// One operand's tile of ROWS rows (columns for the ACROSS ones).  `ld` is the row length of a row-major matrix, the
// number of rows in a block otherwise.  Rows may be gathered through `list`; those past the last one repeat it.
// Reduction indices from the reduction's length on read as zero (BLOCKS are zero there in memory).  A step's
// addresses are a wave-uniform base plus 32-bit lane offsets that do not change from step to step.
template <int ROWS, int NT, int KIND>
struct Tile {
  static constexpr bool TR = KIND == ACROSS || KIND == BLOCKS_ACROSS;
  static constexpr int LD = ROWS * BK / 8 / NT;  // 16-byte copies per thread and step
  static constexpr int NW = NT / 64;
  static constexpr int CH = ROWS / 8;  // across: 16-byte chunks per LDS row, and LDS rows from copy to copy
  static constexpr int RSTEP = NW * 64 / CH;
  static_assert(ROWS * BK / 8 % NT == 0 && LD >= 1, "unsupported tile");
  static_assert(!TR || (64 % CH == 0 && RSTEP % 4 == 0), "the copies of a thread share one swizzle");
  const char *base;  // reduction index 0 of the tile
  uint32_t off[TR ? 1 : LD];
  int64_t ld;
  int wave;

  __device__ __forceinline__ void init(const bf16_t *src, int64_t ld_, int64_t first, int64_t count,
                                       const int32_t *list, int w, int lane) {
    ld = ld_, wave = w;
    const int k0 = first_index(w, lane);
    if constexpr (!TR) {
      const int64_t row = KIND == BLOCKS ? BK : ld;
      base = (const char *)(list ? src : src + first * row);
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int rr = 16 * (i * NW + w) + (lane >> 2);
        const int64_t at = first + rr < count ? rr : count - 1 - first;
        off[i] = (uint32_t)(((list ? list[first + at] : at) * row + k0) * 2);
      }
    } else {
      int64_t c = first + 8 * ((lane % CH) ^ (swz(k0) << 2));
      if (c > count - 8) c = count - 8;  // count % 8 == 0
      if constexpr (KIND == ACROSS) {
        base = (const char *)src;
        off[0] = (uint32_t)((k0 * ld + c) * 2);
      } else {
        base = (const char *)(src + first / 32 * ld * 32);
        off[0] = (uint32_t)((((c - first) / 32 * ld + k0) * 32 + c % 32) * 2);
      }
    }
  }
  // XOR of the 64-byte group index of LDS row r: rows r .. r + 3 then start in different quarters of the 64 banks
  static __device__ __forceinline__ int swz(int r) { return ROWS >= 128 ? (r & 3) : ((r >> 1) & 1); }
  // Reduction index within a step of this thread's first copy (rows: of all, their rows / 4 are equal modulo 4).
  static __device__ __forceinline__ int first_index(int w, int lane) {
    return TR ? w * (64 / CH) + lane / CH : 8 * ((lane & 3) ^ ((lane >> 4) & 3));
  }
  __device__ __forceinline__ const char *at(int64_t step) const {
    return base + step * (KIND == ACROSS || KIND == BLOCKS ? ld * (2 * BK) : KIND == LINES ? 2 * BK : 64 * BK);
  }
  __device__ __forceinline__ int64_t next(int i) const {  // bytes from an across operand's first copy to copy i
    return KIND == ACROSS ? i * (ld * (2 * RSTEP)) : KIND == BLOCKS_ACROSS ? i * 64 * RSTEP : 0;
  }
  // Copy i of this thread.  (Buffer loads take the uniform part of the address in scalar registers; the descriptor
  // spans all of memory behind the base, every address is inside the operand by construction.)
  __device__ __forceinline__ void issue(int64_t step, int i, bf16_t *s) const {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)at(step), 0, -1, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void *)(s + (i * NW + wave) * 512), 16, off[TR ? 0 : i], (int)next(i),
        0, 0);
  }
  // The last step of a reduction that is no multiple of 32 deep: through registers, `left` < 32 indices remain.
  __device__ __forceinline__ void issue_part(int64_t step, int left, bf16_t *s) const {
    const int lane = threadIdx.x & 63, k0 = first_index(wave, lane);
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      u32x4_t v = u32x4_t{0u, 0u, 0u, 0u};
      if (KIND == BLOCKS || k0 + (TR ? i * RSTEP : 0) < left)
        v = *reinterpret_cast<const u32x4_t *>(at(step) + off[TR ? 0 : i] + next(i));
      *reinterpret_cast<u32x4_t *>(s + (i * NW + wave) * 512 + lane * 8) = v;
    }
  }
  // MFMA operand of the 32 rows from `at`, reduction 16 kk .. 16 kk + 15 of the step
  static __device__ __forceinline__ u32x4_t read(const bf16_t *s, int at, int kk, int lane) {
    if constexpr (!TR) {
      const int r = at + (lane & 31), chunk = kk * 2 + (lane >> 5);
      return *reinterpret_cast<const u32x4_t *>(s + r * BK + ((chunk ^ ((r >> 2) & 3)) << 3));
    } else {
      // In each 16-lane group, lane i of a transposing read gets element (i & 3) of the 8 bytes addressed by lane
      // 4 m + (i >> 2): lane a points at row base + (a >> 2), columns 4 (a & 3) .. + 3, and the reads of rows + 0..3
      // and + 4..7 give its 8 reduction values.
      typedef short s4_t __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s4_t lds_s4;
      const int grp = lane >> 4, ai = lane & 15;
      const int r = kk * 16 + 8 * (grp >> 1) + (ai >> 2);
      const int c = at + 16 * (grp & 1) + 4 * (ai & 3);
      const int off = r * ROWS + (c ^ (swz(r) << 5));  // r and r + 4 have the same swizzle
      const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(s + off));
      const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(s + off + 4 * ROWS));
      const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
      return u32x4_t{l2.x, l2.y, h2.x, h2.y};
    }
  }
};

template <class C>
using Acc = f32x16_t[C::WM][C::WN];

// The LDS tiles of one workgroup.  Each is an array of its own, so that the compiler can tell reads of one from the
// direct copies into another and adds no waits.
template <class C>
struct Ring {
  bf16_t *a[STAGES], *b[STAGES];
};
#define QLORA_RING(C, ring)                                                                            \
  __shared__ __attribute__((aligned(16))) bf16_t ra0[BM * BK], ra1[BM * BK], ra2[BM * BK], ra3[BM * BK];   \
  __shared__ __attribute__((aligned(16))) bf16_t rb0[C::BN * BK], rb1[C::BN * BK], rb2[C::BN * BK], rb3[C::BN * BK]; \
  const Ring<C> ring = {{ra0, ra1, ra2, ra3}, {rb0, rb1, rb2, rb3}}

// Wait until at most VM vector-memory operations are in flight and all LDS operations are done, then meet the
// workgroup's other waves (without the full memory fence of __syncthreads, which would wait for every copy).
// s_waitcnt fields: vmcnt[3:0] and [15:14], expcnt[6:4] (7 = no wait), lgkmcnt[11:8].
template <int VM>
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_s_waitcnt((VM & 15) | (VM >> 4 << 14) | 0x0070);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The reduction over steps [s0, s1) into acc; `red` is the reduction's length.
//
// Step s multiplies the tiles of slot s % 4 while the copies of steps s + 1 .. s + 3 are in flight.  Its first MFMAs'
// operands are in registers; the second half's are read under them; then the waves meet (every wave holds the last
// operands of slot s, and step s + 1 has landed), read the first operands of step s + 1 and run the second half's
// MFMAs.  The copies of step s + 3 (into the slot of step s - 1, which all waves have left) are issued one at a time
// between the MFMAs: issued together they would hold the waves up for as long as the load unit takes to accept them.
template <class C, int KA, int KB>
__device__ __forceinline__ void reduce_steps(const Tile<BM, C::NT, KA> &ta, const Tile<C::BN, C::NT, KB> &tb,
                                             int64_t red, int64_t s0, int64_t s1, const Ring<C> &ring, int wm, int wn, int lane,
                                             Acc<C> &acc) {
  typedef Tile<BM, C::NT, KA> TileA;
  typedef Tile<C::BN, C::NT, KB> TileB;
  constexpr int L = TileA::LD + TileB::LD, L1 = L / 2;  // copies per thread and step, those before the meeting
#pragma unroll
  for (int i = 0; i < C::WM; ++i)
#pragma unroll
    for (int j = 0; j < C::WN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  if (s0 >= s1) return;
  u32x4_t a[2][C::WM], b[2][C::WN];
  auto read = [&](int slot, int kk) {
#pragma unroll
    for (int i = 0; i < C::WM; ++i) a[kk][i] = TileA::read(ring.a[slot], (wm * C::WM + i) * 32, kk, lane);
#pragma unroll
    for (int j = 0; j < C::WN; ++j) b[kk][j] = TileB::read(ring.b[slot], (wn * C::WN + j) * 32, kk, lane);
  };
  auto copy = [&](int64_t s, int slot, int q) {
    if (q < TileA::LD)
      ta.issue(s, q, ring.a[slot]);
    else
      tb.issue(s, q - TileA::LD, ring.b[slot]);
  };
  auto copy_all = [&](int64_t s, int slot) {
    if ((s + 1) * BK <= red) {
#pragma unroll
      for (int q = 0; q < L; ++q) copy(s, slot, q);
    } else {
      ta.issue_part(s, (int)(red - s * BK), ring.a[slot]);
      tb.issue_part(s, (int)(red - s * BK), ring.b[slot]);
    }
  };
  // the MFMAs of half kk with copies [q0, q1) of step s spread among them
  auto mma = [&](int kk, int64_t s, int slot, int q0, int q1) {
#pragma unroll
    for (int i = 0; i < C::WM; ++i) {
#pragma unroll
      for (int j = 0; j < C::WN; ++j) acc[i][j] = mfma_32x32x16(a[kk][i], b[kk][j], acc[i][j]);
      fence_sched();
#pragma unroll
      for (int q = q0 + (q1 - q0) * i / C::WM; q < q0 + (q1 - q0) * (i + 1) / C::WM; ++q) {
        copy(s, slot, q);
        fence_sched();
      }
    }
  };
  const int64_t whole = red / BK < s1 ? red / BK : s1;  // steps before this one are full
#pragma unroll
  for (int q = 0; q < STAGES - 1; ++q)
    if (s0 + q < s1) copy_all(s0 + q, q);
  if (s0 + STAGES - 1 <= whole)
    meet<2 * L>();
  else
    meet<0>();
  read(0, 0);
  // steady state: copies of step s + 3 are issued, those of s + 2 and the first ones of s + 3 stay in flight
  auto step = [&](auto pc, int64_t s) {
    constexpr int P = decltype(pc)::value;
    read(P, 1);
    fence_sched();
    mma(0, s + 3, (P + 3) % STAGES, 0, L1);
    meet<L + L1>();
    read((P + 1) % STAGES, 0);
    fence_sched();
    mma(1, s + 3, (P + 3) % STAGES, L1, L);
  };
  // the last steps: at most a part step is still to be copied; everything is waited for
  auto last = [&](auto pc, int64_t s) {
    constexpr int P = decltype(pc)::value;
    read(P, 1);
    if (s + 3 < s1) copy_all(s + 3, (P + 3) % STAGES);
    fence_sched();
    mma(0, 0, 0, 0, 0);
    meet<0>();
    if (s + 1 < s1) read((P + 1) % STAGES, 0);
    fence_sched();
    mma(1, 0, 0, 0, 0);
  };
  int64_t s = s0;
  for (; s + STAGES + 2 < whole; s += STAGES) {  // s + 3 + 3 < whole: four steady steps
    step(std::integral_constant<int, 0>(), s);
    step(std::integral_constant<int, 1>(), s + 1);
    step(std::integral_constant<int, 2>(), s + 2);
    step(std::integral_constant<int, 3>(), s + 3);
  }
  for (; s < s1; s += STAGES) {
    last(std::integral_constant<int, 0>(), s);
    if (s + 1 < s1) last(std::integral_constant<int, 1>(), s + 1);
    if (s + 2 < s1) last(std::integral_constant<int, 2>(), s + 2);
    if (s + 3 < s1) last(std::integral_constant<int, 3>(), s + 3);
  }
  meet<0>();  // the tiles may be reused
}

// Work item of this workgroup: items are numbered so that each XCD (workgroups go round the 8 XCDs) takes a run of
// consecutive ones, and consecutive ones are blocks of 4 m-tiles x all n-tiles: the 32 workgroups of an XCD then
// share 4 + 8 operand tiles.
struct Item {
  int64_t m, n;
  int range;
};
__device__ __forceinline__ bool item_of(int64_t tiles_m, int64_t tiles_n, int ranges, Item *it) {
  const int64_t total = tiles_m * tiles_n * ranges, per = (total + 7) / 8;
  const int64_t lin = blockIdx.x, id = (lin & 7) * per + (lin >> 3);
  if ((lin >> 3) >= per || id >= total) return false;
  const int64_t in = id % (tiles_m * tiles_n);
  it->range = (int)(id / (tiles_m * tiles_n));
  const int64_t band = in / (4 * tiles_n), left = in % (4 * tiles_n);
  const int64_t wide = tiles_m - band * 4 < 4 ? tiles_m - band * 4 : 4;
  it->m = band * 4 + left % wide;
  it->n = left / wide;
  return true;
}

__device__ __forceinline__ int64_t block_rows(const HeadRows &rows, int64_t row0, int64_t tb) {
  const int64_t n = *rows.n - row0;
  return n < tb ? n : tb;
}

// ------------------------------------------------------------------ logits
// m: columns of the vocabulary, n: counted rows of the block.
// X row-major (LINES) or as k_head_prep lays it out (BLOCKS, ldx rows per block).
template <class C, int KX>
__global__ __launch_bounds__(C::NT) void k_head_logits(HeadRows rows, int64_t row0, int64_t tb,
                                                       const bf16_t *__restrict__ X, int64_t ldx,
                                                       const bf16_t *__restrict__ W, int64_t V, int64_t K, float c,
                                                       float2 *__restrict__ stat, int64_t ntile,
                                                       bf16_t *__restrict__ E, int64_t lde, int64_t te) {
  QLORA_RING(C, ring);
  __shared__ float s_max[C::WAVES_M][C::BN], s_sum[C::WAVES_M][C::BN];
  const int64_t n = block_rows(rows, row0, tb);
  if (n <= 0) return;
  Item it;
  if (!item_of(ntile, (n + C::BN - 1) / C::BN, 1, &it)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  const int64_t m0 = it.m * BM, n0 = it.n * C::BN;
  Tile<BM, C::NT, LINES> ta;
  Tile<C::BN, C::NT, KX> tbl;
  ta.init(W, K, m0, V, nullptr, wave, lane);
  tbl.init(X, ldx, n0, n, rows.list + row0, wave, lane);
  f32x16_t acc[C::WM][C::WN];
  reduce_steps<C, LINES, KX>(ta, tbl, K, 0, (K + BK - 1) / BK, ring, wm, wn, lane, acc);

  // element e of acc[i][j]: column m0 + mi + 8 (e / 4) + e % 4, row n0 + nj (nj per lane)
  const int mlane = wm * C::WM * 32 + 4 * (lane >> 5);
  float ref[C::WN];
#pragma unroll
  for (int j = 0; j < C::WN; ++j) {
    const int nj = (wn * C::WN + j) * 32 + (lane & 31);
    const int64_t row = n0 + nj < n ? n0 + nj : n - 1;
    const int64_t t = rows.list[row0 + row];
    ref[j] = rows.ref[t];
    const int64_t rc = rows.refcol[t] - m0;  // the reference's own column stays out of the sums
    if (__any((rc >= 0 && rc < BM) || m0 + BM > V)) {
#pragma unroll
      for (int i = 0; i < C::WM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int m = mlane + 32 * i + 8 * (e >> 2) + (e & 3);
          if (m == rc || m0 + m >= V) acc[i][j][e] = -INFINITY;
        }
    }
    float top = acc[0][j][0];
#pragma unroll
    for (int i = 0; i < C::WM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
    top = fmaxf(top, __shfl_xor(top, 32));
    if (lane < 32) s_max[wm][nj] = top;
  }
  __syncthreads();
  // E's tile is turned through the ring's arrays, 32 rows of 256 columns in each (the narrow tiles use the first ones)
  auto stage = [&](int i) {
    return i == 0 ? ra0 : i == 1 ? ra1 : i == 2 ? ra2 : i == 3 ? ra3 : i == 4 ? rb0 : i == 5 ? rb1 : i == 6 ? rb2 : rb3;
  };
#pragma unroll
  for (int j = 0; j < C::WN; ++j) {
    const int nj = (wn * C::WN + j) * 32 + (lane & 31);
    float top = s_max[0][nj];
#pragma unroll
    for (int w = 1; w < C::WAVES_M; ++w) top = fmaxf(top, s_max[w][nj]);
    const float u = (top - ref[j]) * c > kHeadRange ? top : ref[j];
    float sum = 0.f;
    bf16_t *const srow = stage(nj >> 5) + (nj & 31) * BM;
#pragma unroll
    for (int i = 0; i < C::WM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = __builtin_amdgcn_exp2f((acc[i][j][4 * q + e] - u) * c);
          sum += p[e];
        }
        if (E) {  // 16-byte chunk index swizzled by the row: conflict-free here and in the row-wise reads below
          const int m = mlane + 32 * i + 8 * q;
          *reinterpret_cast<u32x2_t *>(srow + ((((m >> 3) ^ nj) & 31) << 3) + (m & 7)) =
              u32x2_t{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])};
        }
      }
    sum += __shfl_xor(sum, 32);
    if (lane < 32) s_sum[wm][nj] = sum;
  }
  __syncthreads();
  if (tid < C::BN && n0 + tid < n) {
    float top = s_max[0][tid], sum = s_sum[0][tid];
#pragma unroll
    for (int w = 1; w < C::WAVES_M; ++w) top = fmaxf(top, s_max[w][tid]), sum += s_sum[w][tid];
    const float r = rows.ref[rows.list[row0 + n0 + tid]];
    stat[(n0 + tid) * ntile + it.m] = make_float2((top - r) * c > kHeadRange ? top : r, sum);
  }
  if (!E) return;
  // E lies in blocks of 32 columns, [column / 32][row][32]: 16 rows of a block are 1 KB
  for (int at = tid; at < C::BN * 32; at += C::NT) {
    const int nj = (at >> 2) % C::BN, chunk = at / (4 * C::BN) * 4 + (at & 3);
    if (n0 + nj >= n || m0 + chunk * 8 >= lde) continue;
    *reinterpret_cast<u32x4_t *>(E + ((m0 / 32 + (chunk >> 2)) * te + n0 + nj) * 32 + (chunk & 3) * 8) =
        *reinterpret_cast<const u32x4_t *>(stage(nj >> 5) + (nj & 31) * BM + (((chunk ^ nj) & 31) << 3));
  }
}

// ---------------------------------------------------------------------- dX
// m: columns of X, n: counted rows of the block; reduction over the vocabulary (lde of it: E is zero past V).
template <class C>
__global__ __launch_bounds__(C::NT) void k_head_dx(HeadRows rows, int64_t row0, int64_t tb,
                                                   const bf16_t *__restrict__ E, int64_t lde, int64_t te,
                                                   const bf16_t *__restrict__ W, int64_t V, int64_t K,
                                                   const float *__restrict__ scale, float *__restrict__ part,
                                                   bf16_t *__restrict__ dX) {
  QLORA_RING(C, ring);
  const int64_t n = block_rows(rows, row0, tb);
  if (n <= 0) return;
  const int ranges = *rows.ranges;
  Item it;
  if (!item_of((K + BM - 1) / BM, (n + C::BN - 1) / C::BN, ranges, &it)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  const int64_t m0 = it.m * BM, n0 = it.n * C::BN;
  const int64_t steps = lde / BK, per = (steps + ranges - 1) / ranges;
  const int64_t s0 = it.range * per, s1 = s0 + per < steps ? s0 + per : steps;
  Tile<BM, C::NT, ACROSS> ta;
  Tile<C::BN, C::NT, BLOCKS> tbl;
  ta.init(W, K, m0, K, nullptr, wave, lane);
  tbl.init(E, te, n0, n, nullptr, wave, lane);
  f32x16_t acc[C::WM][C::WN];
  reduce_steps<C, ACROSS, BLOCKS>(ta, tbl, V, s0, s1, ring, wm, wn, lane, acc);
#pragma unroll
  for (int j = 0; j < C::WN; ++j) {
    const int64_t i = n0 + (wn * C::WN + j) * 32 + (lane & 31);
    if (i >= n) continue;
    const float f = ranges > 1 ? 1.f : scale[i];
    bf16_t *const out = dX + (int64_t)rows.list[row0 + i] * K;
    float *const psum = part + (it.range * n + i) * K;
#pragma unroll
    for (int mi = 0; mi < C::WM; ++mi)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t m = m0 + (wm * C::WM + mi) * 32 + 8 * q + 4 * (lane >> 5);
        if (m >= K) continue;  // K % 8 == 0: four columns are all in or all out
        const f32x16_t &v = acc[mi][j];
        if (ranges > 1)
          *reinterpret_cast<float4 *>(psum + m) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        else
          *reinterpret_cast<u32x2_t *>(out + m) =
              u32x2_t{pack_bf16x2(v[4 * q] * f, v[4 * q + 1] * f), pack_bf16x2(v[4 * q + 2] * f, v[4 * q + 3] * f)};
      }
  }
}

// ---------------------------------------------------------------------- dW
// m: columns of X, n: columns of the vocabulary; reduction over the block's counted rows.  With `sums` (several
// blocks) the binary32 sums are carried in it from block to block and rounded to dW after the last.
template <class C>
__global__ __launch_bounds__(C::NT) void k_head_dw(HeadRows rows, int64_t row0, int64_t tb,
                                                   const bf16_t *__restrict__ E, int64_t lde, int64_t te,
                                                   const bf16_t *__restrict__ Xs, int64_t V, int64_t K,
                                                   float *__restrict__ sums,
                                                   int first, int last, bf16_t *__restrict__ dW) {
  QLORA_RING(C, ring);
  const int64_t n = block_rows(rows, row0, tb) < 0 ? 0 : block_rows(rows, row0, tb);
  Item it;
  if (!item_of((K + BM - 1) / BM, (V + C::BN - 1) / C::BN, 1, &it)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  const int64_t m0 = it.m * BM, n0 = it.n * C::BN;
  Tile<BM, C::NT, ACROSS> ta;
  Tile<C::BN, C::NT, BLOCKS_ACROSS> tbl;
  ta.init(Xs, K, m0, K, nullptr, wave, lane);
  tbl.init(E, te, n0, lde, nullptr, wave, lane);
  f32x16_t acc[C::WM][C::WN];
  reduce_steps<C, ACROSS, BLOCKS_ACROSS>(ta, tbl, n, 0, (n + BK - 1) / BK, ring, wm, wn, lane, acc);
#pragma unroll
  for (int j = 0; j < C::WN; ++j) {
    const int64_t v = n0 + (wn * C::WN + j) * 32 + (lane & 31);
    if (v >= V) continue;
#pragma unroll
    for (int mi = 0; mi < C::WM; ++mi)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t m = m0 + (wm * C::WM + mi) * 32 + 8 * q + 4 * (lane >> 5);
        if (m >= K) continue;
        float4 o = make_float4(acc[mi][j][4 * q], acc[mi][j][4 * q + 1], acc[mi][j][4 * q + 2], acc[mi][j][4 * q + 3]);
        if (sums) {
          float4 *const p = reinterpret_cast<float4 *>(sums + v * K + m);
          if (!first) {
            const float4 was = *p;
            o = make_float4(o.x + was.x, o.y + was.y, o.z + was.z, o.w + was.w);
          }
          if (!last) {
            *p = o;
            continue;
          }
        }
        *reinterpret_cast<u32x2_t *>(dW + v * K + m) = u32x2_t{pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w)};
      }
  }
}

int64_t items8(int64_t items) { return (items + 7) / 8 * 8; }  // every XCD's run has the same length

}  // namespace

size_t head_part_floats(int64_t tb, int64_t K, int64_t lde) {
  const int bn = head_tile_rows(tb);
  size_t most = 0;
  for (int64_t n = tb;; n = (n - 1) / bn * bn) {  // the largest row count of each number of tiles
    const int s = head_dx_ranges(n, K, lde, bn);
    const size_t need = s > 1 ? (size_t)s * n * K : 0;
    most = need > most ? need : most;
    if (n <= bn) return most;
  }
}

#define QLORA_HEAD_TILES(rows_, CALL)   \
  switch (head_tile_rows(rows_)) {      \
    case 64: { CALL(H64); break; }      \
    case 128: { CALL(H128); break; }    \
    default: { CALL(H256); break; }     \
  }

hipError_t launch_head_logits(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *X, const bf16_t *Xt,
                              int64_t ldx, const bf16_t *W, int64_t V, int64_t K, float c, float2 *stat, int64_t ntile,
                              bf16_t *E, int64_t lde, int64_t te, hipStream_t s) {
#define QLORA_CALL(CFG)                                                                                         \
  const dim3 grid((unsigned)items8(ntile * ((tb + CFG::BN - 1) / CFG::BN)));                                    \
  if (Xt)                                                                                                       \
    launch(k_head_logits<CFG, BLOCKS>, grid, dim3(CFG::NT), 0, s, rows, row0, tb, Xt, ldx, W, V, K, c, stat, ntile, E, lde, \
           te);                                                                                                 \
  else                                                                                                          \
    launch(k_head_logits<CFG, LINES>, grid, dim3(CFG::NT), 0, s, rows, row0, tb, X, K, W, V, K, c, stat, ntile, E, lde, te)
  QLORA_HEAD_TILES(tb, QLORA_CALL)
#undef QLORA_CALL
  return hipGetLastError();
}

hipError_t launch_head_dx(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *E, int64_t lde, int64_t te,
                          const bf16_t *W, int64_t V, int64_t K, const float *scale, float *part, bf16_t *dX,
                          hipStream_t s) {
  const int bn = head_tile_rows(tb);
  int64_t most = 0;  // workgroups over all row counts of the block (the kernel takes as many as the count needs)
  for (int64_t t = 1; t <= (tb + bn - 1) / bn; ++t) {
    const int64_t items = t * ((K + BM - 1) / BM) * head_dx_ranges(t * bn, K, lde, bn);
    most = items > most ? items : most;
  }
#define QLORA_CALL(CFG)                                                                                              \
  launch(k_head_dx<CFG>, dim3((unsigned)items8(most)), dim3(CFG::NT), 0, s, rows, row0, tb, E, lde, te, W, V, K, scale, part, \
         dX)
  QLORA_HEAD_TILES(tb, QLORA_CALL)
#undef QLORA_CALL
  return hipGetLastError();
}

hipError_t launch_head_dw(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *E, int64_t lde, int64_t te,
                          const bf16_t *Xs, int64_t V, int64_t K, float *sums, bool first, bool last, bf16_t *dW,
                          hipStream_t s) {
  launch(k_head_dw<H256>, dim3((unsigned)items8(((K + BM - 1) / BM) * ((V + 255) / 256))), dim3(H256::NT), 0, s, rows,
         row0, tb, E, lde, te, Xs, V, K, sums, first ? 1 : 0, last ? 1 : 0, dW);
  return hipGetLastError();
}

}  // namespace qlora
