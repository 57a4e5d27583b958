// head_gemm.hip -- the three products of the output layer's losses on bf16 MFMAs:
//
//   logits   z = X W^T       per tile: softmax statistics, and E = exp2((z - u) c) in bf16 (never z itself)
//   dX       dX = f o (E W)  reduction over the vocabulary, f the rows' factors
//   dW       dW = (f o E)^T X  reduction over the rows, f split between E and X
//
// (E with its targets' entries put in by k_head_combine; see head_loss.hip for the mathematics.)
//
// One kernel body serves all three: C[n][m] = sum_r A(m, r) B(n, r), the operands read from global memory either
// along the reduction ("rows": [m][r]) or across it ("transposed": [r][m]).  A workgroup of 4 or 8 waves computes a
// 256 x 256, 256 x 128 or 128 x 64 tile (m x n) with v_mfma_f32_32x32x16_bf16; m is the MFMA's row index, so a lane holds
// four consecutive m of one n, which makes the softmax statistics of a row of X (n) a reduction inside the lane.  The
// reduction runs in 32-deep steps over a ring of four LDS tiles that the load unit fills directly (16 bytes per lane, see
// products).
//
// LDS tiles: "rows" [row][32] with the 16-byte chunk index XOR-swizzled by (row / 4) % 4, or in pairs of steps [row][64]
// by (row / 2) % 8; "transposed" [32][cols] with the 64-byte groups of a row XOR-swizzled by row % 4 (a transposing read
// takes four rows at once), all without bank conflicts; the direct copies write lane-consecutive LDS, so the swizzle is
// applied to the source address.
//
// Measured at 3686 counted rows x 128256 x 4096: logits 3051 us (1270 TFLOP/s with the softmax; a plain library product
// of the same data 1310), dX 3135 us (1235; 880); at 1843 x 32000 x 4096 dW 423 us (1141; 820).  Bound by the power that
// the MFMAs draw: under them the clock falls from 2.4 to about 1.6 GHz, of whose cycles the matrix units are busy in 0.73,
// and without its copies dX still takes 0.84 of its time.  Few rows are bound by the stream of W: 48 x 128256 x 4096 188
// us, 5.6 TB/s.
#include <type_traits>

#include "device.h"
#include "head.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int BK = 32;      // reduction depth of a step
constexpr int STAGES = 4;   // tiles in LDS: one being multiplied, three on their way

template <int WAVES_M_, int WAVES_N_, int WM_, int WN_>
struct HeadCfg {
  static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, WM = WM_, WN = WN_;
  static constexpr int NW = WAVES_M * WAVES_N, NT = 64 * NW;
  static constexpr int BM = WAVES_M * WM * 32, BN = WAVES_N * WN * 32;
  // 16-byte copies per thread of a step's tile of the n-side: the last ones of an item's last four steps, which its
  // epilogue need not wait for (the next item asks for them in its third step)
  static constexpr int LB = BN * BK / 8 / NT;
  // Few rows: the logit product is bound by the stream of W's rows, and workgroups that all begin at column 0 of theirs
  // ask for addresses a row's length apart, which for powers of two lie in few memory channels.  Each output tile begins
  // 128 columns after the one before it instead (16 x 32000 x 8192 in two ranges 124 -> 94 us; 128 x 128256 x 4096 221 ->
  // 211; a length that is no power of two: no change).  Wide tiles are bound by the MFMAs and share X's tiles in L2.
  static constexpr bool TURNS = BN < 256;
};
using H256 = HeadCfg<2, 4, 4, 2>;  // 128 x 64 per wave
using H128 = HeadCfg<4, 2, 2, 2>;  // 64 x 64 per wave
using H64 = HeadCfg<2, 2, 2, 1>;   // 128 x 64, 64 x 32 per wave, three workgroups per CU

__device__ __forceinline__ void fence_sched() { __builtin_amdgcn_sched_barrier(0); }

// The LDS tiles of one workgroup, by slot.  Each slot is an array of its own, so that the compiler can tell reads of
// one from the direct copies into another and adds no waits.  `a` and `b` are the m-side's and the n-side's tiles: the
// two halves of a slot's array (QLORA_RING), or, where the m-side's tiles are copied two steps at a time, arrays of
// their own of which slots 0 and 1, and 2 and 3, share one (QLORA_RING_PAIRS).
typedef __attribute__((address_space(3))) char lds_char;
struct Ring {
  lds_char *a[STAGES], *b[STAGES];
};
#define QLORA_RING(C, ring)                                                                                     \
  __shared__ __attribute__((aligned(1024))) char ring0[(C::BM + C::BN) * BK * 2], ring1[(C::BM + C::BN) * BK * 2],    \
      ring2[(C::BM + C::BN) * BK * 2], ring3[(C::BM + C::BN) * BK * 2];                                               \
  const Ring ring = {{(lds_char *)ring0, (lds_char *)ring1, (lds_char *)ring2, (lds_char *)ring3},              \
                     {(lds_char *)ring0 + C::BM * BK * 2, (lds_char *)ring1 + C::BM * BK * 2,                   \
                      (lds_char *)ring2 + C::BM * BK * 2, (lds_char *)ring3 + C::BM * BK * 2}}
#define QLORA_RING_PAIRS(C, ring)                                                                               \
  __shared__ __attribute__((aligned(1024))) char pair0[C::BM * BK * 4], pair1[C::BM * BK * 4], ring0[C::BN * BK * 2],  \
      ring1[C::BN * BK * 2], ring2[C::BN * BK * 2], ring3[C::BN * BK * 2];                                      \
  const Ring ring = {{(lds_char *)pair0, (lds_char *)pair0, (lds_char *)pair1, (lds_char *)pair1},              \
                     {(lds_char *)ring0, (lds_char *)ring1, (lds_char *)ring2, (lds_char *)ring3}}

// Lane offsets into the slots.  An LDS instruction adds at most 65535 to its address register, so where the arrays
// reach further a lane keeps its offset twice, plain and plus `kFar`, the constant then being array - kFar: all the
// reads of a tile share these registers.  The values are hidden from the compiler, which would otherwise keep a
// register for every sum.  (Which of the two is taken follows where the arrays come to lie: slots 0 and 1 of QLORA_RING
// and the pairs below 64 KB, the rest above.  A wrong guess would cost an addition, nothing else.)
constexpr int kFar = 65536;
enum { BY_SLOT, NEAR, FAR };
struct Lane {
  int near, far;
  __device__ __forceinline__ void set(int v) {
    near = v, far = v + kFar;
    asm("" : "+v"(near));
    asm("" : "+v"(far));
  }
};
template <int REACH>
__device__ __forceinline__ lds_char *in_slot(lds_char *base, int slot, const Lane &l, int more) {
  return REACH == NEAR || (REACH == BY_SLOT && slot < 2) ? base + l.near + more : base + l.far + (more - kFar);
}

// How an operand lies in memory (element (i, r): row or column i of the tile's side, reduction index r):
//  LINES:   row-major [i][r]; copied 64 reduction indices (whole 128-byte lines) and two steps at a time: in halves
//           every line is fetched twice (logits of 8192 rows 1308 against 1355 TFLOP/s, of 64 rows x 50257 x 1024 28
//           against 24 us).
//  BLOCKS:  32 reduction indices at a time, [r / 32][i][32]: a step's tile is one contiguous piece.
//  ACROSS:  row-major [r][i].
//  BLOCKS_ACROSS: [i / 32][r][32], what BLOCKS is seen from its other side.
enum { LINES, BLOCKS, ACROSS, BLOCKS_ACROSS };

// One operand's tile of ROWS rows (columns for the ACROSS ones).  `ld` is the row length of a row-major matrix, the
// number of rows in a block otherwise.  BLOCKS rows are gathered through `list` if there is one; rows past the last
// one repeat it.  Steps go to the next multiple of 128 reduction indices: indices past `red` repeat the last one (or
// the last eight), and the other operand holds zeros there in memory.  A step's addresses are a wave-uniform base
// plus 32-bit lane offsets.
template <int ROWS, int NT, int KIND>
struct Tile {
  static constexpr bool TR = KIND == ACROSS || KIND == BLOCKS_ACROSS;
  static constexpr bool PAIR = KIND == LINES;
  static constexpr int LD = ROWS * (PAIR ? 2 : 1) * BK / 8 / NT;  // 16-byte copies per thread and step (pair of steps)
  static constexpr int NW = NT / 64;
  static constexpr int CH = ROWS / 8;  // across: 16-byte chunks per LDS row, and LDS rows from copy to copy
  static constexpr int RSTEP = NW * 64 / CH;
  static_assert(ROWS * (PAIR ? 2 : 1) * BK / 8 % NT == 0 && LD >= 1, "unsupported tile");
  static_assert(!TR || (64 % CH == 0 && RSTEP % 4 == 0), "the copies of a thread share one swizzle");
  const char *base;
  uint32_t off[TR ? 1 : LD];  // across: of the column
  uint32_t k0;                // reduction index of the thread's first copy (rows: of all) within a step
  uint32_t ld;
  int red;

  // XOR of the 64-byte group index of LDS row r: rows r .. r + 3 then start in different quarters of the 64 banks
  static __device__ __forceinline__ int swz(int r) { return ROWS >= 128 ? (r & 3) : ((r >> 1) & 1); }

  __device__ __forceinline__ void init(const bf16_t *src, int64_t ld_, int64_t first, int64_t count, int64_t red_,
                                       const int32_t *list, int wave, int lane) {
    ld = (uint32_t)ld_, red = (int)red_;
    if constexpr (!TR) {
      // the rows of a thread's copies are equal modulo 16
      k0 = PAIR ? 8 * ((lane & 7) ^ (((8 * wave + (lane >> 3)) >> 1) & 7)) : 8 * ((lane & 3) ^ ((lane >> 4) & 3));
      const int64_t row = KIND == BLOCKS ? BK : ld;
      base = (const char *)(list ? src : src + first * row);
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int rr = PAIR ? 8 * (i * NW + wave) + (lane >> 3) : 16 * (i * NW + wave) + (lane >> 2);
        const int64_t at = first + rr < count ? rr : count - 1 - first;
        off[i] = (uint32_t)((list ? list[first + at] : at) * row * 2 + (KIND == BLOCKS ? k0 * 2 : 0));
      }
    } else {
      k0 = wave * (64 / CH) + lane / CH;
      int64_t c = first + 8 * ((lane % CH) ^ (swz(k0) << 2));
      if (c > count - 8) c = count - 8;  // count % 8 == 0
      if constexpr (KIND == ACROSS) {
        base = (const char *)src;
        off[0] = (uint32_t)(c * 2);
      } else {
        base = (const char *)(src + first / 32 * ld * 32);
        off[0] = (uint32_t)((c - first) / 32 * ld * 64 + c % 32 * 2);
      }
    }
  }
  // Copy i of this thread of the tile of step (or pair of steps) `s`.  (Buffer loads take the uniform part of the address
  // in scalar registers; the descriptor spans all of memory behind the base, every address is inside the operand by
  // construction.)
  __device__ __forceinline__ void copy(int s, int i, lds_char *to, int wave) const {
    const char *b = base;
    uint32_t o;
    if constexpr (KIND == LINES) {
      o = off[i] + 2 * min(k0 + s * (2 * BK), (uint32_t)red - 8);
    } else if constexpr (KIND == BLOCKS) {
      b += (int64_t)s * ld * (2 * BK);
      o = off[i];
    } else if constexpr (KIND == ACROSS) {  // ld * 2 < 2^24
      const int r0 = min(s * BK, max(red - BK, 0));
      b += (int64_t)r0 * ld * 2;
      o = off[0] + __umul24(min(k0 + (i * RSTEP + s * BK - r0), (uint32_t)(red - 1 - r0)), ld * 2);
    } else {
      o = off[0] + 64 * min(k0 + (i * RSTEP + s * BK), (uint32_t)red - 1);
    }
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)b, 0, -1, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void *)(to + (i * NW + wave) * 1024), 16, o, 0, 0, 0);
  }
};

// Reads of the MFMA operands of one side: N tiles of 32 rows (columns) from `first` of a ROWS-wide tile.
template <int ROWS, int N, int KIND, int REACH>
struct Operand {
  // rows: [row][32] or, in pairs of steps, [row][64], the 16-byte chunk swizzled (by row / 4 % 4, row / 2 % 8); the
  // quarters differ in a bit or two of the chunk.
  // across: [32][ROWS]: in each 16-lane group, lane i of a transposing read gets element (i & 3) of the 8 bytes
  // addressed by lane 4 m + (i >> 2), so lane a points at row base + (a >> 2), columns 4 (a & 3) .. + 3, and the reads
  // of rows + 0..3 and + 4..7 give its 8 reduction values; the 64-byte group of tile i is swizzled, so each needs its
  // own offset.
  static constexpr bool TR = KIND == ACROSS || KIND == BLOCKS_ACROSS, PAIR = KIND == LINES;
  static constexpr int NO = TR ? N : PAIR ? 4 : 2;
  Lane at[NO];
  __device__ __forceinline__ void init(int base, int first, int lane) {
    if constexpr (!TR) {
      const int r = lane & 31, chunk = (lane >> 5) ^ (PAIR ? (r >> 1) & 7 : (r >> 2) & 3);
#pragma unroll
      for (int q = 0; q < NO; ++q) at[q].set(base + (first + r) * (PAIR ? 128 : 64) + (chunk ^ (2 * q)) * 16);
    } else {
      const int grp = lane >> 4, ai = lane & 15;
      const int r = 8 * (grp >> 1) + (ai >> 2);
      const int swz = ROWS >= 128 ? (r & 3) : ((r >> 1) & 1);
#pragma unroll
      for (int i = 0; i < N; ++i)
        at[i].set(base + (r * ROWS + ((first + 32 * i) ^ (swz << 5)) + 16 * (grp & 1) + 4 * (ai & 3)) * 2);
    }
  }
  // tile i, reduction indices 16 kk .. 16 kk + 15 of the step in `slot`
  __device__ __forceinline__ u32x4_t read(lds_char *const (&side)[STAGES], int slot, int kk, int i) const {
    if constexpr (!TR) {
      const int q = PAIR ? 2 * (slot & 1) + kk : kk;
      return *(const __attribute__((address_space(3))) u32x4_t *)in_slot<REACH>(side[slot], slot, at[q],
                                                                               i * 32 * (PAIR ? 128 : 64));
    } else {
      typedef short s4_t __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s4_t lds_s4;
      const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s4 *)in_slot<REACH>(side[slot], slot, at[i], kk * 32 * ROWS));
      const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s4 *)in_slot<REACH>(side[slot], slot, at[i], kk * 32 * ROWS + 8 * ROWS));
      const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
      return u32x4_t{l2.x, l2.y, h2.x, h2.y};
    }
  }
};

template <class C>
using Acc = f32x16_t[C::WM][C::WN];

// Meet the workgroup's other waves once this one's LDS operations are done, without the full memory fence of
// __syncthreads, which would wait for every copy in flight.
// s_waitcnt fields: vmcnt[3:0] and [15:14], expcnt[6:4] (7 = no wait), lgkmcnt[11:8].
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// All but this wave's last VM copies have landed (called before an epilogue's stores are issued, so that only copies
// are waited for).
template <int VM = 0>
__device__ __forceinline__ void arrive() {
  static_assert(VM < 16, "the low four bits");
  __builtin_amdgcn_s_waitcnt(0x0f70 | VM);
  asm volatile("" ::: "memory");
}

// Output tiles ("items") are numbered so that each XCD (workgroups go round the 8 XCDs) takes a run of consecutive
// ones, and consecutive ones are blocks of 4 m-tiles x all n-tiles: the 32 workgroups of an XCD then share 4 + 8
// operand tiles.  A workgroup takes the items lin, lin + stride, ...
struct Items {
  int tiles_m, tiles_n, ranges;
  int m, n, range;
  __device__ __forceinline__ bool take(uint32_t lin) {
    const uint32_t total = (uint32_t)tiles_m * tiles_n * ranges, per = (total + 7) / 8, id = (lin & 7) * per + (lin >> 3);
    if ((lin >> 3) >= per || id >= total) return false;
    const uint32_t plane = (uint32_t)tiles_m * tiles_n, in = id % plane;
    const uint32_t band = in / (4u * tiles_n), left = in - band * 4u * tiles_n;
    const uint32_t wide = min(tiles_m - band * 4, 4u);
    range = id / plane;
    m = band * 4 + left % wide;
    n = left / wide;
    return true;
  }
};

// A kernel whose rows do not fill whole 256-row tiles gives the last of them to narrower tiles, in a second pass over
// items.  The workgroups that had one item less in the first pass take them, where that is at most two each (a narrow item
// takes 0.6 of the time of a wide one), else all of them.
struct Turn {
  uint32_t lin, stride;
};
__device__ __forceinline__ Turn second_pass(const Items &first, uint32_t more) {
  const uint32_t total = (uint32_t)first.tiles_m * first.tiles_n * first.ranges, per = (total + 7) / 8;
  const uint32_t groups = gridDim.x / 8, at = blockIdx.x >> 3, busy = per % groups, free = groups - busy;
  if ((more + 7) / 8 > 2 * free) return Turn{(at + free) % groups * 8 + (blockIdx.x & 7), gridDim.x};
  return Turn{at < busy ? 0x7ffffff8u : (at - busy) * 8 + (blockIdx.x & 7), free * 8};  // (out of range: none)
}
__device__ __forceinline__ void between_passes() {
  arrive();
  meet();
}

// A workgroup's loop over its items, each a reduction over steps [s0, s1) of both operands' tiles, a multiple of four.
//
// Step s multiplies the tiles of slot s % 4 while the copies of steps s + 1 .. s + 3 are in flight.  Its first MFMAs'
// operands are in registers; the second half's are read under them; then the waves meet (every wave holds the last
// operands of slot s, and step s + 1 has landed), read the first operands of step s + 1 and run the second half's
// MFMAs.  The copies of step s + 4 into the slot just left are issued one at a time between those: issued together they
// would hold the waves up for as long as the load unit takes to accept them.  (Timed without them, without the LDS reads
// and without the MFMAs, the copies alone take 0.7 of the whole time and the MFMAs 0.6, so each copy gets as much time
// as the ring allows: more than two steps.)  The last four steps of an item copy the first four of the next one, so the
// ring never drains and an item's epilogue hides the first latency of the next.
//
//  setup(ta, tb, s0, s1): the tiles and steps of the item just taken; returns the step to begin with (TURNS: s0 + 4 i,
//  after the last step come those before it; else s0)
//  begin(): notes for its epilogue    late(): before its last four steps (loads that the epilogue needs at once)
//  finish(acc): its epilogue; calls arrive<LB>() before its first store
template <class C, int KA, int KB, class Setup, class Begin, class Late, class Finish>
__device__ __forceinline__ void products(Items &items, Turn turn, const Ring &ring, int wave, int lane, Setup setup,
                                         Begin begin, Late late, Finish finish) {
  typedef Tile<C::BM, C::NT, KA> TileA;
  typedef Tile<C::BN, C::NT, KB> TileB;
  constexpr bool PAIR = TileA::PAIR;
  constexpr int LA = TileA::LD, LB = TileB::LD;
  // copies that may be in flight when the waves meet in an even and in an odd step: those of the steps after the next
  // (in pairs: of the n-side, and, in an even step, the m-side's next pair)
  constexpr int EVEN = PAIR ? 2 * LB + LA : 2 * (LA + LB), ODD = PAIR ? 2 * LB : EVEN;
  static_assert(EVEN < 16, "counted in four bits");
  uint32_t lin = turn.lin;
  if (!items.take(lin)) return;
  TileA ta;
  TileB tb;
  int s0, s1, begin_at = setup(ta, tb, &s0, &s1);
  Operand<C::BM, C::WM, KA, PAIR ? NEAR : BY_SLOT> oa;
  Operand<C::BN, C::WN, KB, PAIR ? FAR : BY_SLOT> ob;
  oa.init(0, wave / C::WAVES_N * C::WM * 32, lane);
  ob.init(0, wave % C::WAVES_N * C::WN * 32, lane);
  // copies [q0, q1) of those that go with step s into `slot`: of both sides; in pairs, of the m-side with odd steps
  // only, both steps' together and first
  auto count = [](int slot) { return PAIR && !(slot & 1) ? LB : LA + LB; };
  auto copies = [&](int s, int slot, int q0, int q1) {
#pragma unroll
    for (int q = q0; q < q1; ++q) {
      if (PAIR && !(slot & 1))
        tb.copy(s, q, ring.b[slot], wave);
      else if (q < LA)
        ta.copy(PAIR ? s >> 1 : s, q, ring.a[slot], wave);
      else
        tb.copy(s, q - LA, ring.b[slot], wave);
      fence_sched();
    }
  };
#pragma unroll
  for (int q = 0; q < STAGES; ++q) copies((C::TURNS ? begin_at : s0) + q, q, 0, count(q));
  arrive();
  for (;;) {
    begin();
    f32x16_t acc[C::WM][C::WN];
#pragma unroll
    for (int i = 0; i < C::WM; ++i)
#pragma unroll
      for (int j = 0; j < C::WN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    u32x4_t a[2][C::WM], b[2][C::WN];
    auto read = [&](int slot, int kk) {
#pragma unroll
      for (int i = 0; i < C::WM; ++i) a[kk][i] = oa.read(ring.a, slot, kk, i);
#pragma unroll
      for (int j = 0; j < C::WN; ++j) b[kk][j] = ob.read(ring.b, slot, kk, j);
      fence_sched();
    };
    // the MFMAs of half kk, the copies of step s into `slot` (none: -1) spread among them
    auto mma = [&](int kk, int s, int slot) {
#pragma unroll
      for (int i = 0; i < C::WM; ++i) {
#pragma unroll
        for (int j = 0; j < C::WN; ++j) acc[i][j] = mfma_32x32x16(a[kk][i], b[kk][j], acc[i][j]);
        fence_sched();
        if (slot >= 0) copies(s, slot, count(slot) * i / C::WM, count(slot) * (i + 1) / C::WM);
      }
    };
    // the step in slot P; `s` is the one to copy, `fresh`: the item's first two steps, whose successors are known to
    // have landed (arrive()) while the last epilogue's stores may still be on their way
    auto step = [&](auto pc, int s, bool fresh) {
      constexpr int P = decltype(pc)::value, NEXT = (P + 1) % STAGES;
      read(P, 1);
      mma(0, 0, -1);
      if (!(P < 2 && fresh)) __builtin_amdgcn_s_waitcnt(0x0f70 | (P & 1 ? ODD : EVEN));
      meet();
      read(NEXT, 0);
      mma(1, s, P);
    };
    meet();
    read(0, 0);
    int s = s0;
    for (; s + 4 < s1; s += 4) {
      if constexpr (C::TURNS) begin_at = begin_at + 4 == s1 ? s0 : begin_at + 4;
      const int next = C::TURNS ? begin_at : s + 4;
      step(std::integral_constant<int, 0>(), next, s == s0);
      step(std::integral_constant<int, 1>(), next + 1, s == s0);
      step(std::integral_constant<int, 2>(), next + 2, false);
      step(std::integral_constant<int, 3>(), next + 3, false);
    }
    late();
    lin += turn.stride;
    const bool more = items.take(lin), fresh = s == s0;
    if (more) begin_at = setup(ta, tb, &s0, &s1);  // (else four steps of this item are copied once more)
    const int next = C::TURNS ? begin_at : s0;
    step(std::integral_constant<int, 0>(), next, fresh);
    step(std::integral_constant<int, 1>(), next + 1, fresh);
    step(std::integral_constant<int, 2>(), next + 2, false);
    step(std::integral_constant<int, 3>(), next + 3, false);
    finish(acc);
    if (!more) {
      arrive();  // nothing is left on its way into LDS
      return;
    }
  }
}

// Two lanes of a wave, l and l + 32, hold columns 0..3 and 4..7 of two groups of eight (lo and hi, packed bf16).
// Afterwards l holds all eight of the first group, l + 32 of the second: 16 bytes to store each.
__device__ __forceinline__ u32x4_t join_halves(const u32x2_t &lo, const u32x2_t &hi) {
  const auto x = __builtin_amdgcn_permlane32_swap(lo.x, hi.x, false, false);
  const auto y = __builtin_amdgcn_permlane32_swap(lo.y, hi.y, false, false);
  return u32x4_t{x[0], y[0], x[1], y[1]};
}

// Pieces a and b (16 bytes a lane, rows lane % 32, halves lane / 32) of adjacent columns.  Afterwards a holds rows 0..15
// of both and b rows 16..31: lanes 0..15 and 32..47 the halves of what was a's columns, the others of b's, so a store
// covers 64 contiguous bytes of a row, not 32 (dW of 622 x 50257 x 1024 81 -> 78 us, of 7 x 6463 x 5992 28 -> 25; no
// change where stores are few).
__device__ __forceinline__ void join_rows(u32x4_t &a, u32x4_t &b) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t aw = a[w], bw = b[w];
    const auto x = __builtin_amdgcn_permlane16_swap(aw, bw, false, false);
    a[w] = x[0], b[w] = x[1];
  }
}
// Column of a lane's piece afterwards: halves are `half` columns long, b's columns `next` after a's.
__device__ __forceinline__ int store_column(int lane, int half, int next) {
  return (lane >> 5) * half + (lane >> 4 & 1) * next;
}
// Four binary32 values of an MFMA result as 16 bytes.
__device__ __forceinline__ u32x4_t four(const f32x16_t &v, int q) {
  return u32x4_t{__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                 __float_as_uint(v[4 * q + 3])};
}

__device__ __forceinline__ int block_rows(const HeadRows &rows, int64_t row0, int64_t tb) {
  const int64_t n = *rows.n - row0;
  return n < 0 ? 0 : (int)(n < tb ? n : tb);
}

// ------------------------------------------------------------------ logits
// m: columns of the vocabulary, n: counted rows of the block.
// X as k_head_prep lays it out (ldx rows per block).
struct LogitArgs {
  HeadRows rows;
  int64_t row0, tb;
  const bf16_t *X;
  int64_t ldx;
  const bf16_t *W;
  int64_t V, K;
  float c;
  float2 *stat;
  int64_t ntile;  // entries per row
  int tiles;      // of the vocabulary
  int ranges;     // of the reduction; with more than one its binary32 sums go to part[range][row][lde]
  float *part;
  bf16_t *E;
  int64_t lde, te;
  int k;
};

// Rows [first, n) of the block.
template <class C, bool SPLIT>
__device__ __forceinline__ void logit_items(const LogitArgs &g, int first, int n, Items &items, Turn turn,
                                            const Ring &ring) {
  const HeadRows &rows = g.rows;
  const int64_t row0 = g.row0, V = g.V, K = g.K, ntile = g.ntile, te = g.te;
  const float c = g.c;
  const int k = g.k;
  bf16_t *const E = g.E;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  int m0 = 0, n0 = 0;
  auto setup = [&](Tile<C::BM, C::NT, LINES> &ta, Tile<C::BN, C::NT, BLOCKS> &tbl, int *s0, int *s1) {
    ta.init(g.W, K, (int64_t)items.m * C::BM, V, K, nullptr, wave, lane);
    tbl.init(g.X, g.ldx, first + (int64_t)items.n * C::BN, n, K, rows.list + row0, wave, lane);
    const int fours = (int)((K + 127) / 128), per = SPLIT ? (fours + g.ranges - 1) / g.ranges : fours;
    *s0 = SPLIT ? items.range * per * 4 : 0;
    *s1 = SPLIT ? min(*s0 + per * 4, fours * 4) : fours * 4;
    return C::TURNS ? *s0 + items.m * 4 % (*s1 - *s0) : *s0;
  };
  // The epilogue's first loads are issued before the reduction: the lane's rows in X, and the item's targets (one per
  // lane, the first 64 of them).
  int32_t t[C::WN];
  int t0 = 0, t1 = 0, range = 0, row_of = 0;  // row_of: the item's first row in the row tile of its targets
  uint32_t target = 0;
  const uint32_t *targets = nullptr;
  auto begin = [&]() {
    m0 = items.m * C::BM, n0 = first + items.n * C::BN, range = items.range;
#pragma unroll
    for (int j = 0; j < C::WN; ++j) {
      const int row = n0 + (wn * C::WN + j) * 32 + (lane & 31);
      t[j] = rows.list[row0 + (row < n ? row : n - 1)];
    }
    if (rows.target) {
      const int row_tile = n0 / rows.tile_rows;
      row_of = n0 - row_tile * rows.tile_rows;
      const int32_t *const b = rows.bucket + (int64_t)row_tile * (g.tiles + 1) + items.m;
      t0 = b[0], t1 = b[1];
      targets = rows.target + (int64_t)row_tile * rows.tile_rows * k;
      if (t0 + lane < t1) target = targets[t0 + lane];
    }
  };
  // Logits of the tile's targets, for the loss and the targets' gradient: each wave picks its own out of acc.
  auto pick = [&](Acc<C> &acc) {
    for (int at = t0; at < t1; at += 64) {
      const bool in = at + lane < t1;
      if (at != t0 && in) target = targets[at + lane];
      const int nj = (int)(target >> 16) - row_of, m = target >> 8 & 255;
      uint64_t mine = __ballot(in && nj >= 0 && nj / (C::WN * 32) == wn && m / (C::WM * 32) == wm);
      while (mine) {
        const uint32_t one = __builtin_amdgcn_readlane(target, __builtin_ctzll(mine));
        mine &= mine - 1;
        const int un = (int)(one >> 16) - row_of, um = one >> 8 & 255;
        const int i1 = um / 32 % C::WM, j1 = un / 32 % C::WN, e1 = (um >> 3 & 3) * 4 + (um & 3);
        float z = 0.f;
        int32_t row = 0;
#pragma unroll
        for (int j = 0; j < C::WN; ++j) {
          row = j == j1 ? t[j] : row;
#pragma unroll
          for (int i = 0; i < C::WM; ++i)
            if (i == i1 && j == j1) z = acc[i][j][e1];
        }
        if (lane == (un & 31) + 32 * (um >> 2 & 1)) rows.zt[(int64_t)row * k + (one & 255)] = z;
      }
    }
  };
  float ref[C::WN];
  int rcol[C::WN];
  auto late = [&]() {
#pragma unroll
    for (int j = 0; j < C::WN; ++j) {
      ref[j] = rows.ref[t[j]];
      rcol[j] = rows.refcol[t[j]];
    }
  };
  // element e of acc[i][j]: column m0 + mlane + 32 i + 8 (e / 4) + e % 4 of the lane's row j
  const int mlane = wm * C::WM * 32 + 4 * (lane >> 5);
  auto finish = [&](Acc<C> &acc) {
    if constexpr (SPLIT) {  // k_head_soft does the rest
      arrive<C::LB>();
#pragma unroll
      for (int j = 0; j < C::WN; ++j) {
        const int row = n0 + (wn * C::WN + j) * 32 + (lane & 15), m = m0 + wm * C::WM * 32 + store_column(lane, 4, 8);
        float *const out = g.part + ((int64_t)range * n + row) * g.lde + m;
#pragma unroll
        for (int i = 0; i < C::WM; ++i)
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            u32x4_t lo = four(acc[i][j], q), hi = four(acc[i][j], q + 1);
            join_rows(lo, hi);
            const int at = 32 * i + 8 * q;
            if (m + at < g.lde && row < n) *reinterpret_cast<u32x4_t *>(out + at) = lo;
            if (m + at < g.lde && row + 16 < n) *reinterpret_cast<u32x4_t *>(out + 16 * g.lde + at) = hi;
          }
      }
      return;
    }
    if (rows.target) pick(acc);
#pragma unroll
    for (int j = 0; j < C::WN; ++j) {
      // the reference's own column and those past the vocabulary stay out of the sums
      int rc = rcol[j] - m0 - mlane, end = (int)(V - m0) - mlane;
      if (__any((rc >= -4 && rc < C::BM) || m0 + C::BM > V)) {
        asm("" : "+v"(rc), "+v"(end));
#pragma unroll
        for (int i = 0; i < C::WM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int m = 32 * i + 8 * (e >> 2) + (e & 3);
            acc[i][j][e] = ((m == rc) | (m >= end)) ? -INFINITY : acc[i][j][e];
          }
      }
    }
#pragma unroll
    for (int j = 0; j < C::WN; ++j) {
      // Against the reference (one FMA and one exp2 per logit); where that is out of range, against the largest logit
      // of the wave's columns.  The statistics are per wave: nothing is exchanged.
      float u = ref[j], sum = 0.f;
      const float uc = u * c;
      u32x2_t x[C::WM][4];
#pragma unroll
      for (int i = 0; i < C::WM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(acc[i][j][4 * q + e], c, -uc));
            sum += p[e];
          }
          x[i][q] = u32x2_t{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])};
        }
      sum += __shfl_xor(sum, 32);
      const bool over = !(sum < kHeadRange);
      if (__any(over)) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < C::WM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
        top = fmaxf(top, __shfl_xor(top, 32));
        u = over ? top : u;
        sum = 0.f;
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
            x[i][q] = u32x2_t{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])};
          }
        sum += __shfl_xor(sum, 32);
      }
      if (j == 0) arrive<C::LB>();
      const int row = n0 + (wn * C::WN + j) * 32 + (lane & 31);
      if (row < n && lane < 32 && m0 + wm * C::WM * 32 < V)
        g.stat[(int64_t)row * ntile + m0 / (C::WM * 32) + wm] = make_float2(u, sum);
      if (!E) continue;
      // E lies in blocks of 32 columns, [column / 32][row][32]: a wave's store is 16 whole rows of a block, 1 KB
      const int first_row = n0 + (wn * C::WN + j) * 32 + (lane & 15);
#pragma unroll
      for (int i = 0; i < C::WM; ++i) {
        bf16_t *const out = E + ((m0 / 32 + wm * C::WM + i) * te + first_row) * 32 + store_column(lane, 8, 16);
        u32x4_t lo = join_halves(x[i][0], x[i][1]), hi = join_halves(x[i][2], x[i][3]);
        join_rows(lo, hi);
        const bool in = m0 + (wm * C::WM + i) * 32 < g.lde;
        if (in && first_row < n) *reinterpret_cast<u32x4_t *>(out) = lo;
        if (in && first_row + 16 < n) *reinterpret_cast<u32x4_t *>(out + 16 * 32) = hi;
      }
    }
  };
  products<C, LINES, BLOCKS>(items, turn, ring, wave, lane, setup, begin, late, finish);
}

template <class C, bool SPLIT>
__global__ __launch_bounds__(C::NT) void k_head_logits(LogitArgs g) {
  const int n = block_rows(g.rows, g.row0, g.tb);
  if (n == 0) return;
  const int whole = C::BN == 256 ? g.rows.ranges[3] : n;
  Items items = {g.tiles, (whole + C::BN - 1) / C::BN, SPLIT ? g.ranges : 1};
  const Turn all = {blockIdx.x, gridDim.x};
  QLORA_RING_PAIRS(C, ring);
  if (whole > 0) logit_items<C, SPLIT>(g, 0, whole, items, all, ring);
  if constexpr (C::BN == 256) {
    if (whole == n) return;
    const int narrow = (n - whole + H128::BN - 1) / H128::BN;
    const Turn turn = second_pass(items, (uint32_t)(g.tiles * narrow));
    between_passes();
    items = {g.tiles, narrow, 1};
    logit_items<H128, false>(g, whole, n, items, turn, ring);
  }
}

// ---------------------------------------------------------------------- dX
// m: columns of X, n: counted rows of the block; reduction over the vocabulary (lde of it: E is zero past V).
struct DxArgs {
  HeadRows rows;
  int64_t row0, tb;
  const bf16_t *E;
  int64_t lde, te;
  const bf16_t *W;
  int64_t V, K;
  const float4 *scale;
  float *part;
  bf16_t *dX;
};

// Rows [first, n) of the block in `ranges` ranges; with more than one their sums go to part[range][row - first][K].
template <class C>
__device__ __forceinline__ void dx_items(const DxArgs &g, int first, int n, int ranges, float *part, Items &items,
                                         Turn turn, const Ring &ring) {
  const HeadRows &rows = g.rows;
  const int64_t row0 = g.row0, K = g.K;
  const float4 *const scale = g.scale;
  bf16_t *const dX = g.dX;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  int m0 = 0, n0 = 0, range = 0;
  auto setup = [&](Tile<C::BM, C::NT, ACROSS> &ta, Tile<C::BN, C::NT, BLOCKS> &tbl, int *s0, int *s1) {
    ta.init(g.W, K, (int64_t)items.m * C::BM, K, g.V, nullptr, wave, lane);
    tbl.init(g.E, g.te, first + (int64_t)items.n * C::BN, n, g.lde, nullptr, wave, lane);
    const int fours = (int)(g.lde / 128), per = (fours + ranges - 1) / ranges;
    *s0 = items.range * per * 4;
    *s1 = min(*s0 + per * 4, fours * 4);
    return *s0;
  };
  auto begin = [&]() { m0 = items.m * C::BM, n0 = first + items.n * C::BN, range = items.range; };
  auto late = []() {};
  auto finish = [&](Acc<C> &acc) {
    arrive<C::LB>();
#pragma unroll
    for (int j = 0; j < C::WN; ++j) {
      const int base = n0 + (wn * C::WN + j) * 32;
      const int i = min(base + (lane & 31), n - 1);     // the lane's row of the sums
      const int lo_row = base + (lane & 15), hi_row = lo_row + 16;  // and those that it stores
      const float4 f = scale[i];
      const bf16_t *const w = g.W + rows.refcol[rows.list[row0 + i]] * K + 4 * (lane >> 5);
      const int64_t lo_t = rows.list[row0 + min(lo_row, n - 1)], hi_t = rows.list[row0 + min(hi_row, n - 1)];
#pragma unroll
      for (int mi = 0; mi < C::WM; ++mi) {
        const int64_t m = m0 + (wm * C::WM + mi) * 32;
        const f32x16_t &v = acc[mi][j];
        if (ranges > 1) {
          const int64_t row = (int64_t)range * (n - first) + (lo_row - first);
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            u32x4_t lo = four(v, q), hi = four(v, q + 1);
            join_rows(lo, hi);
            const int64_t mq = m + 8 * q + store_column(lane, 4, 8);
            // K % 8 == 0: eight columns are all in or all out
            if (mq < K && lo_row < n) *reinterpret_cast<u32x4_t *>(part + row * K + mq) = lo;
            if (mq < K && hi_row < n) *reinterpret_cast<u32x4_t *>(part + (row + 16) * K + mq) = hi;
          }
        } else {
          u32x2_t x[4];  // with the first target's remainder times its row of W
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x2_t wv = m + 8 * q < K ? *reinterpret_cast<const u32x2_t *>(w + m + 8 * q) : u32x2_t{0u, 0u};
            x[q] = u32x2_t{pack_bf16x2(fmaf(f.y, bf16_lo_to_f32(wv.x), v[4 * q]) * f.x,
                                       fmaf(f.y, bf16_hi_to_f32(wv.x), v[4 * q + 1]) * f.x),
                           pack_bf16x2(fmaf(f.y, bf16_lo_to_f32(wv.y), v[4 * q + 2]) * f.x,
                                       fmaf(f.y, bf16_hi_to_f32(wv.y), v[4 * q + 3]) * f.x)};
          }
          u32x4_t lo = join_halves(x[0], x[1]), hi = join_halves(x[2], x[3]);
          join_rows(lo, hi);
          const int64_t mq = m + store_column(lane, 8, 16);
          if (mq < K && lo_row < n) *reinterpret_cast<u32x4_t *>(dX + lo_t * K + mq) = lo;
          if (mq < K && hi_row < n) *reinterpret_cast<u32x4_t *>(dX + hi_t * K + mq) = hi;
        }
      }
    }
  };
  products<C, ACROSS, BLOCKS>(items, turn, ring, wave, lane, setup, begin, late, finish);
}

template <class C>
__global__ __launch_bounds__(C::NT) void k_head_dx(DxArgs g) {
  QLORA_RING(C, ring);
  const int n = block_rows(g.rows, g.row0, g.tb);
  if (n == 0) return;
  const int tiles_m = (int)((g.K + C::BM - 1) / C::BM), ranges = g.rows.ranges[0], whole = g.rows.ranges[2];
  Items items = {tiles_m, (whole + C::BN - 1) / C::BN, ranges};
  if (whole > 0) dx_items<C>(g, 0, whole, ranges, g.part, items, Turn{blockIdx.x, gridDim.x}, ring);
  if constexpr (C::BN == 256) {
    if (whole == n) return;
    const int narrow = (n - whole + H128::BN - 1) / H128::BN, more = g.rows.ranges[1];
    const Turn turn = second_pass(items, (uint32_t)(tiles_m * narrow * more));
    between_passes();
    items = {tiles_m, narrow, more};
    dx_items<H128>(g, whole, n, more, g.part + head_first_sums(whole, ranges, g.K), items, turn, ring);
  }
}

// ---------------------------------------------------------------------- dW
// m: columns of X, n: columns of the vocabulary; reduction over the block's counted rows.  With `sums` (several
// blocks) the binary32 sums are carried in it from block to block and rounded to dW after the last; or, with several
// `ranges` of one block's rows, each range's are left in it ([range][V][K], neither the last) for k_head_dw_reduce.
struct DwArgs {
  HeadRows rows;
  int64_t row0, tb;
  const bf16_t *E;
  int64_t lde, te;
  const bf16_t *Xs;
  int64_t V, K;
  float *sums;
  int first, last, ranges;
  bf16_t *dW;
};

// Columns [begin_v, end_v) of the vocabulary.
template <class C>
__device__ __forceinline__ void dw_items(const DwArgs &g, int begin_v, int end_v, Items &items, Turn turn,
                                         const Ring &ring) {
  const int64_t K = g.K;
  float *sums = g.sums;
  bf16_t *const dW = g.dW;
  const int n = block_rows(g.rows, g.row0, g.tb);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  int m0 = 0, n0 = 0;
  // (no rows: four steps over the zeros that k_head_combine leaves behind the block's last row)
  auto setup = [&](Tile<C::BM, C::NT, ACROSS> &ta, Tile<C::BN, C::NT, BLOCKS_ACROSS> &tbl, int *s0, int *s1) {
    const int deep = max((n + 127) / 128, 1);
    ta.init(g.Xs, K, (int64_t)items.m * C::BM, K, deep * 128, nullptr, wave, lane);
    tbl.init(g.E, g.te, begin_v + (int64_t)items.n * C::BN, g.lde, max(n, 1), nullptr, wave, lane);
    const int per = head_dw_steps(n, items.ranges);
    *s0 = items.range * per * 4;
    *s1 = min(*s0 + per * 4, deep * 4);
    return *s0;
  };
  auto begin = [&]() {
    m0 = items.m * C::BM, n0 = begin_v + items.n * C::BN;
    if (sums) sums = g.sums + items.range * g.V * K;
  };
  auto late = []() {};
  auto finish = [&](Acc<C> &acc) {
    arrive<C::LB>();
#pragma unroll
    for (int j = 0; j < C::WN; ++j) {
      const int64_t v = n0 + (wn * C::WN + j) * 32 + (lane & 15);
#pragma unroll
      for (int mi = 0; mi < C::WM; ++mi) {
        const int64_t m = m0 + (wm * C::WM + mi) * 32;
        f32x16_t &o = acc[mi][j];
        if (sums) {
          const int64_t at = n0 + (wn * C::WN + j) * 32 + (lane & 31);  // the lane's row of the sums
          if (!g.first)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int64_t mq = m + 8 * q + 4 * (lane >> 5);
              if (at >= end_v || mq >= K) continue;
              const float4 was = *reinterpret_cast<const float4 *>(sums + at * K + mq);
              o[4 * q] += was.x, o[4 * q + 1] += was.y, o[4 * q + 2] += was.z, o[4 * q + 3] += was.w;
            }
          if (!g.last) {
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
              u32x4_t lo = four(o, q), hi = four(o, q + 1);
              join_rows(lo, hi);
              const int64_t mq = m + 8 * q + store_column(lane, 4, 8);
              if (mq < K && v < end_v) *reinterpret_cast<u32x4_t *>(sums + v * K + mq) = lo;
              if (mq < K && v + 16 < end_v) *reinterpret_cast<u32x4_t *>(sums + (v + 16) * K + mq) = hi;
            }
            continue;
          }
        }
        u32x4_t lo = join_halves(u32x2_t{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])},
                                 u32x2_t{pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])});
        u32x4_t hi = join_halves(u32x2_t{pack_bf16x2(o[8], o[9]), pack_bf16x2(o[10], o[11])},
                                 u32x2_t{pack_bf16x2(o[12], o[13]), pack_bf16x2(o[14], o[15])});
        join_rows(lo, hi);
        const int64_t mq = m + store_column(lane, 8, 16);
        if (mq < K && v < end_v) *reinterpret_cast<u32x4_t *>(dW + v * K + mq) = lo;
        if (mq < K && v + 16 < end_v) *reinterpret_cast<u32x4_t *>(dW + (v + 16) * K + mq) = hi;
      }
    }
  };
  products<C, ACROSS, BLOCKS_ACROSS>(items, turn, ring, wave, lane, setup, begin, late, finish);
}

__global__ __launch_bounds__(H256::NT) void k_head_dw(DwArgs g) {
  QLORA_RING(H256, ring);
  const int tiles_m = (int)((g.K + 255) / 256), whole = head_whole_columns(g.V, tiles_m);
  Items items = {tiles_m, (whole + 255) / 256, 1};
  if (whole > 0) dw_items<H256>(g, 0, whole, items, Turn{blockIdx.x, gridDim.x}, ring);
  if (whole == g.V) return;
  const int narrow = ((int)g.V - whole + H128::BN - 1) / H128::BN;
  // (several ranges: the columns all go to narrow tiles)
  const int n = block_rows(g.rows, g.row0, g.tb), per = head_dw_steps(n, g.ranges);
  const Items second = {tiles_m, narrow, (max((n + 127) / 128, 1) + per - 1) / per};
  const Turn turn = second_pass(items, (uint32_t)(tiles_m * narrow * second.ranges));
  between_passes();
  items = second;
  dw_items<H128>(g, whole, (int)g.V, items, turn, ring);
}

// Few rows (T <= 64): bound by dW's stores, which three workgroups a CU overlap with each other's steps (7 x 6463 x 5992
// 25 us, 3.1 TB/s, 28 in wide tiles; 1 x 1000 x 256 4.4, 7.4).
__global__ __launch_bounds__(H64::NT) void k_head_dw_few(DwArgs g) {
  QLORA_RING(H64, ring);
  Items items = {(int)((g.K + H64::BM - 1) / H64::BM), (int)((g.V + H64::BN - 1) / H64::BN), 1};
  dw_items<H64>(g, 0, (int)g.V, items, Turn{blockIdx.x, gridDim.x}, ring);
}

// Workgroups of a launch over `items` output tiles: as many as run at once (one per CU, three of the narrow tile), each
// taking several; below that one each, in eights (every XCD's run of items has the same length).
int64_t groups(int64_t items, int tile_rows) {
  const int64_t most = tile_rows == 64 ? kHeadSlots64 : 256;
  return items < most ? (items + 7) / 8 * 8 : most;
}

}  // namespace

#define QLORA_HEAD_TILES(rows_, CALL)   \
  switch ((rows_).tile_rows) {          \
    case 64: { CALL(H64); break; }      \
    case 128: { CALL(H128); break; }    \
    default: { CALL(H256); break; }     \
  }

hipError_t launch_head_logits(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *Xt, int64_t ldx,
                              const bf16_t *W, int64_t V, int64_t K, float c, float2 *stat, int64_t ntile, bf16_t *E,
                              int64_t lde, int64_t te, int k, int ranges, float *part, hipStream_t s) {
  const int64_t cols = head_tile_cols(rows.tile_rows), tiles = (V + cols - 1) / cols;
  const int64_t most = rows.tile_rows < 128 ? rows.tile_rows : 128;  // (all rows may take 128-row tiles)
#define QLORA_CALL(CFG)                                                                                            \
  launch(CFG::BN < 256 && ranges > 1 ? k_head_logits<CFG, CFG::BN < 256> : k_head_logits<CFG, false>,              \
         dim3((unsigned)groups(tiles * ((tb + most - 1) / most) * ranges, CFG::BN)), dim3(CFG::NT), 0, s,          \
         LogitArgs{rows, row0, tb, Xt, ldx, W, V, K, c, stat, ntile, (int)tiles, ranges, part, E, lde, te, k})
  QLORA_HEAD_TILES(rows, QLORA_CALL)
#undef QLORA_CALL
  return hipGetLastError();
}

hipError_t launch_head_dx(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *E, int64_t lde, int64_t te,
                          const bf16_t *W, int64_t V, int64_t K, const float4 *scale, float *part, bf16_t *dX,
                          hipStream_t s) {
  const int tr = rows.tile_rows, tc = head_tile_cols(tr);
  const int64_t most = (tb + 127) / 128 * ((K + tc - 1) / tc) * kHeadRanges;  // (all rows may take 128-row tiles)
#define QLORA_CALL(CFG)                                                                                              \
  launch(k_head_dx<CFG>, dim3((unsigned)groups(most, CFG::BN)), dim3(CFG::NT), 0, s, \
         DxArgs{rows, row0, tb, E, lde, te, W, V, K, scale, part, dX})
  QLORA_HEAD_TILES(rows, QLORA_CALL)
#undef QLORA_CALL
  return hipGetLastError();
}

hipError_t launch_head_dw(const HeadRows &rows, int64_t row0, int64_t tb, const bf16_t *E, int64_t lde, int64_t te,
                          const bf16_t *Xs, int64_t V, int64_t K, float *sums, bool first, bool last, int ranges,
                          bf16_t *dW, hipStream_t s) {
  const DwArgs args = {rows, row0, tb, E, lde, te, Xs, V, K, sums, first ? 1 : 0, last ? 1 : 0, ranges, dW};
  if (rows.tile_rows == 64) {
    const int64_t items = (K + H64::BM - 1) / H64::BM * ((V + H64::BN - 1) / H64::BN);
    launch(k_head_dw_few, dim3((unsigned)groups(items, 64)), dim3(H64::NT), 0, s, args);
    return hipGetLastError();
  }
  const int64_t tiles_m = (K + 255) / 256, whole = head_whole_columns(V, (int)tiles_m);
  const int64_t items = tiles_m * (whole > 0 ? (whole + 255) / 256 : (V + H128::BN - 1) / H128::BN * ranges);
  launch(k_head_dw, dim3((unsigned)groups(items, 256)), dim3(H256::NT), 0, s, args);
  return hipGetLastError();
}

}  // namespace qlora
