// norm.hip -- layer norm over the hidden size and its gradients.
//
//   xh = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps),  y = xh w + b
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w
//   dw = sum_t dy xh,  db = sum_t dy
//
// Each kernel reads its rows once and keeps a row in registers between the two sums and the output, so both directions
// are bound by HBM (forward 8192 x 8192 50 us, 5.4 TB/s; backward 4096 x 4096 20 us, 5.0 TB/s, and 4 us for the weights'
// sums).  (The forward of more than 24576 columns has no registers for all of its weights and bias: 68 bytes a thread of
// binary32 ones, 52 of bf16, are in scratch memory; 4096 x 32768 122 and 112 us, 4.4 and 4.8 TB/s, 4096 x 24576 76, 5.3.)  The variance is taken from the centred row (no difference of large sums).  All sums are binary32 in
// a fixed order; bf16 outputs are rounded once.  Workgroups are persistent: they hold the weights (and, backward, the
// running sums of dw and db) of their columns in registers over all of their rows, and load the next row while the
// present one is reduced.  Of few rows the backward reads X and dY twice, from the caches, and is one launch.
#include "step.h"
#include "step_device.h"

namespace qlora {
namespace {

// Eight weights from a column on, as binary32.
template <bool F32>
__device__ __forceinline__ void load_w(const void *__restrict__ w, int64_t d, float out[8]) {
  if (F32) {
    const float4 *p = reinterpret_cast<const float4 *>((const float *)w + d);
    const float4 a = p[0], b = p[1];
    out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w, out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
  } else {
    unpack8(load16((const bf16_t *)w + d), out);
  }
}

// Sum over the NT threads of a row (consecutive waves of the workgroup), the same in all of them.  `at` is LDS that
// no thread still reads from an earlier sum.
template <int NT>
__device__ __forceinline__ float row_sum(float x, float *at, int wave) {
  x = wave_sum(x);
  if (NT == 64) return x;
  if ((threadIdx.x & 63) == 0) at[wave] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) s += at[i];
  return s;
}

// A workgroup of NT threads takes rows blockIdx.x, + gridDim.x, ..; a thread holds C chunks of 8 columns.  Y may be X.
template <int NT, int C, bool F32>
__global__ __launch_bounds__(NT) void k_norm(const bf16_t *X, int64_t T, int64_t D, const void *__restrict__ w,
                                             const void *__restrict__ b, float eps, bf16_t *Y, float *__restrict__ mean,
                                             float *__restrict__ rstd) {
  __shared__ float s_sum[4][NT / 64];
  const int tid = threadIdx.x, wave = tid >> 6;
  bool in[C];
  int64_t d[C];
  float wv[C][8], bv[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    d[c] = ((int64_t)c * NT + tid) * 8;
    in[c] = d[c] < D;
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[c][i] = bv[c][i] = 0.f;
    if (in[c]) {
      load_w<F32>(w, d[c], wv[c]);
      if (b) load_w<F32>(b, d[c], bv[c]);
    }
  }
  const float n = (float)D;
  u32x4_t next[C];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int c = 0; c < C; ++c) next[c] = t < T && in[c] ? load16(X + t * D + d[c]) : u32x4_t{0u, 0u, 0u, 0u};
  };
  load(blockIdx.x);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, turn ^= 2) {
    float x[C][8], sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) unpack8(next[c], x[c]);
    load(t + gridDim.x);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[c][i];
    const float m = row_sum<NT>(sum, s_sum[turn], wave) / n;
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (in[c])
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[c][i] -= m;
          sq = fmaf(x[c][i], x[c][i], sq);
        }
    const float r = 1.f / sqrtf(row_sum<NT>(sq, s_sum[turn + 1], wave) / n + eps);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (in[c]) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(x[c][i] * r, wv[c][i], bv[c][i]);
        store16_once(Y + t * D + d[c], pack8(y));
      }
    if (tid == 0) {
      if (mean) mean[t] = m;
      if (rstd) rstd[t] = r;
    }
  }
}

// Eight columns' sums of dw and db, rows 0 and 1 of `out`.
__device__ __forceinline__ void store_sums(float *__restrict__ out, int64_t D, int64_t d, const float dw[8],
                                           const float db[8]) {
  float4 *pw = reinterpret_cast<float4 *>(out + d), *pb = reinterpret_cast<float4 *>(out + D + d);
  pw[0] = make_float4(dw[0], dw[1], dw[2], dw[3]);
  pw[1] = make_float4(dw[4], dw[5], dw[6], dw[7]);
  pb[0] = make_float4(db[0], db[1], db[2], db[3]);
  pb[1] = make_float4(db[4], db[5], db[6], db[7]);
}

struct NormBwd {
  const bf16_t *X, *dY;
  int64_t T, D;
  const void *w;
  const float *mean, *rstd;
  bf16_t *dX;
  float *part;
};
template <int NT, int C, bool SUMS>
struct BwdShared {
  static constexpr int G = 1024 / NT;
  float sum[2][G][2][NT / 64];
  __attribute__((aligned(16))) float part[SUMS && G > 1 ? NT * C * 16 : 4];
};
// A workgroup of up to 1024 threads in groups of NT, each with a row at a time.  The sums of dw and db stay in registers over
// the workgroup's rows; then the groups add theirs in LDS, one after the other, and the workgroup's go to part[block].
// (C = 4, the longest rows: the sums do not fit the registers beside a row and come from k_norm_columns; 8192 x 32768
// 515 us in all; of 1024 rows it took 86, with spilled registers 191.)
template <int NT, int C, bool F32, bool SUMS>
__device__ __forceinline__ void norm_bwd_rows(const NormBwd &p, int64_t block, int64_t blocks, char *shared) {
  constexpr int G = 1024 / NT, WAVES = NT / 64;
  const bf16_t *__restrict__ const X = p.X;
  const bf16_t *const dY = p.dY;
  const int64_t T = p.T, D = p.D;
  const void *__restrict__ const w = p.w;
  const float *__restrict__ const mean = p.mean, *__restrict__ const rstd = p.rstd;
  bf16_t *const dX = p.dX;
  float *__restrict__ const part = p.part;
  auto &sh = *reinterpret_cast<BwdShared<NT, C, SUMS> *>(shared);
  auto &s_sum = sh.sum;
  float *const s_part = sh.part;
  const int g = __builtin_amdgcn_readfirstlane(threadIdx.x / NT), tid = threadIdx.x % NT;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  bool in[C];
  uint32_t d[C];
  float wv[C][8], dw[SUMS ? C : 1][8], db[SUMS ? C : 1][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    d[c] = (c * NT + tid) * 8;
    in[c] = d[c] < D;
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[c][i] = dw[SUMS ? c : 0][i] = db[SUMS ? c : 0][i] = 0.f;
    if (in[c]) load_w<F32>(w, d[c], wv[c]);
  }
  const float n = (float)D;
  struct Row {
    u32x4_t x[C], g[C];
    float m, r;
  };
  auto load = [&](Row &to, int64_t t) {
    const bool ok = t < T;
    to.m = ok ? mean[t] : 0.f;
    to.r = ok ? rstd[t] : 0.f;
    const bf16_t *const x = X + t * D, *const y = dY + t * D;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      to.x[c] = to.g[c] = u32x4_t{0u, 0u, 0u, 0u};
      if (ok && in[c]) {
        to.x[c] = load16(x + d[c]);
        to.g[c] = load16(y + d[c]);
      }
    }
  };
  const int64_t first = block * G, step = blocks * G;
  // row t of this group (behind the last one a row of zeros: every thread meets the barriers)
  auto work = [&](const Row &row, int64_t t, int turn) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      // (Behind the row's end xh is 0 - mean rstd, which may overflow and must not meet a zero.  With the sums a branch
      // costs more than a select: 4096 x 4096 24.0 us, so 22.8.)
      if (!SUMS && !in[c]) continue;
      float x[8], y[8];
      unpack8(row.x[c], x);
      unpack8(row.g[c], y);
      const float before = b;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (x[i] - row.m) * row.r, gd = y[i] * wv[c][i];
        if (SUMS) {
          dw[c][i] = fmaf(y[i], xh, dw[c][i]);
          db[c][i] += y[i];
        }
        a += gd;
        b = fmaf(gd, xh, b);
      }
      if (SUMS) b = in[c] ? b : before;
    }
    if (!dX) return;
    a = wave_sum(a);
    b = wave_sum(b);
    if (NT > 64) {
      if ((tid & 63) == 0) s_sum[turn][g][0][wave] = a, s_sum[turn][g][1][wave] = b;
      __syncthreads();
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) a += s_sum[turn][g][0][i], b += s_sum[turn][g][1][i];
    }
    if (t >= T) return;
    a /= n;
    b /= n;
    bf16_t *const out = dX + t * D;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (in[c]) {
        float x[8], y[8];
        unpack8(row.x[c], x);
        unpack8(row.g[c], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (x[i] - row.m) * row.r;
          y[i] = (fmaf(y[i], wv[c][i], -a) - xh * b) * row.r;
        }
        store16_once(out + d[c], pack8(y));
      }
  };
  Row even;
  if constexpr (SUMS) {
    Row odd;
    load(even, first + g);
    for (int64_t t0 = first; t0 < T; t0 += 2 * step) {
      load(odd, t0 + step + g);
      work(even, t0 + g, 0);
      if (t0 + step >= T) break;
      load(even, t0 + 2 * step + g);
      work(odd, t0 + step + g, 1);
    }
  } else {  // (one row in the registers)
    int turn = 0;
    for (int64_t t0 = first; t0 < T; t0 += step, turn ^= 1) {
      load(even, t0 + g);
      work(even, t0 + g, turn);
    }
    return;
  }
  if (!part) return;
  if (G > 1) {
    for (int q = 0; q < G; ++q) {
      if (q) __syncthreads();
      if (g != q) continue;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        // (each thread has its column's slot, in steps of 4 bytes from lane to lane)
        float *at = s_part + c * NT * 16 + tid;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (q) dw[c][i] += at[i * NT], db[c][i] += at[(8 + i) * NT];
          if (q + 1 < G) at[i * NT] = dw[c][i], at[(8 + i) * NT] = db[c][i];
        }
      }
    }
    if (g != G - 1) return;
  }
  float *out = part + block * 2 * D;
#pragma unroll
  for (int c = 0; c < (SUMS ? C : 0); ++c)
    if (in[c]) store_sums(out, D, d[c], dw[c], db[c]);
}

template <int NT, int C, bool F32>
__global__ __launch_bounds__(1024 / NT * NT) void k_norm_bwd(NormBwd p) {
  __shared__ __attribute__((aligned(16))) char shared[sizeof(BwdShared<NT, C, C <= 2>)];
  norm_bwd_rows<NT, C, F32, C <= 2>(p, blockIdx.x, gridDim.x, shared);
}

// Few rows: dX in the first workgroups and, from the statistics that the forward left, dw and db in the others: 64 columns
// each, the rows to 128 teams of eight lanes in turn, whose sums are added in a fixed order (17 x 1808 4.1 us, else 4.2 and
// 4.0 in two launches; 512 x 16384 17 us, else 24).
struct ColumnShared {
  float sum[128][8][17];
};
__device__ __forceinline__ void norm_columns_few(const NormBwd &p, int64_t block, bool f32, void *__restrict__ dw,
                                                 void *__restrict__ db, char *shared) {
  auto &s_sum = reinterpret_cast<ColumnShared *>(shared)->sum;
  const int tid = threadIdx.x, lane = tid & 7, team = tid >> 3;
  const int64_t d = block * 64 + lane * 8;
  float sum[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] = 0.f;
  if (d < p.D)
#pragma unroll 4
    for (int64_t t = team; t < p.T; t += 128) {
      const float m = p.mean[t], r = p.rstd[t];
      float x[8], y[8];
      unpack8(load16(p.X + t * p.D + d), x);
      unpack8(load16(p.dY + t * p.D + d), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[i] = fmaf(y[i], (x[i] - m) * r, sum[i]);
        sum[8 + i] += y[i];
      }
    }
#pragma unroll
  for (int i = 0; i < 16; ++i) s_sum[team][lane][i] = sum[i];
  __syncthreads();
  const int of_db = tid >> 6, col = tid & 63;
  const int64_t at = block * 64 + col;
  void *const to = of_db ? db : dw;
  if (of_db > 1 || !to || at >= p.D) return;
  float four[4] = {0.f, 0.f, 0.f, 0.f};  // (teams 0, 4, ..; 1, 5, ..; and so on)
#pragma unroll 16
  for (int q = 0; q < 128; q += 4)
#pragma unroll
    for (int i = 0; i < 4; ++i) four[i] += s_sum[q + i][col >> 3][of_db * 8 + (col & 7)];
  const float all = (four[0] + four[1]) + (four[2] + four[3]);
  if (f32) ((float *)to)[at] = all;
  else ((bf16_t *)to)[at] = f32_to_bf16(all);
}
template <int NT, int C, bool F32>
__global__ __launch_bounds__(1024) void k_norm_few(NormBwd p, int64_t row_blocks, void *__restrict__ dw,
                                                   void *__restrict__ db) {
  constexpr int kRows = sizeof(BwdShared<NT, C, false>), kColumns = sizeof(ColumnShared);
  __shared__ __attribute__((aligned(16))) char shared[kRows > kColumns ? kRows : kColumns];
  if (blockIdx.x < row_blocks) norm_bwd_rows<NT, C, F32, false>(p, blockIdx.x, row_blocks, shared);
  else norm_columns_few(p, blockIdx.x - row_blocks, F32, dw, db, shared);
}

// The sums alone: 2048 columns, every gridDim.y-th row.
__global__ __launch_bounds__(256) void k_norm_columns(const bf16_t *__restrict__ X, const bf16_t *__restrict__ dY, int64_t T,
                                                      int64_t D, const float *__restrict__ mean,
                                                      const float *__restrict__ rstd, float *__restrict__ part) {
  const int64_t d = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (d >= D) return;
  float dw[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.f;
#pragma unroll 4
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    const float m = mean[t], r = rstd[t];
    float x[8], y[8];
    unpack8(load16(X + t * D + d), x);
    unpack8(load16(dY + t * D + d), y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] = fmaf(y[i], (x[i] - m) * r, dw[i]);
      db[i] += y[i];
    }
  }
  store_sums(part + (int64_t)blockIdx.y * 2 * D, D, d, dw, db);
}

// dw and db from the workgroups' sums: 64 columns per workgroup, each of 16 waves adds a sixteenth of the sums, then
// the sixteenths in order.
__global__ __launch_bounds__(1024) void k_norm_reduce(const float *__restrict__ part, int groups, int64_t D, bool f32,
                                                      void *__restrict__ dw, void *__restrict__ db) {
  __shared__ float s_sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;  // of [2][D]
  const int per = (groups + 15) / 16, a = wave * per, b = a + per < groups ? a + per : groups;
  float sum = 0.f;
  if (col < 2 * D)
#pragma unroll 8
    for (int q = a; q < b; ++q) sum += part[(int64_t)q * 2 * D + col];
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (wave > 0 || col >= 2 * D) return;
#pragma unroll
  for (int q = 1; q < 16; ++q) sum += s_sum[q][lane];
  void *to = col < D ? dw : db;
  if (!to) return;
  const int64_t at = col < D ? col : col - D;
  if (f32) ((float *)to)[at] = sum;
  else ((bf16_t *)to)[at] = f32_to_bf16(sum);
}

}  // namespace

#define NORM_CASE(NT_, C_, kern, ...)                                  \
  do {                                                                 \
    if (f32) launch(kern<NT_, C_, true>, __VA_ARGS__);                 \
    else launch(kern<NT_, C_, false>, __VA_ARGS__);                    \
  } while (0)

hipError_t launch_norm(const bf16_t *X, int64_t T, int64_t D, const void *w, const void *b, bool f32, float eps, bf16_t *Y,
                       float *mean, float *rstd, hipStream_t s) {
  // threads of a row: few of them, whose sums need few exchanges, where the rows fill the GPU
  int nt = D <= 2048 ? 64 : D <= 8192 ? 256 : 1024;
  while (nt < 1024 && (int64_t)nt * 8 < D && T * nt < 256 * 1024) nt *= 4;
  // (1024 threads with two chunks would be half idle: 7229 x 8992 63 us, so 47)
  if (D > 8192 && D <= 12288 && T >= 512) nt = 512;
  const int c = (int)((D + nt * 8 - 1) / (nt * 8));
  const int64_t most = 256 * 1024 / nt;
  const dim3 grid((uint32_t)(T < most ? T : most)), block(nt);
#define NORM_ARGS grid, block, 0, s, X, T, D, w, b, eps, Y, mean, rstd
#define NORM_NT(NT_)                                     \
  do {                                                   \
    if (c <= 1) NORM_CASE(NT_, 1, k_norm, NORM_ARGS);    \
    else if (c <= 2) NORM_CASE(NT_, 2, k_norm, NORM_ARGS); \
    else if (c <= 3) NORM_CASE(NT_, 3, k_norm, NORM_ARGS); \
    else NORM_CASE(NT_, 4, k_norm, NORM_ARGS);           \
  } while (0)
  if (nt == 64) NORM_NT(64);
  else if (nt == 256) NORM_NT(256);
  else if (nt == 512) NORM_CASE(512, 3, k_norm, NORM_ARGS);
  else NORM_NT(1024);
#undef NORM_NT
#undef NORM_ARGS
  return hipGetLastError();
}

namespace {
int bwd_threads(int64_t D) { return D <= 1024 ? 64 : D <= 4096 ? 256 : 1024; }
}  // namespace

int norm_bwd_groups(int64_t T, int64_t D) {
  const int64_t g = 1024 / bwd_threads(D), need = (T + g - 1) / g;
  return (int)(need < 1 ? 1 : need < 256 ? need : 256);
}

hipError_t launch_norm_bwd(const bf16_t *X, const bf16_t *dY, int64_t T, int64_t D, const void *w, bool f32,
                           const float *mean, const float *rstd, bf16_t *dX, float *part, hipStream_t s) {
  const int nt = bwd_threads(D), c = (int)((D + nt * 8 - 1) / (nt * 8));
  const dim3 grid((uint32_t)norm_bwd_groups(T, D));
  const NormBwd p{X, dY, T, D, w, mean, rstd, dX, part};
  // (where 1024 threads would be half idle: 4096 x 4104 23.6 us, so 22.0.  Few rows stay with the threads that k_norm_few
  // has, so that dX does not depend on what else is asked for.)
  const bool many = !norm_bwd_few(T, D);
  if (many && D > 4096 && D <= 6144) {
    NORM_CASE(768, 1, k_norm_bwd, grid, dim3(768), 0, s, p);
    return hipGetLastError();
  }
  if (many && D > 8192 && D <= 12288) {
    NORM_CASE(768, 2, k_norm_bwd, grid, dim3(768), 0, s, p);
    return hipGetLastError();
  }
  const dim3 block(1024);
#define NORM_NT(kern, ...)                                             \
  do {                                                                 \
    if (nt == 64 && c <= 1) NORM_CASE(64, 1, kern, __VA_ARGS__);       \
    else if (nt == 64) NORM_CASE(64, 2, kern, __VA_ARGS__);            \
    else if (nt == 256 && c <= 1) NORM_CASE(256, 1, kern, __VA_ARGS__); \
    else if (nt == 256) NORM_CASE(256, 2, kern, __VA_ARGS__);          \
    else if (c <= 1) NORM_CASE(1024, 1, kern, __VA_ARGS__);            \
    else if (c <= 2) NORM_CASE(1024, 2, kern, __VA_ARGS__);            \
    else NORM_CASE(1024, 4, kern, __VA_ARGS__);                        \
  } while (0)
  NORM_NT(k_norm_bwd, grid, block, 0, s, p);
  return hipGetLastError();
}

// Up to 768 rows one launch gains at every width (768 x 4096 10.5 us, else 13.3; x 5992 14.2 and 16.3; x 16384 24.9 and
// 26.5).  At 1024 rows the second reads cost more than the launches where rows do not begin with a line of memory or are long
// (x 5992 17.8 and 17.0, x 8192 18.5 and 18.4, x 16384 32.0 and 30.9); rows of up to 4096 columns would still gain (12.0 and
// 14.1).  2048 x 32768 117 us, with k_norm_columns 146; 8192 x 24576 390 and 379.
bool norm_bwd_few(int64_t T, int64_t D) { return T <= (norm_bwd_columns(D) ? 2048 : 768); }

hipError_t launch_norm_few(const bf16_t *X, const bf16_t *dY, int64_t T, int64_t D, const void *w, bool f32,
                           const float *mean, const float *rstd, bf16_t *dX, void *dw, void *db, hipStream_t s) {
  const int nt = bwd_threads(D), c = (int)((D + nt * 8 - 1) / (nt * 8));
  const int64_t rows = dX ? norm_bwd_groups(T, D) : 0;
  const dim3 grid((uint32_t)(rows + (D + 63) / 64)), block(1024);
  const NormBwd p{X, dY, T, D, w, mean, rstd, dX, nullptr};
  NORM_NT(k_norm_few, grid, block, 0, s, p, rows, dw, db);
#undef NORM_NT
  return hipGetLastError();
}

bool norm_bwd_columns(int64_t D) { return D > 16384; }

hipError_t launch_norm_columns(const bf16_t *X, const bf16_t *dY, int64_t T, int64_t D, const float *mean, const float *rstd,
                               float *part, hipStream_t s) {
  launch(k_norm_columns, dim3((uint32_t)((D + 2047) / 2048), (uint32_t)norm_bwd_groups(T, D)), dim3(256), 0, s, X, dY, T, D,
         mean, rstd, part);
  return hipGetLastError();
}

hipError_t launch_norm_reduce(const float *part, int groups, int64_t D, bool f32, void *dw, void *db, hipStream_t s) {
  launch(k_norm_reduce, dim3((uint32_t)((2 * D + 63) / 64)), dim3(1024), 0, s, part, groups, D, f32, dw, db);
  return hipGetLastError();
}

}  // namespace qlora
