// norm.hip -- layer norm over the hidden size and its gradients.
//
//   xh = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps),  y = xh w + b
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w
//   dw = sum_t dy xh,  db = sum_t dy
//
// Each kernel reads its rows once and keeps a row in registers between the two sums and the output, so both directions
// are bound by HBM.  The variance is taken from the centred row (no difference of large sums).  All sums are binary32 in
// a fixed order; bf16 outputs are rounded once.  Workgroups are persistent: they hold the weights (and, backward, the
// running sums of dw and db) of their columns in registers over all of their rows, and load the next row while the
// present one is reduced.
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

// A workgroup of NT threads takes rows blockIdx.x, + gridDim.x, ..; a thread holds C chunks of 8 columns.
template <int NT, int C, bool F32>
__global__ __launch_bounds__(NT) void k_norm(const bf16_t *__restrict__ X, int64_t T, int64_t D,
                                             const void *__restrict__ w, const void *__restrict__ b, float eps,
                                             bf16_t *__restrict__ Y, float *__restrict__ mean, float *__restrict__ rstd) {
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
        store16(Y + t * D + d[c], pack8(y));
      }
    if (tid == 0) {
      if (mean) mean[t] = m;
      if (rstd) rstd[t] = r;
    }
  }
}

// A workgroup of 1024 threads in groups of NT, each with a row at a time.  The sums of dw and db stay in registers over
// the workgroup's rows; then the groups add theirs in LDS, one after the other, and the workgroup's go to part[block].
template <int NT, int C, bool F32>
__global__ __launch_bounds__(1024) void k_norm_bwd(const bf16_t *__restrict__ X, const bf16_t *__restrict__ dY, int64_t T,
                                                   int64_t D, const void *__restrict__ w, const float *__restrict__ mean,
                                                   const float *__restrict__ rstd, bf16_t *__restrict__ dX,
                                                   float *__restrict__ part) {
  constexpr int G = 1024 / NT, WAVES = NT / 64;
  __shared__ float s_sum[2][G][2][WAVES];
  __shared__ __attribute__((aligned(16))) float s_part[G > 1 ? NT * C * 16 : 1];
  const int g = threadIdx.x / NT, tid = threadIdx.x % NT, wave = tid >> 6;
  bool in[C];
  int64_t d[C];
  float wv[C][8], dw[C][8], db[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    d[c] = ((int64_t)c * NT + tid) * 8;
    in[c] = d[c] < D;
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[c][i] = dw[c][i] = db[c][i] = 0.f;
    if (in[c]) load_w<F32>(w, d[c], wv[c]);
  }
  const float n = (float)D;
  u32x4_t nx[C], ng[C];
  float nm, nr;
  auto load = [&](int64_t t) {
    const bool ok = t < T;
    nm = ok ? mean[t] : 0.f;
    nr = ok ? rstd[t] : 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      nx[c] = ng[c] = u32x4_t{0u, 0u, 0u, 0u};
      if (ok && in[c]) {
        nx[c] = load16(X + t * D + d[c]);
        ng[c] = load16(dY + t * D + d[c]);
      }
    }
  };
  const int64_t first = (int64_t)blockIdx.x * G, step = (int64_t)gridDim.x * G;
  load(first + g);
  int turn = 0;
  for (int64_t t0 = first; t0 < T; t0 += step, turn ^= 1) {
    const int64_t t = t0 + g;  // (a group behind the last row works on zeros: every thread meets the barriers)
    const float m = nm, r = nr;
    u32x4_t rx[C], rg[C];
#pragma unroll
    for (int c = 0; c < C; ++c) rx[c] = nx[c], rg[c] = ng[c];
    load(t + step);
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float x[8], y[8];
      unpack8(rx[c], x);
      unpack8(rg[c], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (x[i] - m) * r, gd = y[i] * wv[c][i];
        dw[c][i] = fmaf(y[i], xh, dw[c][i]);
        db[c][i] += y[i];
        a += gd;
        b = fmaf(gd, xh, b);
      }
    }
    if (!dX) continue;
    a = wave_sum(a);
    b = wave_sum(b);
    if (NT > 64) {
      if ((tid & 63) == 0) s_sum[turn][g][0][wave] = a, s_sum[turn][g][1][wave] = b;
      __syncthreads();
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) a += s_sum[turn][g][0][i], b += s_sum[turn][g][1][i];
    }
    a /= n;
    b /= n;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (t < T && in[c]) {
        float x[8], y[8];
        unpack8(rx[c], x);
        unpack8(rg[c], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (x[i] - m) * r;
          y[i] = (fmaf(y[i], wv[c][i], -a) - xh * b) * r;
        }
        store16(dX + t * D + d[c], pack8(y));
      }
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
  float *out = part + (int64_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (in[c]) {
      float4 *pw = reinterpret_cast<float4 *>(out + d[c]), *pb = reinterpret_cast<float4 *>(out + D + d[c]);
      pw[0] = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
      pw[1] = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
      pb[0] = make_float4(db[c][0], db[c][1], db[c][2], db[c][3]);
      pb[1] = make_float4(db[c][4], db[c][5], db[c][6], db[c][7]);
    }
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
  const int c = (int)((D + nt * 8 - 1) / (nt * 8));
  const int64_t most = 256 * 1024 / nt;
  const dim3 grid((uint32_t)(T < most ? T : most)), block(nt);
#define NORM_ARGS grid, block, 0, s, X, T, D, w, b, eps, Y, mean, rstd
#define NORM_NT(NT_)                                     \
  do {                                                   \
    if (c <= 1) NORM_CASE(NT_, 1, k_norm, NORM_ARGS);    \
    else if (c <= 2) NORM_CASE(NT_, 2, k_norm, NORM_ARGS); \
    else NORM_CASE(NT_, 4, k_norm, NORM_ARGS);           \
  } while (0)
  if (nt == 64) NORM_NT(64);
  else if (nt == 256) NORM_NT(256);
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
  const dim3 grid((uint32_t)norm_bwd_groups(T, D)), block(1024);
#define NORM_ARGS grid, block, 0, s, X, dY, T, D, w, mean, rstd, dX, part
#define NORM_NT(NT_)                                           \
  do {                                                         \
    if (c <= 1) NORM_CASE(NT_, 1, k_norm_bwd, NORM_ARGS);      \
    else NORM_CASE(NT_, 2, k_norm_bwd, NORM_ARGS);             \
  } while (0)
  if (nt == 64) NORM_NT(64);
  else if (nt == 256) NORM_NT(256);
  else if (c <= 2) NORM_NT(1024);
  else NORM_CASE(1024, 4, k_norm_bwd, NORM_ARGS);
#undef NORM_NT
#undef NORM_ARGS
  return hipGetLastError();
}

hipError_t launch_norm_reduce(const float *part, int groups, int64_t D, bool f32, void *dw, void *db, hipStream_t s) {
  launch(k_norm_reduce, dim3((uint32_t)((2 * D + 63) / 64)), dim3(1024), 0, s, part, groups, D, f32, dw, db);
  return hipGetLastError();
}

}  // namespace qlora
