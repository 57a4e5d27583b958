// step_device.h -- device helpers of the step's other kernels (embed.hip, norm.hip, adapters.hip).
#pragma once
#include "device.h"

namespace qlora {

// Sum over the wave's 64 lanes, the same in every lane; the order of the additions is fixed.  Each step adds a
// neighbour's value through the VALU's own lane permutations: no LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float x) {
  const int y = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xf, true);
  return x + __builtin_bit_cast(float, y);
}
__device__ __forceinline__ float wave_sum(float x) {
  x = add_dpp<0x111, 0xf>(x);  // row_shr by 1, 2, 4, 8: lane 15 of each row of 16 holds the row's sum
  x = add_dpp<0x112, 0xf>(x);
  x = add_dpp<0x114, 0xf>(x);
  x = add_dpp<0x118, 0xf>(x);
  x = add_dpp<0x142, 0xa>(x);  // row_bcast:15 into rows 1 and 3, then row_bcast:31 into rows 2 and 3
  x = add_dpp<0x143, 0xc>(x);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

__device__ __forceinline__ void unpack8(const u32x4_t &v, float out[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    out[2 * i] = bf16_lo_to_f32(w);
    out[2 * i + 1] = bf16_hi_to_f32(w);
  }
}
__device__ __forceinline__ u32x4_t pack8(const float v[8]) {
  return u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
__device__ __forceinline__ u32x4_t load16(const bf16_t *p) { return *reinterpret_cast<const u32x4_t *>(p); }
__device__ __forceinline__ void store16(bf16_t *p, const u32x4_t &v) { *reinterpret_cast<u32x4_t *>(p) = v; }
// The same past the caches, for an output that is not read again here (into memory that is not in the caches anyway an
// embedding of 8192 x 8192 53 -> 44 us, a norm of 4096 x 4096 13.4 -> 12.1) and an operand that they cannot hold.
__device__ __forceinline__ u32x4_t load16_once(const bf16_t *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(p));
}
__device__ __forceinline__ void store16_once(bf16_t *p, const u32x4_t &v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t *>(p));
}

}  // namespace qlora
