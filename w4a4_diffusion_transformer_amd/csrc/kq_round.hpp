// 64-bit arithmetic between bf16 rows: reading a piece of 8 channels, rounding
// once to bf16, sums over lanes (gfx950 only).
//
// fp64 multiply-adds issue at the rate of fp32 ones here, so a kernel that
// streams rows can afford them, and what it rounds is the formula's value to
// about 2^-50: its bf16 outputs and the codes taken from them are those of a
// 64-bit evaluation, also next to the border between two codes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_device.hpp"

namespace kq {

typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

// The 8 values of a 16-byte piece of a bf16 row.
__device__ __forceinline__ void piece_values(u32x4 v, double x[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = (double)bf16_lo(v[j]);
    x[2 * j + 1] = (double)bf16_hi(v[j]);
  }
}

// An fp32 value that rounds to bf16 as v does: the upper half of v's bits with
// its last bit set if the lower half is not zero (rounding to odd).  That has
// 21 significant bits, so the conversion to fp32 is exact (above 2^-126).
__device__ __forceinline__ float to_odd(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = (unsigned)b, hi = (unsigned)(b >> 32) | (lo < 1u ? lo : 1u);
  return (float)__builtin_bit_cast(double, (uint64_t)hi << 32);
}

// 8 values rounded once to bf16 (nearest even), packed.
__device__ __forceinline__ u32x4 round_piece(const double y[8]) {
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{to_odd(y[2 * j]), to_odd(y[2 * j + 1])}, bf16x2));
  return w;
}

// MXFP4 of a piece whose block of 32 channels lies in four adjacent lanes.
__device__ __forceinline__ void quantize_piece(u32x4 v, unsigned& word, unsigned& byte) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[2 * j] = bf16_lo(v[j]);
    y[2 * j + 1] = bf16_hi(v[j]);
  }
  byte = e8m0_byte(block_amax<LAYOUT_QUAD>(y));
  word = pack_fp4(y, byte);
}

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)b, CTRL, 0xF, 0xF, false);
  const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), CTRL, 0xF, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over each aligned group of 2^LOG lanes (LOG up to 6), in every lane: lanes 1 and 2 apart by quad
// permutations, then mirrors of 8 and 16 lanes, then the swaps of 16 and 32 lanes.
template <int LOG>
__device__ __forceinline__ double group_sum(double v) {
  if constexpr (LOG >= 1) v = dpp_add<0xB1>(v);
  if constexpr (LOG >= 2) v = dpp_add<0x4E>(v);
  if constexpr (LOG >= 3) v = dpp_add<0x141>(v);
  if constexpr (LOG >= 4) v = dpp_add<0x140>(v);
  if constexpr (LOG >= 5) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const auto lo = __builtin_amdgcn_permlane16_swap((unsigned)b, (unsigned)b, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    v = __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
  }
  if constexpr (LOG >= 6) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const auto lo = __builtin_amdgcn_permlane32_swap((unsigned)b, (unsigned)b, false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    v = __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
  }
  return v;
}

}  // namespace kq
