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
  unsigned any;  // one instruction, where min(lo, 1) would be compiled to a comparison and a selection
  asm("v_min_u32_e32 %0, 1, %1" : "=v"(any) : "v"((unsigned)b));
  return (float)__builtin_bit_cast(double, (uint64_t)((unsigned)(b >> 32) | any) << 32);
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

// 1 / sqrt(a): the estimate and two Newton steps (some 2^-52); the estimate itself where those do not apply (0 gives
// infinity, infinity 0).
__device__ __forceinline__ double inverse_sqrt(double a) {
  const double e = __builtin_amdgcn_rsq(a);
  double y = fma(0.5 * e, fma(-a * e, e, 1.0), e);
  y = fma(0.5 * y, fma(-a * y, y, 1.0), y);
  return a > 0.0 && a < __builtin_huge_val() ? y : e;
}

template <int CTRL>
__device__ __forceinline__ double from_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = (unsigned)__builtin_amdgcn_mov_dpp((int)(unsigned)b, CTRL, 0xF, 0xF, true);
  const unsigned hi = (unsigned)__builtin_amdgcn_mov_dpp((int)(unsigned)(b >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Permutations within a row of 16 lanes.
enum { DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_ROTATE4 = 0x124, DPP_ROTATE8 = 0x128, DPP_MIRROR8 = 0x141 };

// v of this lane plus v of the lane 16 (32) away.
__device__ __forceinline__ double add_swap16(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const auto lo = __builtin_amdgcn_permlane16_swap((unsigned)b, (unsigned)b, false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
  return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
}

__device__ __forceinline__ double add_swap32(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const auto lo = __builtin_amdgcn_permlane32_swap((unsigned)b, (unsigned)b, false, false);
  const auto hi = __builtin_amdgcn_permlane32_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
  return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
}

// Sum over each aligned group of 2^LOG lanes (LOG up to 4), in every lane.
template <int LOG>
__device__ __forceinline__ double group_sum(double v) {
  if constexpr (LOG >= 1) v += from_dpp<DPP_XOR1>(v);
  if constexpr (LOG >= 2) v += from_dpp<DPP_XOR2>(v);
  if constexpr (LOG == 3) v += from_dpp<DPP_MIRROR8>(v);  // quads are equal: the other one of 8 lanes
  if constexpr (LOG >= 4) {
    v += from_dpp<DPP_ROTATE4>(v);
    v += from_dpp<DPP_ROTATE8>(v);
  }
  return v;
}

// Two sums over each aligned group of 2^LOG lanes (LOG 2 to 6) at the cost of one: after a first exchange even lanes
// carry the first and odd lanes the second, and no later step mixes them.  Even lanes return the first sum.
template <int LOG>
__device__ __forceinline__ double group_sums(double s, double q) {
  const bool odd = threadIdx.x & 1;
  double v = (odd ? q : s) + from_dpp<DPP_XOR1>(odd ? s : q);
  v += from_dpp<DPP_XOR2>(v);
  if constexpr (LOG == 3) {  // the other quad by way of the mirror and the neighbour
    v += from_dpp<DPP_XOR1>(from_dpp<DPP_MIRROR8>(v));
  } else if constexpr (LOG >= 4) {
    v += from_dpp<DPP_ROTATE4>(v);
    v += from_dpp<DPP_ROTATE8>(v);
  }
  if constexpr (LOG >= 5) v = add_swap16(v);
  if constexpr (LOG >= 6) v = add_swap32(v);
  return v;
}

}  // namespace kq
