// Reading MXFP4 on the device: values of codes, the index arithmetic of paged
// caches, and wave-private LDS (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_internal.h"

namespace kq {

typedef __attribute__((ext_vector_type(8))) __bf16 mx_bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 mx_bf16x2;

// The eight values of a code word (low nibble first) under scale byte
// `byte`, in bf16: v_cvt_scalef32_pk_bf16_fp4 multiplies by 2^(exponent field
// of its scale operand - 127), field 0 reading as 2^-127, exactly.
__device__ __forceinline__ mx_bf16x8 mx_values8(unsigned word, unsigned byte) {
  const float scale = __uint_as_float(byte << 23);
  const mx_bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 0);
  const mx_bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 1);
  const mx_bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 2);
  const mx_bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 3);
  return mx_bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// n / d for 0 <= n < 2^31 by one multiply: with l = ceil(log2 d) and
// m = floor(2^(31 + l) / d) + 1, m d = 2^(31 + l) + e with 0 < e <= d <= 2^l,
// so n m / 2^(31 + l) exceeds n / d by n e / (d 2^(31 + l)) < 1 / d: the floors agree.
__device__ __forceinline__ unsigned fast_div(unsigned n, Divisor d) {
  return (unsigned)(((uint64_t)n * d.m) >> d.shift);
}

// Orders a wave's own LDS accesses for the compiler; the hardware runs them in order.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace kq
