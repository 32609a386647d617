// Epilogue of the W4A4 products on fp32 sums (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq.h"
#include "kq_internal.h"
#include "kq_mxval.hpp"

namespace kq {

// exp(x) as 2^(x log2 e): relative error about |x| 2^-24 beside the instruction's one ulp.
__device__ __forceinline__ float exp_f32(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// x / (1 + exp(-u)): with u = x SiLU, with u = 2 sqrt(2 / pi) (x + 0.044715 x^3) the tanh form of
// GELU, since (1 + tanh(u / 2)) / 2 = 1 / (1 + exp(-u)).  exp overflows to infinity only where the
// result is zero; the reciprocal is the one-ulp instruction.
__device__ __forceinline__ float times_sigmoid(float x, float u) {
  return x * __builtin_amdgcn_rcpf(1.0f + exp_f32(-u));
}

// The N values of one column `col` of a lane; row(r) is value r's row.  fp32, one operation each in
// this order: + bias, activation, * gate, + residual.
template <int N, class Row>
__device__ __forceinline__ void epilogue(const Epilogue& e, float (&v)[N], const float (&res)[N], int col, int cols,
                                         Row&& row) {
  if (e.bias) {
    const float b = e.bias[col];
#pragma unroll
    for (int r = 0; r < N; ++r) v[r] += b;
  }
  if (e.act == KQ_ACT_GELU_TANH) {
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const float x = v[r];
      v[r] = times_sigmoid(x, x * (1.5957691216057308f + 0.07135481627260025f * (x * x)));
    }
  } else if (e.act == KQ_ACT_GELU_ERF) {
#pragma unroll
    for (int r = 0; r < N; ++r) v[r] = 0.5f * v[r] * (1.0f + erff(v[r] * 0.7071067811865476f));
  } else if (e.act == KQ_ACT_SILU) {
#pragma unroll
    for (int r = 0; r < N; ++r) v[r] = times_sigmoid(v[r], v[r]);
  }
  if (e.gate) {
#pragma unroll
    for (int r = 0; r < N; ++r) v[r] *= e.gate[(int64_t)fast_div((unsigned)row(r), e.by_rows) * cols + col];
  }
  if (e.residual) {
#pragma unroll
    for (int r = 0; r < N; ++r) v[r] = res[r] + v[r];
  }
}

}  // namespace kq
