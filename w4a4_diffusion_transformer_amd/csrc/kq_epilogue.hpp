// Epilogue of the W4A4 products on fp32 sums (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq.h"
#include "kq_device.hpp"
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

__device__ __forceinline__ float activation(int act, float x) {
  if (act == KQ_ACT_GELU_TANH) return times_sigmoid(x, x * (1.5957691216057308f + 0.07135481627260025f * (x * x)));
  if (act == KQ_ACT_GELU_ERF) return 0.5f * x * (1.0f + erff(x * 0.7071067811865476f));
  if (act == KQ_ACT_SILU) return times_sigmoid(x, x);
  return x;
}

// The epilogue for a lane whose values are C consecutive channels n .. of any
// row: + bias, activation, * gate, + residual, one fp32 operation each in
// this order.  cols: how many of the channels there are.
template <int C>
struct LaneColumns {
  int n, cols;
  bool one_sample = false;  // gate holds the only sample that the lane's rows have (uniform)
  float bias[C], gate[C];

  __device__ __forceinline__ LaneColumns(const Epilogue& e, int n_, int cols_) : n(n_), cols(cols_) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      bias[c] = e.bias && c < cols ? e.bias[n + c] : 0.0f;
      gate[c] = 0.0f;
    }
  }

  // Keeps the gate in registers where rows `first` .. `last` (uniform) are of one sample.
  __device__ __forceinline__ void load_gate(const GemmArgs& g, int first, int last) {
    if (!g.epi.gate || first > last) return;
    const int s = (int)fast_div((unsigned)first, g.epi.by_rows);
    one_sample = s == (int)fast_div((unsigned)last, g.epi.by_rows);
    if (!one_sample) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < cols) gate[c] = g.epi.gate[(int64_t)s * g.N + n + c];
  }

  // res: the residual's values, if there is one.
  __device__ __forceinline__ void apply(const GemmArgs& g, float (&v)[C], int m, const float (&res)[C]) const {
    const Epilogue& e = g.epi;
    if (e.bias) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] += bias[c];
    }
    if (e.act == KQ_ACT_GELU_TANH) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = activation(KQ_ACT_GELU_TANH, v[c]);
    } else if (e.act == KQ_ACT_GELU_ERF) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = activation(KQ_ACT_GELU_ERF, v[c]);
    } else if (e.act == KQ_ACT_SILU) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = activation(KQ_ACT_SILU, v[c]);
    }
    if (e.gate) {
      if (one_sample) {
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] *= gate[c];
      } else {
        const float* row = e.gate + (int64_t)fast_div((unsigned)m, e.by_rows) * g.N + n;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c < cols) v[c] *= row[c];
      }
    }
    if (e.residual) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = res[c] + v[c];
    }
  }

  // One row, element by element: for rows and pointers of any alignment.
  __device__ __forceinline__ void apply_and_store(const GemmArgs& g, float (&v)[C], int m) const {
    const int64_t at = (int64_t)m * g.N + n;
    float res[C];
#pragma unroll
    for (int c = 0; c < C; ++c) res[c] = g.epi.residual && c < cols ? bf16_lo(g.epi.residual[at + c]) : 0.0f;
    apply(g, v, m, res);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (c >= cols) continue;
      if (g.y_f32) g.y_f32[at + c] = v[c];
      if (g.y_bf16) g.y_bf16[at + c] = __builtin_bit_cast(uint16_t, (__bf16)v[c]);
    }
  }
};

}  // namespace kq
