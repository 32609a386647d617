// W4A4 product for few rows: Y = deq(A) deq(B)^T with the epilogue, where the
// 256 x 256 tiles of kq_gemm.hip would leave most of the GPU idle (a decode
// batch, the modulation vectors of a guidance pair), and K = 32.
//
// v_mfma_scale_f32_16x16x128_f8f6f4, both operands E2M1: lane l holds 32
// consecutive K values (16 bytes, one MX block) of row l % 16 at K offset
// 32 (l / 16), and that block's E8M0 byte; result register r is
// D[4 (l / 16) + r][l % 16].  A is the row operand, so a lane's column is one
// output channel.
//
// The cost is the latency of reading B once: a workgroup owns only 16 or 32
// channels, so that there are many, and its eight waves take K steps of 128
// in turn, each with its own operands straight from global memory into
// registers (a step reads 64 contiguous bytes of each row; nothing is shared
// between waves, so there is nothing to stage).  The waves' sums meet in LDS,
// added in wave order, so the result does not depend on timing.
#include <algorithm>

#include "kq_device.hpp"
#include "kq_epilogue.hpp"
#include "kq_internal.h"

namespace kq {

namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kAhead = 4;  // K steps whose loads are in flight at once

__device__ __forceinline__ i32x8 fp4_operand(i32x4 w) { return __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1); }

// Tile of 16 T x 16 T.
template <int T>
__global__ __launch_bounds__(kThreads) void gemm_rows_kernel(GemmArgs g) {
  __shared__ float sums[kWaves][T * T * 256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int gm = (g.M + 16 * T - 1) / (16 * T);
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int m0 = id % gm * (16 * T), n0 = id / gm * (16 * T);
  const int kbytes = g.K >> 1, kblocks = g.K >> 5, steps = (kblocks + 3) >> 2;
  const int blk = lane >> 4;

  // rows past the end read the last row; their results are not stored
  const uint8_t* ac[T];
  const uint8_t* as[T];
  const uint8_t* bc[T];
  const uint8_t* bs[T];
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int64_t m = min(m0 + 16 * i + (lane & 15), g.M - 1), n = min(n0 + 16 * i + (lane & 15), g.N - 1);
    ac[i] = g.a_codes + m * kbytes + 16 * blk;
    as[i] = g.a_scales + m * kblocks + blk;
    bc[i] = g.b_codes + n * kbytes + 16 * blk;
    bs[i] = g.b_scales + n * kblocks + blk;
  }
  f32x4 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  for (int s0 = wv; s0 < steps; s0 += kWaves * kAhead) {
    i32x4 a[kAhead][T], b[kAhead][T];
    int sa[kAhead][T], sb[kAhead][T];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int s = s0 + k * kWaves;
      const bool in = 4 * s + blk < kblocks;  // blocks past K: zero codes
#pragma unroll
      for (int i = 0; i < T; ++i) {
        a[k][i] = b[k][i] = i32x4{0, 0, 0, 0};
        sa[k][i] = sb[k][i] = 127;
        if (in) {
          a[k][i] = *reinterpret_cast<const i32x4*>(ac[i] + 64 * (int64_t)s);
          b[k][i] = *reinterpret_cast<const i32x4*>(bc[i] + 64 * (int64_t)s);
          sa[k][i] = as[i][4 * s];
          sb[k][i] = bs[i][4 * s];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (s0 + k * kWaves < steps) {
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
          for (int j = 0; j < T; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[k][i]), fp4_operand(b[k][j]),
                                                                         acc[i][j], 4, 4, 0, sa[k][i], 0, sb[k][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wv][((i * T + j) * 4 + r) * 64 + lane] = acc[i][j][r];
  __syncthreads();

  // output x of the tile: row x / (16 T), channel x % (16 T)
  for (int x = tid; x < T * T * 256; x += kThreads) {
    const int tm = x / (16 * T), tn = x % (16 * T);
    const int at = (((tm >> 4) * T + (tn >> 4)) * 4 + (tm & 3)) * 64 + ((tm & 15) >> 2) * 16 + (tn & 15);
    float v[1] = {0.0f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v[0] += sums[w][at];
    const int m = m0 + tm, n = n0 + tn;
    if (m < g.M && n < g.N) LaneColumns<1>(g.epi, n, 1).apply_and_store(g, v, m);
  }
}

}  // namespace

hipError_t launch_gemm_rows(const GemmArgs& args, hipStream_t stream) {
  GemmArgs g = args;
  const int t = g.M <= 16 ? 1 : 2;
  const int64_t grid = (int64_t)((g.M + 16 * t - 1) / (16 * t)) * ((g.N + 16 * t - 1) / (16 * t));
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  void* kargs[] = {&g};
  return hipLaunchKernel(t == 1 ? (const void*)&gemm_rows_kernel<1> : (const void*)&gemm_rows_kernel<2>,
                         dim3((unsigned)grid), dim3(kThreads), kargs, 0, stream);
}

}  // namespace kq
