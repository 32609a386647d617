// W4A4 product for few rows: Y = deq(A) deq(B)^T with the epilogue, where the
// 256 x 256 tiles of kq_gemm.hip would leave most of the GPU idle (a decode
// batch, the modulation vectors of a guidance pair).
//
// v_mfma_scale_f32_16x16x128_f8f6f4, both operands E2M1: lane l holds 32
// consecutive K values (16 bytes, one MX block) of row l % 16 at K offset
// 32 (l / 16), and that block's E8M0 byte; result register r is
// D[4 (l / 16) + r][l % 16].  A is the row operand, so a lane's column is one
// output channel.
//
// The cost is reading B once: a workgroup owns only 16 or 32 channels, so
// that there are many, and its eight waves take K steps of 128 in turn, each
// with its own operands straight from global memory into registers (nothing
// is shared between waves, so nothing waits for a barrier).  Four adjacent
// lanes read the 64 bytes of a row, since loads are merged among adjacent
// lanes only, and the operands change lanes through wave-private LDS; in the
// operand order every lane was an access of its own (16 x 4608 x 12288 23.7
// us, 12.5 so; 64 rows 44.7 and 22.5).  The waves' sums meet in LDS, added in wave order, so the result does
// not depend on timing.
#include <algorithm>

#include "kq_device.hpp"
#include "kq_epilogue.hpp"
#include "kq_internal.h"

namespace kq {

namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kAhead = 4;  // K steps whose loads a wave has in flight at once: the bytes of a scale register

__device__ __forceinline__ i32x8 fp4_operand(i32x4 w) { return __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1); }

// D += A B of one step, the operands' scales in byte K of their registers.
template <int K>
__device__ __forceinline__ f32x4 multiply(i32x4 a, int sa, i32x4 b, int sb, f32x4 d) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a), fp4_operand(b), d, 4, 4, K, sa, K, sb);
}

// Tile of 16 T x 16 T.
template <int T>
__global__ __launch_bounds__(kThreads) void gemm_rows_kernel(GemmArgs g) {
  constexpr int kSums = T * T * 256, kStep = 2 * T * 256;  // floats: a wave's sums, and its operands of one step
  __shared__ __attribute__((aligned(16))) float sums[kWaves][kSums > kStep ? kSums : kStep];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int gm = (g.M + 16 * T - 1) / (16 * T);
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int m0 = id % gm * (16 * T), n0 = id / gm * (16 * T);
  const int kbytes = g.K >> 1, kblocks = g.K >> 5, steps = (kblocks + 3) >> 2;
  const int lrow = lane >> 2, lblk = lane & 3;  // loaded: row and block of the step; multiplied: lane % 16, lane / 16

  // rows past the end read the last row; their results are not stored
  const uint8_t* codes[2 * T];
  const uint8_t* scales[2 * T];
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int64_t m = min(m0 + 16 * i + lrow, g.M - 1), n = min(n0 + 16 * i + lrow, g.N - 1);
    codes[i] = g.a_codes + m * kbytes + 16 * lblk;
    scales[i] = g.a_scales + m * kblocks + lblk;
    codes[T + i] = g.b_codes + n * kbytes + 16 * lblk;
    scales[T + i] = g.b_scales + n * kblocks + lblk;
  }
  // 16-byte pieces of a row swizzled, so that eight rows' pieces of one block fall on distinct banks
  i32x4* mine = reinterpret_cast<i32x4*>(sums[wv]);
  const int put = 4 * lrow + (lblk ^ ((lrow >> 1) & 3));
  const int get = 4 * (lane & 15) + ((lane >> 4) ^ ((lane >> 1) & 3));
  f32x4 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  for (int s0 = wv; s0 < steps; s0 += kWaves * kAhead) {
    i32x4 in[kAhead][2 * T];
    unsigned byte[kAhead][2 * T];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int s = s0 + k * kWaves;
      const bool there = 4 * s + lblk < kblocks;  // blocks past K: zero codes
#pragma unroll
      for (int i = 0; i < 2 * T; ++i) {
        in[k][i] = i32x4{0, 0, 0, 0};
        byte[k][i] = 127;
        if (there) {
          in[k][i] = *reinterpret_cast<const i32x4*>(codes[i] + 64 * (int64_t)s);
          byte[k][i] = scales[i][4 * s];
        }
      }
    }
    int sc[2 * T];
#pragma unroll
    for (int i = 0; i < 2 * T; ++i)
      sc[i] = __shfl((int)(byte[0][i] | (byte[1][i] << 8) | (byte[2][i] << 16) | (byte[3][i] << 24)),
                     4 * (lane & 15) + (lane >> 4));
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (s0 + k * kWaves < steps) {
        i32x4 op[2 * T];
#pragma unroll
        for (int i = 0; i < 2 * T; ++i) mine[64 * i + put] = in[k][i];
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < 2 * T; ++i) op[i] = mine[64 * i + get];
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
          for (int j = 0; j < T; ++j) {
            f32x4& d = acc[i][j];
            const i32x4 a = op[i], b = op[T + j];
            const int sa = sc[i], sb = sc[T + j];
            d = k == 0 ? multiply<0>(a, sa, b, sb, d)
                : k == 1 ? multiply<1>(a, sa, b, sb, d)
                : k == 2 ? multiply<2>(a, sa, b, sb, d)
                         : multiply<3>(a, sa, b, sb, d);
          }
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
