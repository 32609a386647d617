// The residual stream between two blocks: a block's output, normalised and
// gated, added to the stream, and the next block's norm and modulation of it.
//
// Mathematics.  Per row, with N the RMS or layer norm or nothing,
//   u  = N_post(y) post_w gate[s],   x' = bf16(a x + u),
//   h  = N_pre(x') pre_w (1 + scale[s]) + shift[s],
// every factor optional; out come x', bf16(h), the MXFP4 of bf16(h), or the
// (mean, 1 / deviation) of x' that kq_quantize_adaln reads.  Sums and the
// arithmetic up to each rounding are fp64.  sum (x - mean)^2 is taken as
// sum x^2 - mean sum x where that keeps 2^-40, else in a second pass.
//
// Layout.  A row's 16-byte pieces are spread over the lanes of one wave (no
// barrier) or of a workgroup's four, and stay in registers between the passes;
// each row of x and y is read once.  Four adjacent lanes hold a block of 32.
// Rows past what registers hold are read again from memory.
#include "kq_device.hpp"
#include "kq_internal.h"
#include "kq_mxval.hpp"
#include "kq_round.hpp"

namespace kq {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// Sums of a and b over the WPR waves of a row.
template <int WPR>
__device__ __forceinline__ void row_sums(double& a, double& b, double* red) {
  a = group_sum<6>(a);
  b = group_sum<6>(b);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // red may still be read
    if ((threadIdx.x & 63) == 0) {
      red[w] = a;
      red[kWaves + w] = b;
    }
    __syncthreads();
    a = b = 0.0;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      a += red[i];
      b += red[kWaves + i];
    }
  }
}

__device__ __forceinline__ void add_moments(u32x4 v, double& s, double& q) {
  double x[8];
  piece_values(v, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s += x[j];
    q = fma(x[j], x[j], q);
  }
}

// f[j] *= (v[j] + plus) for 8 channels of a vector, where there is one.
__device__ __forceinline__ void times(double f[8], const float* v, int64_t at, double plus) {
  if (v) {  // uniform
    const f32x4* p = reinterpret_cast<const f32x4*>(v + at);
    const f32x4 lo = p[0], hi = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] *= (double)lo[j] + plus;
      f[4 + j] *= (double)hi[j] + plus;
    }
  }
}

// The piece of x' at channel `ch` of a row of sample s: a x + (y - mean) rstd post_w gate.
__device__ __forceinline__ u32x4 add_block(const NormArgs& a, u32x4 x, u32x4 y, double mean, double rstd, int64_t sample,
                                           int ch) {
  double xs[8], u[8];
  piece_values(x, xs);
  piece_values(y, u);
  if (a.post != 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = (u[j] - mean) * rstd;
  }
  times(u, a.post_w, ch, 0.0);
  times(u, a.gate, sample * a.d + ch, 0.0);
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = fma(xs[j], a.residual_scale, u[j]);
  return round_piece(u);
}

// The piece of h, stored as rows and as codes.
__device__ __forceinline__ void store_next(const NormArgs& a, u32x4 x, double mean, double rstd, int64_t row,
                                           int64_t sample, int ch) {
  double h[8];
  piece_values(x, h);
  if (a.pre != 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = (h[j] - mean) * rstd;
  }
  times(h, a.pre_w, ch, 0.0);
  times(h, a.mod_scale, sample * a.d + ch, 1.0);
  if (a.mod_shift) {
    const f32x4* p = reinterpret_cast<const f32x4*>(a.mod_shift + sample * a.d + ch);
    const f32x4 lo = p[0], hi = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] += (double)lo[j];
      h[4 + j] += (double)hi[j];
    }
  }
  const u32x4 v = round_piece(h);
  if (a.h) *reinterpret_cast<u32x4*>(a.h + row * a.h_stride + ch) = v;
  if (a.codes) {
    unsigned word, byte;
    quantize_piece(v, word, byte);
    *reinterpret_cast<unsigned*>(a.codes + row * (a.d >> 1) + (ch >> 1)) = word;
    if ((ch & 31) == 0) a.scales[row * (a.d >> 5) + (ch >> 5)] = (uint8_t)byte;
  }
}

// WPR waves of a row (1, or the workgroup's four), MAXP pieces a lane in registers (0: from memory).
template <int WPR, int MAXP>
__global__ __launch_bounds__(kThreads) void residual_norm_kernel(NormArgs a) {
  __shared__ double red[2 * kWaves];
  constexpr int kLanes = 64 * WPR, kRows = kWaves / WPR;
  const int lane = threadIdx.x % kLanes;
  const int own = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kLanes));
  const int pieces = a.d >> 3;
  const double inv_d = 1.0 / a.d;

  for (int64_t row = (int64_t)blockIdx.x * kRows + own; row < a.tokens; row += (int64_t)gridDim.x * kRows) {
    const int64_t sample = fast_div((unsigned)row, a.by_sample);
    const uint16_t* const x = a.x + row * a.x_stride;
    const uint16_t* const y = a.y ? a.y + row * a.y_stride : nullptr;
    uint16_t* const out = a.x_out + row * a.x_out_stride;
    double mean = 0.0, rstd = 1.0;

    // mean and 1 / deviation from the sums of a row and, where those cancel, of its pieces again
    auto settle = [&](int norm, double s, double q, auto&& again) {
      row_sums<WPR>(s, q, red);
      mean = norm == 2 ? s * inv_d : 0.0;
      double m2 = norm == 2 ? q - s * mean : q;  // s of an infinite row may be NaN
      if (norm == 2 && m2 * 0x1p12 < q) {  // uniform over the row
        double far = 0.0, none = 0.0;
        again([&](u32x4 v) {
          double z[8];
          piece_values(v, z);
#pragma unroll
          for (int j = 0; j < 8; ++j) far = fma(z[j] - mean, z[j] - mean, far);
        });
        row_sums<WPR>(far, none, red);
        m2 = far;
      }
      rstd = 1.0 / sqrt(m2 * inv_d + a.eps);
    };

    if constexpr (MAXP > 0) {
      u32x4 xr[MAXP], yr[MAXP];
#pragma unroll
      for (int k = 0; k < MAXP; ++k) {
        const int p = lane + kLanes * k;
        xr[k] = yr[k] = u32x4{0, 0, 0, 0};
        if (p < pieces) {
          xr[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x) + p);
          if (y) yr[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(y) + p);
        }
      }
      auto pieces_of = [&](const u32x4* v) {
        return [=](auto&& use) {
#pragma unroll
          for (int k = 0; k < MAXP; ++k)
            if (lane + kLanes * k < pieces) use(v[k]);
        };
      };
      double s = 0.0, q = 0.0;
      if (y) {
        if (a.post) {
#pragma unroll
          for (int k = 0; k < MAXP; ++k) add_moments(yr[k], s, q);
          settle(a.post, s, q, pieces_of(yr));
        }
#pragma unroll
        for (int k = 0; k < MAXP; ++k) {
          const int p = lane + kLanes * k;
          if (p < pieces) {
            xr[k] = add_block(a, xr[k], yr[k], mean, rstd, sample, 8 * p);
            *(reinterpret_cast<u32x4*>(out) + p) = xr[k];
          }
        }
      }
      if (!a.next) continue;
      if (a.pre) {
        s = q = 0.0;
#pragma unroll
        for (int k = 0; k < MAXP; ++k) add_moments(xr[k], s, q);
        settle(a.pre, s, q, pieces_of(xr));
      }
      if (a.h || a.codes) {
#pragma unroll
        for (int k = 0; k < MAXP; ++k) {
          const int p = lane + kLanes * k;
          if (p < pieces) store_next(a, xr[k], mean, rstd, row, sample, 8 * p);
        }
      }
    } else {
      auto pieces_of = [&](const uint16_t* v) {
        return [=](auto&& use) {
          for (int p = lane; p < pieces; p += kLanes) use(*(reinterpret_cast<const u32x4*>(v) + p));
        };
      };
      double s = 0.0, q = 0.0;
      auto moments = [&](u32x4 v) { add_moments(v, s, q); };
      const uint16_t* next = x;
      if (y) {
        if (a.post) {
          pieces_of(y)(moments);
          settle(a.post, s, q, pieces_of(y));
          s = q = 0.0;
        }
        for (int p = lane; p < pieces; p += kLanes) {
          const u32x4 v = add_block(a, *(reinterpret_cast<const u32x4*>(x) + p), *(reinterpret_cast<const u32x4*>(y) + p),
                                    mean, rstd, sample, 8 * p);
          *(reinterpret_cast<u32x4*>(out) + p) = v;
          moments(v);
        }
        next = out;  // each lane reads back the pieces that it wrote
      }
      if (!a.next) continue;
      if (a.pre) {
        if (!y) pieces_of(next)(moments);
        settle(a.pre, s, q, pieces_of(next));
      }
      if (a.h || a.codes)
        for (int p = lane; p < pieces; p += kLanes)
          store_next(a, *(reinterpret_cast<const u32x4*>(next) + p), mean, rstd, row, sample, 8 * p);
    }
    if (a.stats && lane == 0) {
      a.stats[2 * row] = (float)mean;
      a.stats[2 * row + 1] = (float)rstd;
    }
  }
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& args, hipStream_t stream) {
  NormArgs a = args;
  const int pieces = a.d / 8;
  const void* fn;
  int rows = kWaves;  // of a workgroup
  if (pieces <= 64 * 2) {
    fn = (const void*)&residual_norm_kernel<1, 2>;
  } else if (pieces <= 64 * 3) {
    fn = (const void*)&residual_norm_kernel<1, 3>;
  } else if (pieces <= 64 * 5) {
    fn = (const void*)&residual_norm_kernel<1, 5>;
  } else {
    rows = 1;
    if (pieces <= kThreads * 3) fn = (const void*)&residual_norm_kernel<kWaves, 3>;
    else if (pieces <= kThreads * 6) fn = (const void*)&residual_norm_kernel<kWaves, 6>;
    else if (pieces <= kThreads * 8) fn = (const void*)&residual_norm_kernel<kWaves, 8>;
    else fn = (const void*)&residual_norm_kernel<kWaves, 0>;
  }
  const int64_t slots = (int64_t)cu_count() * resident_per_cu(fn, kThreads);
  const int64_t need = (a.tokens + rows - 1) / rows;
  void* kargs[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)(need < slots ? need : slots)), dim3(kThreads), kargs, 0, stream);
}

}  // namespace kq
