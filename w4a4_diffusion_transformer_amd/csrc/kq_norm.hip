// The residual stream between two blocks: a block's output, normalised and
// gated, added to the stream, and the next block's norm and modulation of it.
//
// Mathematics.  Per row, with N the RMS or layer norm or nothing,
//   u  = N_post(y) post_w gate[s],   x' = bf16(a x + u),
//   h  = N_pre(x') pre_w (1 + scale[s]) + shift[s],
// every factor optional; out come x', bf16(h), the MXFP4 of bf16(h), or the
// (mean, 1 / deviation) of x' that kq_quantize_adaln reads.  Sums and the
// arithmetic up to each rounding are fp64: a norm is fma(x, rstd, -mean rstd)
// and the vectors are folded into one factor before x' and a factor and a term
// after it.  sum (x - mean)^2 is taken as sum x^2 - mean sum x where that
// keeps 2^-40, else in a second pass.
//
// Layout.  A lane holds 16-byte pieces of a row; four adjacent lanes hold a
// block of 32.  Three kernels:
//   rows   a row to a wave (several narrow rows to one), up to 6 pieces a lane;
//          the folded vectors of the sample lie in LDS for all waves of the
//          workgroup, and nothing but a change of the sample needs a barrier;
//   wide   a row to a workgroup, one or two pieces a lane, the folded vectors in
//          its registers, the next row's loads in flight; for rows too wide for
//          a wave, for few rows, and for samples of few rows;
//   long   a row to a workgroup, read from memory again for each step.
// In the first two each row of x and y is read once.
#include "kq_device.hpp"
#include "kq_internal.h"
#include "kq_mxval.hpp"
#include "kq_round.hpp"

namespace kq {

namespace {

typedef __attribute__((ext_vector_type(2))) double f64x2;

constexpr int kMaxWaves = 16;
constexpr int kLong = 1024;  // threads of a workgroup whose rows stay in memory

// A row, or a vector of a sample, by pieces.  UNIFORM: the same one for the whole wave, a buffer of its own: its
// address stays in scalar registers, pieces past its end read as zero and are not written.  Else each lane has its
// own, `there` or not.
template <bool UNIFORM>
struct Row {
  __amdgpu_buffer_rsrc_t r;
  __device__ Row(const void* base, int64_t bytes, bool) : r(rsrc_uniform(base, bytes)) {}
  __device__ u32x4 load(int p) const { return __builtin_amdgcn_raw_buffer_load_b128(r, 16 * p, 0, kNT); }
  __device__ void store(int p, u32x4 v) const { __builtin_amdgcn_raw_buffer_store_b128(v, r, 16 * p, 0, 0); }
  __device__ void store_codes(int p, unsigned w) const { __builtin_amdgcn_raw_buffer_store_b32(w, r, 4 * p, 0, 0); }
  __device__ void store_scale(int p, unsigned b) const {
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)b, r, p & 3 ? (int)kOut : p >> 2, 0, 0);
  }
};

template <>
struct Row<false> {
  uint8_t* base;
  int64_t bytes;  // 0: not there
  __device__ Row(const void* b, int64_t n, bool there) : base((uint8_t*)b), bytes(there ? n : 0) {}
  __device__ u32x4 load(int p) const {
    u32x4 v{0, 0, 0, 0};
    if (16 * p < bytes) v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base + 16 * p));
    return v;
  }
  __device__ void store(int p, u32x4 v) const {
    if (16 * p < bytes) *reinterpret_cast<u32x4*>(base + 16 * p) = v;
  }
  __device__ void store_codes(int p, unsigned w) const {
    if (4 * p < bytes) *reinterpret_cast<unsigned*>(base + 4 * p) = w;
  }
  __device__ void store_scale(int p, unsigned b) const {
    if ((p & 3) == 0 && p >> 2 < bytes) base[p >> 2] = (uint8_t)b;
  }
};

__device__ __forceinline__ void add_moments(const double x[8], double& s, double& q) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s += x[j];
    q = fma(x[j], x[j], q);
  }
}

// The five vectors at a piece (8 channels) of sample s; all their loads go out before the first is used.
struct Vectors {
  f32x4 post_w[2], gate[2], pre_w[2], scale[2], shift[2];
};

__device__ __forceinline__ void load_vector(const float* v, int d, int p, float missing, f32x4 out[2]) {
  out[0] = out[1] = f32x4{missing, missing, missing, missing};
  if (v) {  // uniform
    const auto r = rsrc_uniform(v, (int64_t)d * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      out[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 32 * p + 16 * i, 0, 0));
  }
}

// The row of sample s in a vector of samples.
__device__ __forceinline__ const float* of_sample(const NormArgs& a, const float* v, int64_t s) {
  return v ? v + s * a.d : nullptr;
}

__device__ __forceinline__ void load_block_vectors(const NormArgs& a, int64_t s, int p, Vectors& v) {
  load_vector(a.post_w, a.d, p, 1.0f, v.post_w);
  load_vector(of_sample(a, a.gate, s), a.d, p, 1.0f, v.gate);
}

__device__ __forceinline__ void load_next_vectors(const NormArgs& a, int64_t s, int p, Vectors& v) {
  load_vector(a.pre_w, a.d, p, 1.0f, v.pre_w);
  load_vector(of_sample(a, a.mod_scale, s), a.d, p, 0.0f, v.scale);
  load_vector(of_sample(a, a.mod_shift, s), a.d, p, -0.0f, v.shift);  // leaves a zero its sign
}

// The factor of a block's output; the factor and the term of the next block's input.
__device__ __forceinline__ void block_factor(const Vectors& v, double f[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (double)v.post_w[j >> 2][j & 3] * (double)v.gate[j >> 2][j & 3];
}

__device__ __forceinline__ void next_factor(const Vectors& v, double f[8], double t[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = (double)v.pre_w[j >> 2][j & 3] * ((double)v.scale[j >> 2][j & 3] + 1.0);
    t[j] = (double)v.shift[j >> 2][j & 3];
  }
}

// A row's norm: n = fma(x, rstd, shift).
struct Norm {
  double mean = 0.0, rstd = 1.0, shift = -0.0;
};

__device__ __forceinline__ u32x4 add_block(const NormArgs& a, u32x4 x, u32x4 y, const Norm& n, const double f[8]) {
  double xs[8], u[8];
  piece_values(x, xs);
  piece_values(y, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = fma(fma(u[j], n.rstd, n.shift), f[j], xs[j] * a.residual_scale);
  return round_piece(u);
}

template <bool UNIFORM>
__device__ __forceinline__ void store_next(const NormArgs& a, u32x4 x, const Norm& n, const double f[8], const double t[8],
                                           int64_t row, int p, bool there) {
  double h[8];
  piece_values(x, h);
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = fma(fma(h[j], n.rstd, n.shift), f[j], t[j]);
  const u32x4 v = round_piece(h);
  if (a.h) Row<UNIFORM>(a.h + row * a.h_stride, 2 * a.d, there).store(p, v);
  if (a.codes) {
    unsigned word, byte;
    quantize_piece(v, word, byte);
    Row<UNIFORM>(a.codes + row * (a.d >> 1), a.d >> 1, there).store_codes(p, word);
    Row<UNIFORM>(a.scales + row * (a.d >> 5), a.d >> 5, there).store_scale(p, byte);
  }
}

// Sums of (s, q) over a row of 2^LOG lanes.
template <int LOG>
struct WaveSum {
  __device__ __forceinline__ void operator()(double& s, double& q) {
    const double v = group_sums<LOG>(s, q);
    if constexpr (LOG == 6) {
      s = from_first<0>(v);
      q = from_first<1>(v);
    } else {
      const double other = from_dpp<DPP_XOR1>(v);
      const bool odd = threadIdx.x & 1;
      s = odd ? other : v;
      q = odd ? v : other;
    }
  }
  template <int LANE>
  static __device__ __forceinline__ double from_first(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)b, LANE);
    const uint64_t hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(b >> 32), LANE);
    return __builtin_bit_cast(double, hi << 32 | lo);
  }
};

// The same over the waves of a workgroup, through LDS; two buffers in turn, so that one barrier parts a sum's writes
// from its reads and its reads from the next writes.
struct WorkgroupSum {
  double (*red)[2 * kMaxWaves];
  int waves, turn = 0;
  __device__ __forceinline__ void operator()(double& s, double& q) {
    const double v = group_sums<6>(s, q);
    const unsigned lane = threadIdx.x & 63;
    if (lane < 2) red[turn][2 * (threadIdx.x >> 6) + lane] = v;
    __syncthreads();
    s = q = 0.0;
#pragma unroll 1
    for (int i = 0; i < waves; ++i) {
      s += red[turn][2 * i];
      q += red[turn][2 * i + 1];
    }
    turn ^= 1;
  }
};

// The norm of a row from its sums; `again` calls its argument on each of this lane's pieces.
template <class Sum, class Again>
__device__ __forceinline__ Norm settle(const NormArgs& a, int kind, double s, double q, Sum& sum, Again&& again) {
  Norm n;
  sum(s, q);
  n.mean = kind == 2 ? s * a.inv_d : 0.0;
  double m2 = kind == 2 ? q - s * n.mean : q;  // s of an infinite row may be NaN
  const bool cancels = kind == 2 && m2 * 0x1p12 < q;
  // the whole wave (and, as sums are equal in all of them, the workgroup) if any row of it
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(cancels) != 0, 0)) {
    double far = 0.0, none = 0.0;
    again([&](u32x4 v) {
      double z[8];
      piece_values(v, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) far = fma(z[j] - n.mean, z[j] - n.mean, far);
    });
    sum(far, none);
    m2 = cancels ? far : m2;
  }
  n.rstd = inverse_sqrt(fma(m2, a.inv_d, a.eps));
  n.shift = kind == 2 ? -n.mean * n.rstd : -0.0;
  return n;
}

// A row of 2^LOG lanes with P pieces each (P > 1: LOG = 6).
template <int LOG, int P, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void rows_kernel(NormArgs a) {
  constexpr int kLanes = 1 << LOG, kRows = 64 >> LOG, kPieces = kLanes * P;
  constexpr bool UNIFORM = LOG == 6;
  // the folded vectors, two channels of each piece at a time: lanes read whole lines
  __shared__ f64x2 vectors[3][4][kPieces];
  const int pieces = a.d >> 3;
  const int lane = threadIdx.x & (kLanes - 1), sub = (int)(threadIdx.x & 63) >> LOG;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t row0 = (int64_t)blockIdx.x * a.group_rows;
  const int64_t row1 = row0 + a.group_rows < a.tokens ? row0 + a.group_rows : a.tokens;
  auto vector = [&](int which, int p, double f[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f64x2 v = vectors[which][j][p];
      f[2 * j] = v[0];
      f[2 * j + 1] = v[1];
    }
  };
  auto again = [](u32x4* v) {  // an empty asm: values are converted again rather than held over the sums
#pragma unroll
    for (int k = 0; k < P; ++k) asm volatile("" : "+v"(v[k]));
  };
  WaveSum<LOG> sum;
  for (int64_t first = row0; first < row1;) {
    const int64_t sample = fast_div((unsigned)first, a.by_sample);
    const int64_t end = (sample + 1) * a.sample_rows < row1 ? (sample + 1) * a.sample_rows : row1;
    if (first > row0) __syncthreads();
    for (int p = threadIdx.x; p < pieces; p += THREADS) {
      Vectors v;
      load_block_vectors(a, sample, p, v);
      load_next_vectors(a, sample, p, v);
      double f[3][8];
      block_factor(v, f[0]);
      next_factor(v, f[1], f[2]);
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) vectors[i][j][p] = f64x2{f[i][2 * j], f[i][2 * j + 1]};
    }
    __syncthreads();
    for (int64_t at = first + wave * kRows; at < end; at += THREADS / 64 * kRows) {
      const bool there = at + sub < end;
      const int64_t row = there ? at + sub : end - 1;
      u32x4 x[P], y[P];
      const Row<UNIFORM> xs(a.x + row * a.x_stride, 2 * a.d, true);
#pragma unroll
      for (int k = 0; k < P; ++k) x[k] = xs.load(lane + kLanes * k);
      if (a.y) {
        const Row<UNIFORM> ys(a.y + row * a.y_stride, 2 * a.d, true);
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = ys.load(lane + kLanes * k);
      }
      auto moments = [&](const u32x4* v, double& s, double& q) {
        s = q = 0.0;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          double z[8];
          piece_values(v[k], z);
          add_moments(z, s, q);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      auto pieces_of = [&](const u32x4* v) {
        return [=](auto&& use) {
#pragma unroll
          for (int k = 0; k < P; ++k)
            if (lane + kLanes * k < pieces) use(v[k]);
        };
      };
      Norm n;
      double s = 0.0, q = 0.0;
      if (a.y) {
        if (a.post) {
          moments(y, s, q);
          again(y);
          n = settle(a, a.post, s, q, sum, pieces_of(y));
          again(y);
        }
        const Row<UNIFORM> out(a.x_out + row * a.x_out_stride, 2 * a.d, there);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const int p = lane + kLanes * k;
          double f[8];
          vector(0, p, f);
          x[k] = add_block(a, x[k], y[k], n, f);
          out.store(p, x[k]);
          if (p >= pieces) x[k] = u32x4{0, 0, 0, 0};
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (!a.next) continue;
      n = Norm{};
      if (a.pre) {
        moments(x, s, q);
        again(x);
        n = settle(a, a.pre, s, q, sum, pieces_of(x));
        again(x);
      }
      if (a.h || a.codes) {
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const int p = lane + kLanes * k;
          double f[8], t[8];
          vector(1, p, f);
          vector(2, p, t);
          store_next<UNIFORM>(a, x[k], n, f, t, row, p, there);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (a.stats && lane == 0 && there) {
        a.stats[2 * row] = (float)n.mean;
        a.stats[2 * row + 1] = (float)n.rstd;
      }
    }
    first = end;
  }
}

// A row to a workgroup, P pieces a lane; KEEP: the folded vectors stay in registers.
template <int P, bool KEEP, int THREADS>
__global__ __launch_bounds__(THREADS) void wide_kernel(NormArgs a) {
  __shared__ double red[2][2 * kMaxWaves];
  const int lane = threadIdx.x, lanes = blockDim.x;
  const int64_t row0 = (int64_t)blockIdx.x * a.group_rows;
  const int64_t row1 = row0 + a.group_rows < a.tokens ? row0 + a.group_rows : a.tokens;
  const int pieces = a.d >> 3;
  WorkgroupSum sum{red, lanes >> 6};

  u32x4 nx[P], ny[P];
  auto load = [&](int64_t row) {
    const Row<true> xs(a.x + row * a.x_stride, 2 * a.d, true);
#pragma unroll
    for (int k = 0; k < P; ++k) nx[k] = xs.load(lane + lanes * k);
    if (a.y) {
      const Row<true> ys(a.y + row * a.y_stride, 2 * a.d, true);
#pragma unroll
      for (int k = 0; k < P; ++k) ny[k] = ys.load(lane + lanes * k);
    }
  };
  auto again = [](u32x4* v) {
#pragma unroll
    for (int k = 0; k < P; ++k) asm volatile("" : "+v"(v[k]));
  };
  double f[KEEP ? P : 1][8], nf[KEEP ? P : 1][8], nt[KEEP ? P : 1][8];
  int64_t sample_of_vectors = -1;
  if (row0 < row1) load(row0);
  for (int64_t row = row0; row < row1; ++row) {
    const int64_t sample = fast_div((unsigned)row, a.by_sample);
    if (KEEP && sample != sample_of_vectors) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int p = lane + lanes * k;
        Vectors v;
        load_block_vectors(a, sample, p, v);
        load_next_vectors(a, sample, p, v);
        block_factor(v, f[k]);
        next_factor(v, nf[k], nt[k]);
      }
      sample_of_vectors = sample;
    }
    u32x4 x[P], y[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      x[k] = nx[k];
      y[k] = ny[k];
    }
    if (row + 1 < row1) load(row + 1);
    auto moments = [&](const u32x4* v, double& s, double& q) {
      s = q = 0.0;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        double z[8];
        piece_values(v[k], z);
        add_moments(z, s, q);
      }
    };
    auto pieces_of = [&](const u32x4* v) {
      return [=](auto&& use) {
#pragma unroll
        for (int k = 0; k < P; ++k)
          if (lane + lanes * k < pieces) use(v[k]);
      };
    };
    Norm n;
    double s, q;
    if (a.y) {
      if (a.post) {
        moments(y, s, q);
        again(y);
        n = settle(a, a.post, s, q, sum, pieces_of(y));
        again(y);
      }
      const Row<true> out(a.x_out + row * a.x_out_stride, 2 * a.d, true);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int p = lane + lanes * k;
        if (!KEEP) {
          Vectors v;
          load_block_vectors(a, sample, p, v);
          block_factor(v, f[0]);
        }
        x[k] = add_block(a, x[k], y[k], n, f[KEEP ? k : 0]);
        out.store(p, x[k]);
        if (p >= pieces) x[k] = u32x4{0, 0, 0, 0};
      }
    }
    if (!a.next) continue;
    n = Norm{};
    if (a.pre) {
      moments(x, s, q);
      again(x);
      n = settle(a, a.pre, s, q, sum, pieces_of(x));
      again(x);
    }
    if (a.h || a.codes) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int p = lane + lanes * k;
        if (!KEEP) {
          Vectors v;
          load_next_vectors(a, sample, p, v);
          next_factor(v, nf[0], nt[0]);
        }
        store_next<true>(a, x[k], n, nf[KEEP ? k : 0], nt[KEEP ? k : 0], row, p, true);
      }
    }
    if (a.stats && lane == 0) {
      a.stats[2 * row] = (float)n.mean;
      a.stats[2 * row + 1] = (float)n.rstd;
    }
  }
}

// Rows of any length: a workgroup each, read again for each step.
__global__ __launch_bounds__(kLong) void long_rows_kernel(NormArgs a) {
  __shared__ double red[2][2 * kMaxWaves];
  const int pieces = a.d >> 3;
  WorkgroupSum sum{red, kLong / 64};
  for (int64_t row = blockIdx.x; row < a.tokens; row += gridDim.x) {
    const int64_t sample = fast_div((unsigned)row, a.by_sample);
    auto each = [&](const uint16_t* v, int64_t stride) {
      const u32x4* const p = reinterpret_cast<const u32x4*>(v + row * stride);
      return [=](auto&& use) {
        for (int i = threadIdx.x; i < pieces; i += kLong) use(p[i]);
      };
    };
    double s = 0.0, q = 0.0;
    auto moments = [&](u32x4 v) {
      double z[8];
      piece_values(v, z);
      add_moments(z, s, q);
    };
    Norm n;
    const uint16_t* stream = a.x;
    int64_t stride = a.x_stride;
    if (a.y) {
      if (a.post) {
        each(a.y, a.y_stride)(moments);
        n = settle(a, a.post, s, q, sum, each(a.y, a.y_stride));
        s = q = 0.0;
      }
      const u32x4* const x = reinterpret_cast<const u32x4*>(a.x + row * a.x_stride);
      const u32x4* const y = reinterpret_cast<const u32x4*>(a.y + row * a.y_stride);
      for (int i = threadIdx.x; i < pieces; i += kLong) {
        Vectors w;
        load_block_vectors(a, sample, i, w);
        double f[8];
        block_factor(w, f);
        const u32x4 v = add_block(a, x[i], y[i], n, f);
        *(reinterpret_cast<u32x4*>(a.x_out + row * a.x_out_stride) + i) = v;
        moments(v);
      }
      stream = a.x_out;  // each lane reads back the pieces that it wrote
      stride = a.x_out_stride;
    }
    if (!a.next) continue;
    n = Norm{};
    if (a.pre) {
      if (!a.y) each(stream, stride)(moments);
      n = settle(a, a.pre, s, q, sum, each(stream, stride));
    }
    if (a.h || a.codes) {
      for (int i = threadIdx.x; i < pieces; i += kLong) {
        Vectors w;
        load_next_vectors(a, sample, i, w);
        double f[8], t[8];
        next_factor(w, f, t);
        store_next<true>(a, *(reinterpret_cast<const u32x4*>(stream + row * stride) + i), n, f, t, row, i, true);
      }
    }
    if (a.stats && threadIdx.x == 0) {
      a.stats[2 * row] = (float)n.mean;
      a.stats[2 * row + 1] = (float)n.rstd;
    }
  }
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& args, hipStream_t stream) {
  NormArgs a = args;
  a.inv_d = 1.0 / a.d;
  const int64_t pieces = a.d / 8, cus = cu_count();
  void* kargs[] = {&a};
  if (pieces > 128 * kMaxWaves) {
    const int64_t slots = 2 * cus;
    return hipLaunchKernel((const void*)&long_rows_kernel, dim3((unsigned)(a.tokens < slots ? a.tokens : slots)),
                           dim3(kLong), kargs, 0, stream);
  }
  const void* fn;
  int threads;
  int64_t rows, slots;  // rows of a step of a workgroup; workgroups that run at once
  if (pieces <= 64 || (pieces <= 384 && a.tokens > 4 * cus && a.sample_rows >= 64)) {
    static const void* const narrow[] = {(const void*)&rows_kernel<2, 1, 512>, (const void*)&rows_kernel<3, 1, 512>,
                                         (const void*)&rows_kernel<4, 1, 512>, (const void*)&rows_kernel<5, 1, 512>};
    static const void* const whole[] = {(const void*)&rows_kernel<6, 1, 512>, (const void*)&rows_kernel<6, 2, 512>,
                                        (const void*)&rows_kernel<6, 3, 512>, (const void*)&rows_kernel<6, 4, 512>,
                                        (const void*)&rows_kernel<6, 5, 512>, (const void*)&rows_kernel<6, 6, 512>};
    int log = 2;
    while (log < 6 && (1 << log) < pieces) ++log;
    const int64_t per = (pieces + 63) / 64;
    fn = log < 6 ? narrow[log - 2] : whole[per - 1];
    threads = 512;
    rows = threads >> log;
    slots = cus * resident_per_cu(fn, threads);
  } else {
    const int64_t per = pieces <= 64 * kMaxWaves ? 1 : 2;
    const int64_t waves = (pieces + 64 * per - 1) / (64 * per);
    threads = (int)(64 * waves);
    fn = per == 1         ? (const void*)&wide_kernel<1, true, 1024>
         : threads <= 768 ? (const void*)&wide_kernel<2, true, 768>
                          : (const void*)&wide_kernel<2, false, 1024>;
    rows = 1;
    // workgroups are dealt to the four SIMDs of a compute unit from the first on: 5 waves take the room of 8
    const int64_t room = 16 / ((waves + 3) / 4 * 4);
    slots = cus * (room > 1 ? room : 1);
  }
  const int64_t steps = (a.tokens + rows - 1) / rows;
  a.group_rows = (steps + slots - 1) / slots * rows;
  const int64_t groups = (a.tokens + a.group_rows - 1) / a.group_rows;
  return hipLaunchKernel(fn, dim3((unsigned)groups), dim3(threads), kargs, 0, stream);
}

}  // namespace kq
