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
// keeps 2^-40, else in a second pass.  A channel that equals the mean has to
// come out as 0, or MXFP4 gives a block of them a scale and codes: the mean is
// the sum's correctly rounded quotient, and rstd keeps 45 bits, with which its
// product with a mean that is a bf16 value (8 bits) is exact.  (x - mean) rstd
// would do that too: 8192 x 1152 19.4 us for 19.0, 18432 x 2240 75.3 for 74.2.
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
//
// What bounds it, measured (kernel alone; a copy reaches 5.09 TB/s).  Many
// rows: memory.  18432 x 2240, RMS norms on both sides, gate, modulation, rows:
// 70 to 75 us, 4.4 to 4.7 TB/s.  Where each wave has one step, vectors, rows,
// sums and stores follow one another on all of the GPU at once: 8192 x 1152 to
// codes 19 us, of them 9 of instructions, and 12 without Y; 4097 x 2240 to
// statistics 14.5.  Wide rows, one workgroup a compute unit: 1009 x 12288 to codes
// 25 us, 15 of instructions and two barriers a row beside 16 of memory; 1009 x
// 24576, rows read again, 62 for 32 of memory.  Few rows (8 x 2240): the launch
// and one row's chain, 4.8 to 4.9 us.
//
// Cache policy.  What the next kernel reads is stored as usual: past the caches
// this one would end sooner, but with the reader behind it the two take longer
// (8192 x 1152 to codes, and the codes read: 25.3 us and 27.2).  The stream,
// where h or codes are what the next kernel reads, is not touched again before
// the block ends and passes the caches by (24.3; 1009 x 12288 35.6 and 32.6).
// Were it read next after all (two such norms in a row, 2240 channels): no
// difference from 8 to 256 rows (8.8 and 8.8, 9.4 and 9.4 us), 4096 rows 41.0 for
// 40.2, 18432 rows 136 for 127.
#include <algorithm>

#include "kq_device.hpp"
#include "kq_internal.h"
#include "kq_mxval.hpp"
#include "kq_round.hpp"

namespace kq {

namespace {

typedef __attribute__((ext_vector_type(2))) double f64x2;

// Which of h and codes a kernel writes.  Where the next row's loads are in flight it has to be known when compiling:
// with stores that may or may not be issued behind them, the wait for those loads is one for the stores too.
enum { OUT_ROWS = 1, OUT_CODES = 2, OUT_ANY = 4 };

constexpr int kMaxWaves = 16;
constexpr int kMaxPieces = 6;      // of a lane of the rows kernel
constexpr int kRowsThreads = 512;  // of its workgroups
constexpr int kLong = 1024;  // threads of a workgroup whose rows stay in memory

// A lane's place: its row of the wave's (LOG < 6) and its piece, and whether it has its pieces but the last, and the last.
struct Lane {
  int sub, piece;
  bool there, last;
};

// This lane's pieces of a wave's rows, P pieces `step` bytes apart: of one row, a buffer of its own (address in scalar
// registers, pieces past its end read as zero and are not written), or with LOG < 6 of row `sub` of several rows
// `stride` bytes apart in one buffer.
template <int LOG, int P>
struct Rows {
  __amdgpu_buffer_rsrc_t r;
  int main, last;
  // offset: of the lane's first piece in its row
  __device__ Rows(const void* base, int64_t stride, int64_t bytes, const Lane& l, int offset)
      : r(rsrc_uniform(base, bytes + (LOG < 6 ? ((64 >> LOG) - 1) * stride : 0))) {
    main = last = offset;
    if constexpr (LOG < 6) {
      constexpr int kPast = (int)0x80000000u;  // and any step from it lie past every buffer
      const int at = l.sub * (int)stride + offset;
      main = l.there ? at : kPast;
      last = l.last ? at : kPast;
    }
  }
  template <int STEP>
  __device__ int offset(int k) const { return (k == P - 1 ? last : main) + k * STEP * (1 << LOG); }
  __device__ u32x4 load(int k) const { return __builtin_amdgcn_raw_buffer_load_b128(r, offset<16>(k), 0, 0); }
  template <int POLICY>
  __device__ void store(int k, u32x4 v) const { __builtin_amdgcn_raw_buffer_store_b128(v, r, offset<16>(k), 0, POLICY); }
  __device__ void store_codes(int k, unsigned w) const {
    __builtin_amdgcn_raw_buffer_store_b32(w, r, offset<4>(k), 0, 0);
  }
  // four lanes have a scale: `first` of them writes it
  __device__ void store_scale(int k, unsigned b, bool first) const {
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)b, r, first ? (k == P - 1 ? last : main) + k * (1 << LOG) / 4 : (int)kOut,
                                         0, 0);
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

template <class T>
__device__ __forceinline__ void next_factor(const Vectors& v, double f[8], T t[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = (double)v.pre_w[j >> 2][j & 3] * ((double)v.scale[j >> 2][j & 3] + 1.0);
    t[j] = (T)v.shift[j >> 2][j & 3];
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

// Piece k of this lane of h, in rows from `first` on.
template <int LOG, int P, int OUT = OUT_ANY, class T>
__device__ __forceinline__ void store_next(const NormArgs& a, u32x4 x, const Norm& n, const double f[8], const T t[8],
                                           int64_t first, const Lane& l, int k) {
  double h[8];
  piece_values(x, h);
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = fma(fma(h[j], n.rstd, n.shift), f[j], (double)t[j]);
  const u32x4 v = round_piece(h);
  if (OUT == OUT_ANY ? a.h != nullptr : (OUT & OUT_ROWS) != 0)
    Rows<LOG, P>(a.h + first * a.h_stride, 2 * a.h_stride, 2 * a.d, l, 16 * l.piece).template store<0>(k, v);
  if (OUT == OUT_ANY ? a.codes != nullptr : (OUT & OUT_CODES) != 0) {
    unsigned word, byte;
    quantize_piece(v, word, byte);
    Rows<LOG, P>(a.codes + first * (a.d >> 1), a.d >> 1, a.d >> 1, l, 4 * l.piece).store_codes(k, word);
    Rows<LOG, P>(a.scales + first * (a.d >> 5), a.d >> 5, a.d >> 5, l, l.piece >> 2).store_scale(k, byte, (l.piece & 3) == 0);
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

// The same over the waves of a workgroup, through LDS: a wave's two sums go to two neighbouring words, and each wave
// adds up the words as lanes of its own.  Two buffers in turn, so that one barrier parts a sum's writes from its reads
// and its reads from the next writes.
struct WorkgroupSum {
  double (*red)[2 * kMaxWaves];
  int waves, turn = 0;
  __device__ __forceinline__ void operator()(double& s, double& q) {
    double v = group_sums<6>(s, q);
    const unsigned lane = threadIdx.x & 63;
    if (lane < 2) red[turn][2 * (threadIdx.x >> 6) + lane] = v;
    __syncthreads();
    v = 0.0;
    if (lane < 2 * (unsigned)waves) v = red[turn][lane];
    turn ^= 1;
    v += from_dpp<DPP_XOR2>(v);  // 32 words
    v += from_dpp<DPP_ROTATE4>(v);
    v += from_dpp<DPP_ROTATE8>(v);
    v = add_swap16(v);
    s = WaveSum<6>::from_first<0>(v);
    q = WaveSum<6>::from_first<1>(v);
  }
};

// The norm of a row from its sums; `again` calls its argument on each of this lane's pieces.
template <class Sum, class Again>
__device__ __forceinline__ Norm settle(const NormArgs& a, int kind, double s, double q, Sum& sum, Again&& again) {
  Norm n;
  sum(s, q);
  if (kind == 2) {
    // s / d, correctly rounded: the product with the rounded reciprocal, corrected by its exact remainder
    n.mean = s * a.inv_d;
    const double m = fma(fma(-n.mean, (double)a.d, s), a.inv_d, n.mean);
    n.mean = m == m ? m : n.mean;  // an infinite sum has no remainder
  }
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
  // less by 2^-44 of itself at most; mean rstd is exact where a channel can equal the mean
  n.rstd = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, n.rstd) & ~uint64_t(0xFF));
  n.shift = kind == 2 ? -n.mean * n.rstd : -0.0;
  return n;
}

// A row of 2^LOG lanes with P pieces each.
template <int LOG, int P, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void rows_kernel(NormArgs a) {
  constexpr int kLanes = 1 << LOG, kRows = 64 >> LOG, kPieces = kLanes * P;
  constexpr int kStep = THREADS / 64 * kRows;  // rows of the workgroup's waves
  // the folded vectors, two channels of each piece at a time: lanes read whole lines
  __shared__ f64x2 vectors[3][4][kPieces];
  const int pieces = a.d >> 3;
  const int lane = threadIdx.x & (kLanes - 1), sub = (int)(threadIdx.x & 63) >> LOG;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t row0 = (int64_t)blockIdx.x * a.group_rows;
  const int64_t row1 = row0 + a.group_rows < a.tokens ? row0 + a.group_rows : a.tokens;
  const bool last_there = lane + kLanes * (P - 1) < pieces;  // of a lane's pieces only the last may be past the row
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
    for (int64_t at = first + wave * kRows; at < end; at += kStep) {
      const Lane l{sub, lane, at + sub < end, at + sub < end && last_there};
      u32x4 x[P], y[P];
      const Rows<LOG, P> xs(a.x + at * a.x_stride, 2 * a.x_stride, 2 * a.d, l, 16 * lane);
#pragma unroll
      for (int k = 0; k < P; ++k) x[k] = xs.load(k);
      if (a.y) {
        const Rows<LOG, P> ys(a.y + at * a.y_stride, 2 * a.y_stride, 2 * a.d, l, 16 * lane);
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = ys.load(k);
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
            if (k < P - 1 || last_there) use(v[k]);
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
        const Rows<LOG, P> out(a.x_out + at * a.x_out_stride, 2 * a.x_out_stride, 2 * a.d, l, 16 * lane);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const int p = lane + kLanes * k;
          double f[8];
          vector(0, p, f);
          x[k] = add_block(a, x[k], y[k], n, f);
          if (a.h || a.codes) out.template store<kNT>(k, x[k]);  // uniform
          else out.template store<0>(k, x[k]);
          if (k == P - 1 && !last_there) x[k] = u32x4{0, 0, 0, 0};
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
          store_next<LOG, P>(a, x[k], n, f, t, at, l, k);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (a.stats && lane == 0 && at + sub < end) {
        a.stats[2 * (at + sub)] = (float)n.mean;
        a.stats[2 * (at + sub) + 1] = (float)n.rstd;
      }
    }
    first = end;
  }
}

// A row to a workgroup, P pieces a lane; KEEP: the folded vectors stay in registers.
// Y: there is a block's output; OUT: of h and codes, what is written.
template <int P, bool KEEP, int THREADS, bool Y, int OUT>
__global__ __launch_bounds__(THREADS) void wide_kernel(NormArgs a) {
  __shared__ double red[2][2 * kMaxWaves];
  const int lane = threadIdx.x, lanes = blockDim.x;
  const int64_t row0 = (int64_t)blockIdx.x * a.group_rows;
  const int64_t row1 = row0 + a.group_rows < a.tokens ? row0 + a.group_rows : a.tokens;
  const int pieces = a.d >> 3;
  WorkgroupSum sum{red, lanes >> 6};

  u32x4 nx[P], ny[P];
  auto load = [&](int64_t row) {
    auto piece = [&](const uint16_t* base, int k) {
      return Rows<6, 1>(base, 0, 2 * a.d, Lane{}, 16 * (lane + lanes * k)).load(0);
    };
#pragma unroll
    for (int k = 0; k < P; ++k) nx[k] = piece(a.x + row * a.x_stride, k);
    if constexpr (Y) {
#pragma unroll
      for (int k = 0; k < P; ++k) ny[k] = piece(a.y + row * a.y_stride, k);
    }
  };
  auto again = [](u32x4* v) {
#pragma unroll
    for (int k = 0; k < P; ++k) asm volatile("" : "+v"(v[k]));
  };
  double f[KEEP ? P : 1][8], nf[KEEP ? P : 1][8];
  float nt[KEEP ? P : 1][8];
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
    if constexpr (Y) {
      if (a.post) {
        moments(y, s, q);
        again(y);
        n = settle(a, a.post, s, q, sum, pieces_of(y));
        again(y);
      }
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int p = lane + lanes * k;
        if (!KEEP) {
          Vectors v;
          load_block_vectors(a, sample, p, v);
          block_factor(v, f[0]);
        }
        x[k] = add_block(a, x[k], y[k], n, f[KEEP ? k : 0]);
        Rows<6, 1>(a.x_out + row * a.x_out_stride, 0, 2 * a.d, Lane{}, 16 * p)
            .template store<OUT != 0 ? kNT : 0>(0, x[k]);
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
    if constexpr (OUT != 0) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int p = lane + lanes * k;
        if (!KEEP) {
          Vectors v;
          load_next_vectors(a, sample, p, v);
          next_factor(v, nf[0], nt[0]);
        }
        store_next<6, 1, OUT>(a, x[k], n, nf[KEEP ? k : 0], nt[KEEP ? k : 0], row, Lane{0, p}, 0);
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
        store_next<6, 1>(a, *(reinterpret_cast<const u32x4*>(stream + row * stride) + i), n, f, t, row, Lane{0, i}, 0);
      }
    }
    if (a.stats && threadIdx.x == 0) {
      a.stats[2 * row] = (float)n.mean;
      a.stats[2 * row + 1] = (float)n.rstd;
    }
  }
}

#define KQ_ROWS(LOG)                                                                                            \
  {(const void*)&rows_kernel<LOG, 1, kRowsThreads>, (const void*)&rows_kernel<LOG, 2, kRowsThreads>,            \
   (const void*)&rows_kernel<LOG, 3, kRowsThreads>, (const void*)&rows_kernel<LOG, 4, kRowsThreads>,            \
   (const void*)&rows_kernel<LOG, 5, kRowsThreads>, (const void*)&rows_kernel<LOG, 6, kRowsThreads>}
const void* const rows_kernels[5][kMaxPieces] = {KQ_ROWS(2), KQ_ROWS(3), KQ_ROWS(4), KQ_ROWS(5), KQ_ROWS(6)};
#undef KQ_ROWS
#define KQ_WIDE(P, KEEP, THREADS, Y)                                                                            \
  {(const void*)&wide_kernel<P, KEEP, THREADS, Y, 0>, (const void*)&wide_kernel<P, KEEP, THREADS, Y, OUT_ROWS>, \
   (const void*)&wide_kernel<P, KEEP, THREADS, Y, OUT_CODES>,                                                   \
   (const void*)&wide_kernel<P, KEEP, THREADS, Y, OUT_ROWS | OUT_CODES>}
const void* const wide_kernels[3][2][4] = {{KQ_WIDE(1, true, 1024, false), KQ_WIDE(1, true, 1024, true)},
                                           {KQ_WIDE(2, true, 768, false), KQ_WIDE(2, true, 768, true)},
                                           {KQ_WIDE(2, false, 1024, false), KQ_WIDE(2, false, 1024, true)}};
#undef KQ_WIDE

}  // namespace

hipError_t launch_residual_norm(const NormArgs& args, hipStream_t stream) {
  NormArgs a = args;
  a.inv_d = 1.0 / a.d;
  // rows so far apart that the offsets between those of a wave might not hold 31 bits have a wave each
  const int64_t most = std::max({a.x_stride, a.y ? a.y_stride : 0, a.y ? a.x_out_stride : 0, a.h ? a.h_stride : 0});
  const bool far = most > int64_t(1) << 20;
  const int64_t pieces = a.d / 8, cus = cu_count();
  void* kargs[] = {&a};
  if (pieces > 128 * kMaxWaves) {
    const int64_t slots = 2 * cus;
    return hipLaunchKernel((const void*)&long_rows_kernel, dim3((unsigned)(a.tokens < slots ? a.tokens : slots)),
                           dim3(kLong), kargs, 0, stream);
  }
  const void* fn;
  int threads;
  int64_t rows, slots;  // rows of a step of a wave; workgroups that run at once
  // A row to a workgroup: 16 waves run on a compute unit, and workgroups are dealt to its four SIMDs from the first on,
  // so that 3 waves take the room of 4 and 5 that of 8.
  const int64_t wide_per = pieces <= 64 * kMaxWaves ? 1 : 2;
  const int64_t waves = (pieces + 64 * wide_per - 1) / (64 * wide_per);
  const int64_t room = waves > 2 ? (waves + 3) / 4 * 4 : waves;
  // A row to a wave where there are rows for it: measured (us, norms on both sides, to codes; rows to waves and to
  // workgroups) 512 channels 4096 rows 9.1 and 7.7, 8192 12.0 and 12.3; 736 channels 4096 rows 12.0 and 12.0; 1152
  // channels 1536 rows 9.0 and 9.2, 4096 14.0 and 18.0; 2240 channels 1024 rows 10.9 and 10.2, 2048 13.4 and 17.6. And
  // where a sample has rows for the waves of a workgroup, whose vectors are its own: samples of 8, 16, 64 and 256 rows,
  // layer norm, gate and modulation to codes, in waves 21.4, 19.1, 18.7, 18.5 and in workgroups 25.0, 24.4, 23.8, 22.9
  // (8192 x 1152); 18.9, 18.8, 19.1, 18.3 and 23.3, 23.3, 23.3, 22.1 (4096 x 2240); 27.0, 17.7, 16.3, 16.2 and 18.2, 17.3,
  // 15.8, 14.6 (16384 x 512); 31.2, 20.2, 10.2, 10.0 and 24.0, 23.9, 23.8, 23.9 (32768 x 96): wide rows would gain from 8
  // on, narrow ones lose there. Samples of one row, in workgroups: 8192 x 1152 38 us, of them 34 of memory for rows and
  // vectors; 16384 x 64 17, of them 4.
  if (pieces <= 64 * kMaxPieces && a.tokens * room > 28 * cus && a.sample_rows >= 64) {
    // Rows of a wave and pieces of a lane by the fewest instructions: some 225 a piece and 120 for a row's sums, which
    // all rows of a wave share, as long as there are waves for the GPU. 8192 rows of 1152 (144 pieces): 2 rows a wave
    // with 5 pieces a lane 19.2 us, one row with 3 pieces 21.3.
    int log = 6;
    double best = 0.0;
    for (int l = 6; l >= 2; --l) {
      const int64_t per = (pieces + (1 << l) - 1) >> l;
      if (per > kMaxPieces || (l < 6 && far)) break;
      const double turns = (double)a.tokens / (double)((64 >> l) * 16 * cus);
      const double cost = (turns > 1.0 ? turns : 1.0) * (double)(225 * per + 120);
      if (l == 6 || cost < best) {
        log = l;
        best = cost;
      }
    }
    fn = rows_kernels[log - 2][((pieces + (1 << log) - 1) >> log) - 1];
    threads = kRowsThreads;
    rows = 64 >> log;
    slots = cus * resident_per_cu(fn, threads);
  } else {
    threads = (int)(64 * waves);
    fn = wide_kernels[wide_per == 1 ? 0 : threads <= 768 ? 1 : 2][a.y != nullptr]
                     [(a.h ? OUT_ROWS : 0) | (a.codes ? OUT_CODES : 0)];
    rows = 1;
    slots = cus * std::max<int64_t>(16 / room, 1);
  }
  // the same number of rows, of whole waves, for each workgroup that runs at once
  a.group_rows = ((a.tokens + slots - 1) / slots + rows - 1) / rows * rows;
  const int64_t groups = (a.tokens + a.group_rows - 1) / a.group_rows;
  return hipLaunchKernel(fn, dim3((unsigned)groups), dim3(threads), kargs, 0, stream);
}

}  // namespace kq
