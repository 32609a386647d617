// Rotary positions with several axes, over heads that may be normalised first,
// and the same on the way into the MXFP4 key/value cache.
//
// Mathematics.  Per head of D channels: n = x, or x w / sqrt(sum x^2 / D + eps).
// Pair p of the R/2 pairs that turn belongs to axis a(p) and has the angle
// positions[t][a(p)] freqs[p]; with (u, v) = n at its two channels,
//   (u, v) -> (u cos - v sin, u sin + v cos),
// so each channel is y = r (A x + B x') with x' its partner, A and B the
// cosine and signed sine with the weights folded in, and r the head's 1 / rms.
// Everything is fp64 up to one rounding to bf16; keys are then quantized from
// that bf16 as kq_cache_write does.
//
// Layout.  A lane holds one 8-channel piece (16 bytes) of a head.  A unit is
// the fewest heads whose pieces are whole blocks of 32 (one head for rows that
// are not quantized); a wave takes as many tokens as units fit its 64 lanes
// and goes over the units of those tokens, so a lane's channels and position
// never change and A and B are formed once.
#include "kq_device.hpp"
#include "kq_internal.h"
#include "kq_mxval.hpp"
#include "kq_round.hpp"

namespace kq {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // units whose loads a lane has in flight

enum { ROT_NONE = 0, ROT_PAIRS = 1, ROT_SOME_PAIRS = 2, ROT_HALVES = 3 };

// sin and cos of x quarter turns: the nearest whole number of quarters comes off exactly (1.5 2^52 added and taken
// away leaves it in the last bits), and the Taylor series on [-pi/4, pi/4] end below 2^-44.
__device__ __forceinline__ void sincos_quarters(double x, double& s, double& c) {
  const double m = x + 0x1.8p52;
  const unsigned quarter = (unsigned)__builtin_bit_cast(uint64_t, m);
  const double t = (x - (m - 0x1.8p52)) * 1.57079632679489661923;
  const double z = t * t;
  double p = fma(z, 1.0 / 6227020800.0, -1.0 / 39916800.0);
  p = fma(z, p, 1.0 / 362880.0);
  p = fma(z, p, -1.0 / 5040.0);
  p = fma(z, p, 1.0 / 120.0);
  p = fma(z, p, -1.0 / 6.0);
  const double sn = fma(t * z, p, t);
  double q = fma(z, -1.0 / 87178291200.0, 1.0 / 479001600.0);
  q = fma(z, q, -1.0 / 3628800.0);
  q = fma(z, q, 1.0 / 40320.0);
  q = fma(z, q, -1.0 / 720.0);
  q = fma(z, q, 1.0 / 24.0);
  q = fma(z, q, -0.5);
  const double cs = fma(z, q, 1.0);
  const double a = quarter & 1 ? cs : sn, b = quarter & 1 ? sn : cs;
  s = quarter & 2 ? -a : a;
  c = (quarter + 1) & 2 ? -b : b;
}

__device__ __forceinline__ double from_lane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = (unsigned)__builtin_amdgcn_ds_bpermute(4 * lane, (int)(unsigned)b);
  const unsigned hi = (unsigned)__builtin_amdgcn_ds_bpermute(4 * lane, (int)(unsigned)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the `pieces` lanes of a head, which start at lane `first`; c is this lane's place among them.  With a
// power of two the heads are aligned groups.  Otherwise a lane adds windows of 1, 2, 4, .. lanes that begin at its
// own place (wrapping round within the head), of the sizes in the binary form of `pieces`.
__device__ __forceinline__ double head_sum(double v, int pieces, int first, int c) {
  if ((pieces & (pieces - 1)) == 0) {
    if (pieces == 16) return group_sum<4>(v);
    if (pieces == 8) return group_sum<3>(v);
    if (pieces == 4) return group_sum<2>(v);
    return pieces == 2 ? group_sum<1>(v) : v;
  }
  double total = 0.0;
  int done = 0;  // lanes that total covers
  for (int w = 1; w <= pieces; w <<= 1) {
    if (pieces & w) {
      int at = c + done;
      at -= at >= pieces ? pieces : 0;
      total += done ? from_lane(v, first + at) : v;
      done += w;
    }
    if (2 * w <= pieces) {
      int at = c + w;
      at -= at >= pieces ? pieces : 0;
      v += from_lane(v, first + at);
    }
  }
  return total;
}

template <int ROT, bool NORM>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
  __shared__ u32x4 stage[ROT == ROT_HALVES ? kThreads : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int pieces = a.head_dim >> 3;
  for (int64_t index = (int64_t)blockIdx.x * (kThreads / 64) + wave; index < a.waves;
       index += (int64_t)gridDim.x * (kThreads / 64)) {
    int64_t i = index;
    int which = 0;
    while (i >= a.part[which].waves) i -= a.part[which++].waves;
    const RopePart& s = a.part[which];
    const int64_t tile = i / s.chunks;
    const int unit0 = (int)(i - tile * s.chunks) * s.per;
    const int unit1 = unit0 + s.per < s.units ? unit0 + s.per : s.units;
    // this lane's token, head within a unit and piece within the head
    const int of_token = lane / s.lanes;
    const bool used = of_token < s.tokens;  // lanes past the last whole unit do as lane 0
    const int in_unit = used ? lane - of_token * s.lanes : 0;
    const int of_head = in_unit / pieces, c = in_unit - of_head * pieces;
    const int first = used ? lane - c : 0;  // the head's first lane
    const int64_t t = tile * s.tokens + of_token;
    bool live = used && t < a.tokens;
    const int64_t row = t < a.tokens ? t : a.tokens - 1;  // lanes without a token read one that is there
    const bool cache = s.codes != nullptr;
    int64_t slot = 0;
    if (cache) {
      const int at = a.slots[row];
      live = live && (unsigned)at < (unsigned)a.n_slots;  // a token without a slot writes nothing
      slot = live ? at : 0;
    }
    const uint16_t* const x = s.x + row * s.x_stride + 8 * c;

    double A[8], B[8];
    bool turns[8];
    if (s.turn) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int ch = 8 * c + j;
        const bool upper = ROT == ROT_HALVES ? ch >= a.pairs : ch & 1;
        const int pair = ROT == ROT_HALVES ? (upper ? ch - a.pairs : ch) : ch >> 1;
        const bool turn = ROT != ROT_NONE && (ROT == ROT_PAIRS || pair < a.pairs);
        turns[j] = turn;
        A[j] = 1.0;
        B[j] = 0.0;
        if (turn) {
          // two channels of an adjacent pair share their angle
          if ((ROT == ROT_PAIRS || ROT == ROT_SOME_PAIRS) && (j & 1)) {
            A[j] = A[j - 1];
            B[j] = -B[j - 1];
          } else {
            int axis = 0;
            for (int k = 0; k < a.n_axes - 1; ++k) axis += pair >= a.axis_end[k];
            const double turned = a.freqs[pair] * 0.63661977236758134308;  // 2 / pi
            double sn, cs;
            sincos_quarters((double)a.positions[row * a.n_axes + axis] * turned, sn, cs);
            A[j] = cs;
            B[j] = upper ? sn : -sn;
          }
        }
      }
      if (NORM && s.weight) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int ch = 8 * c + j;
          int partner = ch;
          if constexpr (ROT == ROT_PAIRS || ROT == ROT_SOME_PAIRS) partner = ch ^ 1;
          if constexpr (ROT == ROT_HALVES) partner = !turns[j] ? ch : ch >= a.pairs ? ch - a.pairs : ch + a.pairs;
          A[j] *= (double)s.weight[ch];
          B[j] *= (double)s.weight[partner];
        }
      }
    }

    for (int u0 = unit0; u0 < unit1; u0 += kBatch) {
      u32x4 in[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        int head = (u0 + k) * s.unit_heads + of_head;
        head = head < s.heads ? head : s.heads - 1;
        in[k] = *reinterpret_cast<const u32x4*>(x + (int64_t)head * a.head_dim);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (u0 + k >= unit1) break;  // uniform
        const int head = (u0 + k) * s.unit_heads + of_head;
        u32x4 v = in[k];
        if (s.turn) {
          double y[8], other[8];
          piece_values(v, y);
          if constexpr (ROT == ROT_PAIRS || ROT == ROT_SOME_PAIRS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) other[j] = ROT == ROT_PAIRS || turns[j] ? y[j ^ 1] : 0.0;
          } else if constexpr (ROT == ROT_HALVES) {
            // the partners come through the wave's own LDS: a piece of them where halves are whole pieces
            u32x4* const mine = stage + (threadIdx.x & ~63u);
            mine[lane] = v;
            wave_lds_fence();
            if ((a.pairs & 7) == 0) {
              const int from = !turns[0] ? c : 8 * c >= a.pairs ? c - (a.pairs >> 3) : c + (a.pairs >> 3);
              piece_values(mine[first + from], other);
#pragma unroll
              for (int j = 0; j < 8; ++j) other[j] = turns[j] ? other[j] : 0.0;
            } else {
              const uint16_t* const head0 = reinterpret_cast<const uint16_t*>(mine + first);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int ch = 8 * c + j;
                const int from = !turns[j] ? ch : ch >= a.pairs ? ch - a.pairs : ch + a.pairs;
                other[j] = turns[j] ? (double)__uint_as_float((unsigned)head0[from] << 16) : 0.0;
              }
            }
            wave_lds_fence();
          }
          double r = 1.0;
          if constexpr (NORM) {
            double q = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) q = fma(y[j], y[j], q);
            r = inverse_sqrt(fma(head_sum(q, pieces, first, c), a.inv_dim, a.eps));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y[j] *= A[j];
            if constexpr (ROT != ROT_NONE) y[j] = fma(B[j], other[j], y[j]);
            if constexpr (NORM) y[j] *= r;
          }
          v = round_piece(y);
        }
        if (cache) {
          unsigned word, byte;
          quantize_piece(v, word, byte);
          if (live) {
            const int chunk = head * pieces + c;
            *reinterpret_cast<unsigned*>(s.codes + slot * (s.heads * pieces * 4) + 4 * chunk) = word;
            if ((chunk & 3) == 0) s.scales[slot * (s.heads * pieces >> 2) + (chunk >> 2)] = (uint8_t)byte;
          }
        } else if (live && head < s.heads) {
          *reinterpret_cast<u32x4*>(s.out + row * s.out_stride + (int64_t)head * a.head_dim + 8 * c) = v;
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& args, hipStream_t stream) {
  RopeArgs a = args;
  a.inv_dim = 1.0 / a.head_dim;
  const int pieces = a.head_dim / 8;
  const int rot = a.n_axes == 0 ? ROT_NONE
                  : a.halves    ? ROT_HALVES
                  : 2 * a.pairs == a.head_dim ? ROT_PAIRS : ROT_SOME_PAIRS;
  a.waves = 0;
  for (RopePart& p : a.part) {
    p.waves = 0;
    if (p.heads == 0) continue;
    p.unit_heads = 1;
    if (p.codes)
      while (p.unit_heads * a.head_dim % 32 != 0) ++p.unit_heads;
    p.lanes = p.unit_heads * pieces;
    p.tokens = 64 / p.lanes;
    p.units = (p.heads + p.unit_heads - 1) / p.unit_heads;
    const int64_t tiles = (a.tokens + p.tokens - 1) / p.tokens;
    // units of a wave: all of a token's, or fewer where that leaves the GPU idle
    int64_t chunks = (int64_t)cu_count() * 8 / tiles;
    chunks = chunks < 1 ? 1 : chunks > p.units ? p.units : chunks;
    p.per = (int)((p.units + chunks - 1) / chunks);
    p.chunks = (p.units + p.per - 1) / p.per;
    p.waves = tiles * p.chunks;
    a.waves += p.waves;
  }
  const int64_t most = int64_t(1) << 22, need = (a.waves + 3) / 4;
  const dim3 grid((unsigned)(need < most ? need : most));
  static const void* const kernels[4][2] = {
      {(const void*)&rope_kernel<ROT_NONE, false>, (const void*)&rope_kernel<ROT_NONE, true>},
      {(const void*)&rope_kernel<ROT_PAIRS, false>, (const void*)&rope_kernel<ROT_PAIRS, true>},
      {(const void*)&rope_kernel<ROT_SOME_PAIRS, false>, (const void*)&rope_kernel<ROT_SOME_PAIRS, true>},
      {(const void*)&rope_kernel<ROT_HALVES, false>, (const void*)&rope_kernel<ROT_HALVES, true>}};
  void* kargs[] = {&a};
  return hipLaunchKernel(kernels[rot][a.norm], grid, dim3(kThreads), kargs, 0, stream);
}

}  // namespace kq
