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
// Layout.  A lane holds 8 channels of a head: four whole pairs, that is one
// 16-byte piece where pairs are neighbours, two of 8 bytes, R/2 apart, where
// they are halves, and the piece of its own where they do not turn.  A wave
// takes as many tokens as heads fit its 64 lanes and goes over the heads of
// those tokens, four at a time, so a lane's channels and position never change
// and its cosines and sines, with the weights, are formed once.  Keys then go
// through the wave's own LDS, four heads of its tokens as one run of pieces:
// blocks of 32 channels that span heads come out in four adjacent lanes, as
// kq_cache_write's do.  Values are taken as that call takes them.  R that is no
// multiple of 8 takes a slower form: a lane holds a piece and fetches each
// partner.
//
// What bounds it, measured (kernel alone; a copy reaches 5.09 TB/s).  Many
// tokens: memory.  32761 tokens of 16 heads of 128, three axes, norm: 56 us,
// 4.75 TB/s; 20481 tokens of 32 queries, 8 keys and 8 values of 128 to the
// cache: 98 us, 4.5 TB/s.  Some thousand tokens: a wave's chain of position,
// frequency, sines, heads and, for keys, the way through LDS, which all waves
// go through at the same time.  8192 tokens of 16 heads of 72: 10.4 to 10.8 us, a
// copy 6.5.  4095 of 16 keys and values of 72, normalised: 13.8 to 14.2 us; the
// keys alone 12.5, values alone 5.3, the same heads turned into rows 11.1, without
// the norm 8.4: it is the keys' chain, the norm's sums a quarter of it.  A few
// tokens: the launch and that chain, 4.7 to 4.9 us.  R that is no multiple of 8:
// 32761 tokens as above 71 (neighbours) and 73 us (halves), every partner a
// 16-bit read from LDS; 20481 as above 122 us.
#include <algorithm>
#include <type_traits>

#include "kq_device.hpp"
#include "kq_internal.h"
#include "kq_mxval.hpp"
#include "kq_round.hpp"

namespace kq {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads (pieces of values) that a lane has in flight

// How pairs lie: not at all; neighbours or halves with R a multiple of 8; either with any R.
enum { ROT_NONE = 0, ROT_PAIRS = 1, ROT_HALVES = 2, ROT_ANY_PAIRS = 3, ROT_ANY_HALVES = 4 };

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

// Position and frequency of pair p at a token; all loads of a lane's pairs go out before the first is used.
struct Angle {
  int position;
  double freq;
  __device__ __forceinline__ void load(const RopeArgs& a, int64_t row, int p) {
    int axis = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) axis += p >= a.axis_end[k];  // of axes that are not there, past every pair
    position = a.positions[row * a.n_axes + axis];
    freq = a.freqs[p];
  }
  __device__ __forceinline__ void turn(double& sn, double& cs) const {
    sincos_quarters((double)position * (freq * 0.63661977236758134308), sn, cs);  // 2 / pi
  }
};

// 1 / rms of the head that this lane's values are of.
__device__ __forceinline__ double head_scale(const RopeArgs& a, const double y[8], int pieces, int first, int c) {
  double q = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) q = fma(y[j], y[j], q);
  return inverse_sqrt(fma(head_sum(q, pieces, first, c), a.inv_dim, a.eps));
}

// Lanes with whole pairs: values j and partner(j) of a lane are a pair.
template <int ROT>
struct WholePairs {
  static constexpr bool kHalves = ROT == ROT_HALVES;
  double cu[4], sv[4], su[4], cv[4];  // cosine and sine times the weight of the first (u) or second (v) channel
  bool turns;

  static __device__ constexpr int first_of(int j) { return kHalves ? j : 2 * j; }
  static __device__ constexpr int second_of(int j) { return kHalves ? 4 + j : 2 * j + 1; }

  // lo, hi: the channels of the lane's first and last four values
  __device__ __forceinline__ void form(const RopeArgs& a, int64_t row, const float* weight, int c, int lo, int hi) {
    turns = ROT != ROT_NONE && 4 * c < a.pairs;
    Angle angle[4];
    float wu[4], wv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (ROT != ROT_NONE) angle[j].load(a, row, turns ? 4 * c + j : 0);
      wu[j] = wv[j] = 1.0f;
      if (weight) {  // uniform
        wu[j] = weight[first_of(j) < 4 ? lo + first_of(j) : hi + first_of(j) - 4];
        wv[j] = weight[second_of(j) < 4 ? lo + second_of(j) : hi + second_of(j) - 4];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      double sn = 0.0, cs = 1.0;
      if constexpr (ROT != ROT_NONE) {
        angle[j].turn(sn, cs);
        sn = turns ? sn : 0.0;
        cs = turns ? cs : 1.0;
      }
      cu[j] = (double)wu[j] * cs;
      sv[j] = (double)wv[j] * sn;
      su[j] = (double)wu[j] * sn;
      cv[j] = (double)wv[j] * cs;
    }
  }
  __device__ __forceinline__ void apply(double y[8], double r) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double u = y[first_of(j)], v = y[second_of(j)];
      double nu = cu[j] * u, nv = cv[j] * v;
      if (ROT != ROT_NONE && turns) {  // else the other channel may be infinite
        nu = fma(-sv[j], v, nu);
        nv = fma(su[j], u, nv);
      }
      y[first_of(j)] = nu * r;
      y[second_of(j)] = nv * r;
    }
  }
};

// Lanes with one piece, of which any channels turn, with partners anywhere in the head.
template <int ROT>
struct AnyPairs {
  double A[8], B[8];
  int from[8];  // the partner's channel, or the channel itself
  bool turns[8];

  __device__ __forceinline__ void form(const RopeArgs& a, int64_t row, const float* weight, int c, int, int) {
    Angle angle[8];
    float own[8], other[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ch = 8 * c + j;
      const bool upper = ROT == ROT_ANY_HALVES ? ch >= a.pairs : ch & 1;
      const int pair = ROT == ROT_ANY_HALVES ? (upper ? ch - a.pairs : ch) : ch >> 1;
      turns[j] = pair < a.pairs;
      from[j] = !turns[j] ? ch : ROT == ROT_ANY_HALVES ? (upper ? pair : ch + a.pairs) : ch ^ 1;
      angle[j].load(a, row, turns[j] ? pair : 0);
      own[j] = other[j] = 1.0f;
      if (weight) {  // uniform
        own[j] = weight[ch];
        other[j] = weight[from[j]];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool upper = ROT == ROT_ANY_HALVES ? 8 * c + j >= a.pairs : j & 1;
      double sn, cs;
      angle[j].turn(sn, cs);
      A[j] = (double)own[j] * (turns[j] ? cs : 1.0);
      B[j] = turns[j] ? (double)other[j] * (upper ? sn : -sn) : 0.0;  // an infinite weight's product would be NaN
    }
  }
  // head: the raw channels of the head
  __device__ __forceinline__ void apply(double y[8], double r, const uint16_t* head) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // -0 leaves a channel that does not turn its sign
      const double other = turns[j] ? (double)__uint_as_float((unsigned)head[from[j]] << 16) : -0.0;
      y[j] = fma(B[j], other, A[j] * y[j]) * r;
    }
  }
};

// Codes and scale of a piece at place `chunk` of slot `slot`; the piece's block lies in four adjacent lanes.
__device__ __forceinline__ void store_piece(const RopeArgs& a, const RopePart& s, u32x4 v, int slot, int chunk) {
  unsigned word, byte;
  quantize_piece(v, word, byte);
  if ((unsigned)slot < (unsigned)a.n_slots) {  // a token without a slot writes nothing
    const int chunks = s.heads * (a.head_dim >> 3);
    *reinterpret_cast<unsigned*>(s.codes + (int64_t)slot * (4 * chunks) + 4 * chunk) = word;
    if ((chunk & 3) == 0) s.scales[(int64_t)slot * (chunks >> 2) + (chunk >> 2)] = (uint8_t)byte;
  }
}

// Values: kBatch * 64 consecutive pieces of the rows.
__device__ __forceinline__ void write_values(const RopeArgs& a, const RopePart& s, int64_t index, int lane) {
  const int chunks = s.heads * (a.head_dim >> 3);
  const int64_t base = index * (64 * kBatch);
  const int64_t row0 = base / chunks;
  const unsigned first = (unsigned)(base - row0 * chunks) + lane;
  u32x4 in[kBatch];
  int slot[kBatch], chunk[kBatch];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const unsigned at = first + 64 * k, r = fast_div(at, a.by_value_chunks);
    const int64_t row = row0 + r;
    chunk[k] = (int)(at - r * (unsigned)chunks);
    in[k] = u32x4{0, 0, 0, 0};
    slot[k] = -1;
    if (row < a.tokens) {
      in[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(s.x + row * s.x_stride + 8 * chunk[k]));
      slot[k] = a.slots[row];
    }
  }
#pragma unroll
  for (int k = 0; k < kBatch; ++k) store_piece(a, s, in[k], slot[k], chunk[k]);
}

template <int ROT, bool NORM>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
  constexpr bool kAny = ROT >= ROT_ANY_PAIRS;
  __shared__ u32x4 stage[kThreads * kBatch];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  u32x4* const mine = stage + 64 * kBatch * wave;
  const int pieces = a.head_dim >> 3;
  int64_t i = a.first_wave + (int64_t)blockIdx.x * (kThreads / 64) + wave;
  if (i >= a.waves) return;
  int which = 0;
  while (i >= a.part[which].waves) i -= a.part[which++].waves;
  const RopePart& s = a.part[which];
  if (!s.turn) {
    write_values(a, s, i, lane);
    return;
  }
  const int64_t tile = i / s.chunks;
  const int head0 = (int)(i - tile * s.chunks) * s.per;
  const int head1 = head0 + s.per < s.heads ? head0 + s.per : s.heads;
  // this lane's token and place within a head
  const int of_token = lane / pieces;
  const bool used = of_token < s.tokens;  // lanes past the last whole head do as lane 0
  const int token = used ? of_token : 0, c = used ? lane - token * pieces : 0;
  const int first = token * pieces;  // the head's first lane
  const int64_t t0 = tile * s.tokens, t = t0 + token;
  const bool live = used && t < a.tokens;
  const int64_t row = t < a.tokens ? t : a.tokens - 1;
  const bool cache = s.codes != nullptr;
  // channels of the first and the last four values
  const bool apart = ROT == ROT_HALVES && 4 * c < a.pairs;
  const int lo = apart ? 4 * c : 8 * c, hi = apart ? a.pairs + 4 * c : 8 * c + 4;

  // the rows of the wave's tokens are one buffer; heads are added as a scalar offset
  const int64_t rows = t0 + s.tokens < a.tokens ? s.tokens : a.tokens - t0;
  const auto rx = rsrc_uniform(s.x + t0 * s.x_stride, 2 * ((rows - 1) * s.x_stride + (int64_t)s.heads * a.head_dim));
  const int of_row = 2 * (int)(row - t0) * (int)s.x_stride;
  const int at_lo = of_row + 2 * lo, at_hi = of_row + 2 * hi;
  constexpr int kPast = (int)0x80000000u;  // it and what a head adds lie past every buffer: nothing is read or written
  auto load = [&](int head) {
    const int at = head * a.head_dim * 2;
    const bool there = head < head1;  // uniform
    if constexpr (ROT == ROT_HALVES) {
      const u32x2 l = __builtin_amdgcn_raw_buffer_load_b64(rx, there ? at_lo : kPast, there ? at : 0, 0);
      const u32x2 h = __builtin_amdgcn_raw_buffer_load_b64(rx, there ? at_hi : kPast, there ? at : 0, 0);
      return u32x4{l[0], l[1], h[0], h[1]};
    } else {
      return __builtin_bit_cast(u32x4,
                                __builtin_amdgcn_raw_buffer_load_b128(rx, there ? at_lo : kPast, there ? at : 0, 0));
    }
  };
  u32x4 in[kBatch];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) in[k] = load(head0 + k);
  const int slot = cache && live ? a.slots[row] : -1;

  std::conditional_t<kAny, AnyPairs<ROT>, WholePairs<ROT>> turns;
  turns.form(a, row, NORM ? s.weight : nullptr, c, lo, hi);
  const auto ro = rsrc_uniform(s.out + t0 * s.out_stride, 2 * ((rows - 1) * s.out_stride + (int64_t)s.heads * a.head_dim));
  const int of_out = 2 * (int)(row - t0) * (int)s.out_stride;
  const int out_lo = live ? of_out + 2 * lo : kPast, out_hi = live ? of_out + 2 * hi : kPast;

  // Head k of the batch of `heads` from h0 on.  As soon as a head's values are out of their registers, those of the
  // head kBatch further on are on their way into them.  Keys and rows have loops of their own, and whole batches one
  // without a condition, so that how many stores lie behind a load is known when compiling, and with it the wait.
  auto turn_head = [&](auto keys, int h0, int heads, int k) {
    u32x4 v = in[k];
    double y[8];
    piece_values(v, y);
    in[k] = load(h0 + kBatch + k);
    double r = 1.0;
    if constexpr (NORM) r = head_scale(a, y, pieces, first, c);
    u32x4* const head = mine + (token * heads + k) * pieces;  // a run of heads for each token
    if constexpr (kAny) {
      if (used) head[c] = v;
      wave_lds_fence();
      turns.apply(y, r, reinterpret_cast<const uint16_t*>(head));
      wave_lds_fence();
    } else {
      turns.apply(y, r);
    }
    v = round_piece(y);
    if constexpr (decltype(keys)::value) {
      u32x2* const fours = reinterpret_cast<u32x2*>(head);
      if (used) {
        fours[lo >> 2] = u32x2{v[0], v[1]};
        fours[hi >> 2] = u32x2{v[2], v[3]};
      }
    } else {
      // The head is added to the lane's offset, not given as the instruction's scalar one: a 16-byte store with a
      // scalar register for an offset reads its last lanes' data so late that the next instruction may have replaced
      // it (seen as zeros in four lanes of 16), and the compiler puts the wait only behind stores without one.
      const int at = (h0 + k) * a.head_dim * 2;
      if constexpr (ROT == ROT_HALVES) {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{v[0], v[1]}, ro, out_lo + at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{v[2], v[3]}, ro, out_hi + at, 0, 0);
      } else {
        __builtin_amdgcn_raw_buffer_store_b128(v, ro, out_lo + at, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto batches = [&](auto keys) {
    auto write_keys = [&](int h0, int heads) {
      if constexpr (decltype(keys)::value) {
        wave_lds_fence();
        const int run = heads * pieces;                       // pieces of a token, whole blocks of 32
        const unsigned by_run = 65536u / (unsigned)run + 1u;  // n / run for n < 256: n by_run >> 16
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int n = 64 * k + lane;
          const int tk = (int)((unsigned)n * by_run >> 16);
          const int at = __builtin_amdgcn_ds_bpermute(4 * tk * pieces, slot);
          store_piece(a, s, mine[n], tk < s.tokens ? at : -1, h0 * pieces + n - tk * run);
        }
        wave_lds_fence();
      }
    };
    int h0 = head0;
    for (; h0 + kBatch <= head1; h0 += kBatch) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) turn_head(keys, h0, kBatch, k);
      write_keys(h0, kBatch);
    }
    const int heads = head1 - h0;
    if (heads > 0) {
#pragma unroll
      for (int k = 0; k < kBatch - 1; ++k)
        if (k < heads) turn_head(keys, h0, heads, k);
      write_keys(h0, heads);
    }
  };
  if (cache) batches(std::true_type{});
  else batches(std::false_type{});
}

}  // namespace

hipError_t launch_rope(const RopeArgs& args, hipStream_t stream) {
  RopeArgs a = args;
  a.inv_dim = 1.0 / a.head_dim;
  const int pieces = a.head_dim / 8;
  const bool eights = a.pairs % 4 == 0;
  const int rot = a.n_axes == 0 ? ROT_NONE
                  : a.halves    ? (eights ? ROT_HALVES : ROT_ANY_HALVES)
                                : (eights ? ROT_PAIRS : ROT_ANY_PAIRS);
  a.waves = 0;
  for (RopePart& p : a.part) {
    p.waves = 0;
    if (p.heads == 0) continue;
    if (!p.turn) {
      a.by_value_chunks = make_divisor((unsigned)(p.heads * pieces));
      p.waves = (a.tokens * p.heads * pieces + 64 * kBatch - 1) / (64 * kBatch);
      a.waves += p.waves;
      continue;
    }
    // tokens of a wave: their rows lie within the 2^31 bytes of a buffer
    const int64_t row_bytes = 2 * std::max(p.x_stride, p.codes ? 0 : p.out_stride);
    p.tokens = (int)std::clamp<int64_t>((int64_t(1) << 30) / row_bytes, 1, 64 / pieces);
    const int64_t tiles = (a.tokens + p.tokens - 1) / p.tokens;
    // Heads of a wave: all of its tokens', or fewer (but whole blocks of 32) where there would be less than 8 waves a
    // compute unit. Aimed at 2, 4, 8 and 16 waves (us): 8192 tokens of 16 heads of 72 11.2, 11.3, 11.3 and 13.0, 4095
    // tokens of 16 keys and values of 72 22, 17, 14.5 and 14.3, 6001 tokens of 20 + 10 + 10 heads of 96 22.1, 22.6, 21.8
    // and 24.1: fewer leave the GPU idle, more form the same sines again.
    int unit = 1;
    while (p.codes && unit * a.head_dim % 32 != 0) ++unit;
    const int64_t units = (p.heads + unit - 1) / unit;
    const int64_t chunks = std::clamp<int64_t>((8 * (int64_t)cu_count() + tiles - 1) / tiles, 1, units);
    p.per = (int)((units + chunks - 1) / chunks) * unit;
    if (p.per > kBatch) p.per = (p.per + kBatch - 1) / kBatch * kBatch;
    p.chunks = (p.heads + p.per - 1) / p.per;
    p.waves = tiles * p.chunks;
    a.waves += p.waves;
  }
#define KQ_ROPE(ROT) {(const void*)&rope_kernel<ROT, false>, (const void*)&rope_kernel<ROT, true>}
  static const void* const kernels[5][2] = {KQ_ROPE(ROT_NONE), KQ_ROPE(ROT_PAIRS), KQ_ROPE(ROT_HALVES),
                                            KQ_ROPE(ROT_ANY_PAIRS), KQ_ROPE(ROT_ANY_HALVES)};
#undef KQ_ROPE
  const int64_t most = int64_t(1) << 23;  // workgroups of a launch, which has less than 2^32 threads
  for (a.first_wave = 0; a.first_wave < a.waves; a.first_wave += most * (kThreads / 64)) {
    const int64_t need = (a.waves - a.first_wave + kThreads / 64 - 1) / (kThreads / 64);
    void* kargs[] = {&a};
    const hipError_t e = hipLaunchKernel(kernels[rot][a.norm], dim3((unsigned)std::min(need, most)), dim3(kThreads), kargs,
                                         0, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace kq
