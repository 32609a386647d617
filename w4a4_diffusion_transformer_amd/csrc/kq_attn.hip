// Attention of bf16 queries over an MXFP4 key/value cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - m_i),
//   lse_i = m_i + log(sum_j p_ij),      m_i the running maximum,
//
// one pass over the keys.  Keys and values are the quantizer's rows (codes
// and E8M0 scales) at the slots that a page table names; they are read once
// per row tile as 4-bit codes and widened to bf16 on chip, which is exact.
//
// Precision.  q, k and v enter the matrix cores (v_mfma_f32_32x32x16_bf16)
// unrounded; scores, maxima, sums and outputs are fp32; p is rounded once to
// bf16 (half a step, at most 2^-8 relative) as the second product's operand, and o
// once when it is stored.
//
// Orientation.  Both products are computed transposed, S^T = K Q^T and
// O^T = V^T P^T, so that a lane holds one query (column l % 32) in both: the
// maximum and the sum over keys are within a lane and one exchange between
// the halves of the wave, the rescaling of O is one factor per lane, and the
// registers of S^T are already the B operand of the second product.  For
// that, K index j of lane half h in 16-key step s stands for key
// 16 s + 8 (j / 4) + 4 h + j % 4, which is the order S^T has; V^T is read in
// the same order from row-major LDS with the transposing load
// (ds_read_b64_tr_b16: 16 lanes read four rows of 16 values, lane i gets
// column i; checked on MI355X).
//
// Rows.  The q_heads / kv_heads = G heads that share a key head are packed as
// rows r = query * G + head of one tile, so keys are widened once for all of them.
#include <algorithm>

#include "kq_device.hpp"
#include "kq_internal.h"
#include "kq_mxval.hpp"

namespace kq {

namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float swap_max32(float v) {
  const unsigned u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

__device__ __forceinline__ float swap_sum32(float v) {
  const unsigned u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Sum over the four quarters of a wave.
__device__ __forceinline__ float quarter_sum(float v) {
  const unsigned u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return swap_sum32(__uint_as_float(s[0]) + __uint_as_float(s[1]));
}

// Orders a wave's own LDS accesses for the compiler; the hardware runs them in order.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// What one sequence and key head is to a workgroup.
struct Seq {
  int64_t row0;  // first row of its queries in q, out and lse
  int nq, len;   // queries and cached keys
};

__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
  Seq s;
  int64_t r0, r1;
  if (a.q_start) {
    r0 = a.q_start[b];
    r1 = a.q_start[b + 1];
  } else {
    r0 = (int64_t)b * a.max_q;
    r1 = r0 + a.max_q;
  }
  r0 = max((int64_t)0, min(r0, a.q_rows));  // a range outside q has no queries
  r1 = max(r0, min(r1, a.q_rows));
  s.row0 = r0;
  s.nq = (int)(r1 - r0);
  s.len = max(0, min(a.kv_len[b], a.capacity));
  return s;
}

// Slot of key `key` of sequence b, or -1 where there is none: past the
// length, or on a page that the cache does not have.
__device__ __forceinline__ int slot_of(const AttnArgs& a, int b, int key, int len) {
  if (key >= len) return -1;
  const int p = (int)fast_div((unsigned)key, a.by_page);
  const int64_t at = (int64_t)b * a.pages_per_seq + p;
  const int64_t page = a.table ? (int64_t)a.table[at] : at;
  if (page < 0 || page >= a.n_pages) return -1;
  return (int)page * a.page_size + (key - p * a.page_size);
}

// Scores of NK tiles of 32 keys -> probabilities in bf16 (the B operand of
// 2 NK steps), with the running maximum m (of unscaled scores), sum l and O^T.
template <int NK, int NT>
__device__ __forceinline__ void softmax_step(f32x16 (&s)[NK], float c, float& m, float& l, f32x16 (&o)[NT],
                                             bf16x8 (&p)[2 * NK]) {
  float top = s[0][0];
#pragma unroll
  for (int k = 0; k < NK; ++k)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, s[k][r]);
  const float mn = fmaxf(m, swap_max32(top));
  if (__builtin_amdgcn_ballot_w64(mn > m) != 0) {  // else nothing to rescale
    const float alpha = mn > m ? __builtin_amdgcn_exp2f((m - mn) * c) : 1.0f;  // m = -inf: 0
    l *= alpha;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[t][r] *= alpha;
    m = mn;
  }
  const float base = m == -__builtin_inff() ? 0.0f : m * c;  // nothing seen yet: every p is exp2(-inf) = 0
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < NK; ++k)
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][8 * g + j], c, -base));
        sum += e;
        p[2 * k + g][j] = (__bf16)e;
      }
  l += sum;
}

// Masks scores: bit x of `seen` (wave-uniform) says whether the tile's key x
// is there, `upto` is the last key of the tile that this lane's query sees.
template <int NK>
__device__ __forceinline__ void mask_scores(f32x16 (&s)[NK], uint64_t seen, int upto, int half) {
#pragma unroll
  for (int k = 0; k < NK; ++k)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int x = 32 * k + 8 * (r >> 2) + (r & 3);  // key of half 0; half 1 has x + 4
      const bool there = half ? (seen >> (x + 4)) & 1 : (seen >> x) & 1;
      if (!there || x + 4 * half > upto) s[k][r] = -__builtin_inff();
    }
}

// Adds P V of one 16-key step: V rows at `v` (this step's first key), row
// stride `stride` elements.
template <int NT>
__device__ __forceinline__ void add_pv(f32x16 (&o)[NT], const uint16_t* v, int stride, const bf16x8& p, int lane) {
  typedef __attribute__((address_space(3))) s16x4 lds4;
  const int g = lane >> 4, i = lane & 15;
  // 16 lanes: key rows 4 h .. 4 h + 3 (and + 8), columns 16 (g % 2) .. + 15 of each 32-column tile
  const uint16_t* at = v + (4 * (g >> 1) + (i >> 2)) * stride + 16 * (g & 1) + 4 * (i & 3);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 32 * t));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 8 * stride + 32 * t));
    const bf16x8 w = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, p, o[t], 0, 0, 0);
  }
}

// Writes a lane's query: the output and lse, or, in a split launch, this
// range's unnormalised output, maximum (in log2 units) and sum.
template <int NT>
__device__ __forceinline__ void store_row(const AttnArgs& a, const f32x16 (&o)[NT], float m, float l, int64_t row,
                                          int head, int split, int half, bool live) {
  if (!live) return;
  const float base = m == -__builtin_inff() ? m : m * a.c;
  if (a.nsplits > 1) {
    const int64_t n = a.q_rows * a.q_heads, at = split * n + row * a.q_heads + head;
    if (half == 0) {
      float* ml = a.part + (int64_t)a.nsplits * n * a.head_dim + 2 * at;
      ml[0] = base;
      ml[1] = l;
    }
    if (l == 0.0f) return;  // the join reads no output of an empty range
    float* dst = a.part + at * a.head_dim;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int d = 32 * t + 8 * g + 4 * half;
        if (d < a.head_dim)
          *reinterpret_cast<f32x4*>(dst + d) = f32x4{o[t][4 * g], o[t][4 * g + 1], o[t][4 * g + 2], o[t][4 * g + 3]};
      }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // an empty row: zeros
  if (a.lse && half == 0) a.lse[row * a.q_heads + head] = kLn2 * (base + __builtin_amdgcn_logf(l));
  uint16_t* dst = a.out + row * a.out_stride + (int64_t)head * a.head_dim;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * t + 8 * g + 4 * half;
      if (d < a.head_dim) {
        typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
        const bf16x4 w = {(__bf16)(o[t][4 * g] * inv), (__bf16)(o[t][4 * g + 1] * inv),
                          (__bf16)(o[t][4 * g + 2] * inv), (__bf16)(o[t][4 * g + 3] * inv)};
        *reinterpret_cast<u32x2*>(dst + d) = __builtin_bit_cast(u32x2, w);
      }
    }
}

// ---------------------------------------------------------------- many rows

// Workgroup: 4 waves of 32 rows over the same keys.  Tiles of 64 keys are
// widened once per workgroup into LDS (row-major, padded so that fragment
// reads and transposing reads fall on distinct banks), double buffered: the
// codes of tile t + 1 are loaded before tile t is multiplied and widened after.
constexpr int kRowsWaves = 4, kRowsTile = 32 * kRowsWaves, kKeys = 64;

template <int DP>
__global__ __launch_bounds__(64 * kRowsWaves, 2) void attn_rows_kernel(AttnArgs a) {
  constexpr int KS = DP + 8, VS = DP + 16;  // row strides of the staged tiles, elements
  constexpr int NT = DP / 32, ND = DP / 16, NC = DP / 8, U = kKeys * NC / (64 * kRowsWaves);
  __shared__ __attribute__((aligned(16))) uint16_t ks[2][kKeys * KS];
  __shared__ __attribute__((aligned(16))) uint16_t vs[2][kKeys * VS];

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  int id = xcd_remap(blockIdx.x, gridDim.x);
  const int split = id % a.nsplits;
  id /= a.nsplits;
  const int tile = id % a.row_tiles;
  id /= a.row_tiles;
  const int kvh = id % a.kv_heads, b = id / a.kv_heads;
  const Seq sq = sequence(a, b);
  const int rows = min(sq.nq, a.max_q) * a.group;
  const int r0 = tile * kRowsTile;
  if (r0 >= rows) return;

  // keys of this workgroup: what its last query sees, this split's share of it
  const int last_q = (int)fast_div((unsigned)(min(r0 + kRowsTile, rows) - 1), a.by_group);
  const int see = a.causal ? max(0, min(sq.len, sq.len - sq.nq + last_q + 1)) : sq.len;
  const int share = ((see + a.nsplits - 1) / a.nsplits + kKeys - 1) & ~(kKeys - 1);
  const int key0 = split * share, key1 = min(see, key0 + share);

  const int r = r0 + 32 * wv + col;
  const bool live = r < rows;
  const int qi = (int)fast_div((unsigned)min(r, rows - 1), a.by_group);
  const int head = kvh * a.group + (min(r, rows - 1) - qi * a.group);
  const int64_t row = sq.row0 + qi;
  const int upto = a.causal ? sq.len - sq.nq + qi : sq.len;  // last key this query sees
  const int upto_min = __builtin_amdgcn_readfirstlane(upto);  // rows ascend, lane 0 has the first query
  const int upto_max = __builtin_amdgcn_readlane(upto, 31);

  bf16x8 qf[ND];
  const uint16_t* qp = a.q + row * a.q_stride + (int64_t)head * a.head_dim;
#pragma unroll
  for (int s = 0; s < ND; ++s) {
    const int d = 16 * s + 8 * half;
    u32x4 w = {0, 0, 0, 0};
    if (live && d < a.head_dim) w = *reinterpret_cast<const u32x4*>(qp + d);
    qf[s] = __builtin_bit_cast(bf16x8, w);
  }

  const int chunk0 = kvh * (a.head_dim >> 3);      // the head's first 8-channel chunk in a slot's row
  const int nc = a.head_dim >> 3;
  const int64_t width8 = (int64_t)a.kv_heads * nc;  // chunks of a slot's row
  unsigned kw[U], kb[U], vw[U], vb[U];
  // Lane l looks up key l of the tile; the unit (key, chunk) u * 256 + tid takes its slot from there.
  auto load = [&](int slot) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = u * (64 * kRowsWaves) + tid, key = unit / NC, ch = unit % NC;
      const int sl = __shfl(slot, key);
      const bool in = sl >= 0 && ch < nc;
      const int64_t at = in ? (int64_t)sl * width8 + chunk0 + ch : 0;  // slot 0 is always there
      kw[u] = in ? *reinterpret_cast<const unsigned*>(a.k_codes + 4 * at) : 0u;
      kb[u] = in ? a.k_scales[at >> 2] : 0u;
      vw[u] = in ? *reinterpret_cast<const unsigned*>(a.v_codes + 4 * at) : 0u;
      vb[u] = in ? a.v_scales[at >> 2] : 0u;
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = u * (64 * kRowsWaves) + tid, key = unit / NC, ch = unit % NC;
      *reinterpret_cast<bf16x8*>(&ks[buf][key * KS + 8 * ch]) = mx_values8(kw[u], kb[u]);
      *reinterpret_cast<bf16x8*>(&vs[buf][key * VS + 8 * ch]) = mx_values8(vw[u], vb[u]);
    }
  };

  f32x16 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int x = 0; x < 16; ++x) o[t][x] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;

  if (key0 < key1) {
    int slot = slot_of(a, b, key0 + lane, key1);
    uint64_t seen = __builtin_amdgcn_ballot_w64(slot >= 0), seen_next = 0;
    load(slot);
    stage(0);
    __syncthreads();
    int buf = 0;
    for (int key = key0; key < key1; key += kKeys, buf ^= 1) {
      const bool more = key + kKeys < key1;  // uniform
      if (more) {
        slot = slot_of(a, b, key + kKeys + lane, key1);
        seen_next = __builtin_amdgcn_ballot_w64(slot >= 0);
        load(slot);
      }
      if (seen != 0 && key <= upto_max) {
        f32x16 s[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int x = 0; x < 16; ++x) s[k][x] = 0.0f;
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const bf16x8 kf = *reinterpret_cast<const bf16x8*>(&ks[buf][(32 * k + col) * KS + 16 * d + 8 * half]);
            s[k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[d], s[k], 0, 0, 0);
          }
        }
        if (seen != ~(uint64_t)0 || upto_min < key + kKeys - 1) mask_scores<2>(s, seen, upto - key, half);
        bf16x8 p[4];
        softmax_step<2, NT>(s, a.c, m, l, o, p);
#pragma unroll
        for (int x = 0; x < 4; ++x) add_pv<NT>(o, &vs[buf][16 * x * VS], VS, p[x], lane);
      }
      if (more) {
        stage(buf ^ 1);
        __syncthreads();
        seen = seen_next;
      }
    }
  }
  store_row<NT>(a, o, m, swap_sum32(l), row, head, split, half, live);
}

// ---------------------------------------------------------------- few rows

// A workgroup owns up to 16 rows; its four waves take 64-key tiles in turn,
// each with its own loads, softmax and O, and join at the end.  What bounds
// it is reading the cache: every code is read once, straight into registers
// in the operand order of v_mfma_f32_16x16x32_bf16 (lane l: key l % 16 and
// the l / 16-th quarter of the head's channels, which at head_dim 128 is one
// MX block: one 16-byte load and one scale byte), the next tile's while this
// one is multiplied.  Values pass through a wave-private LDS tile for their
// transposition (32 keys at a time), so no wave waits for another.  Key order
// within a 32-key step of the second product: index j of quarter g is key
// 4 g + j (j < 4) or 16 + 4 g + j - 4, the order S^T has.
// The key heads of one sequence and range follow one another on one XCD: they
// read neighbouring parts of the same cache lines.
constexpr int kTokenRows = 16, kTokenWaves = 4;

template <int DP, bool ALIGNED>
__global__ __launch_bounds__(64 * kTokenWaves, DP <= 64 ? 4 : 3) void attn_tokens_kernel(AttnArgs a) {
  constexpr int NS = DP / 32, NO = DP / 16, VS = DP + 16, OS = DP + 4;
  constexpr int kVBytes = kTokenWaves * 32 * VS * 2, kOBytes = kTokenWaves * kTokenRows * OS * 4;
  __shared__ __attribute__((aligned(16))) uint8_t shared[kVBytes > kOBytes ? kVBytes : kOBytes];
  __shared__ float wave_m[kTokenWaves][kTokenRows], wave_l[kTokenWaves][kTokenRows];

  const int tid = threadIdx.x, lane = tid & 63, quarter = lane >> 4, col = lane & 15;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  int id = xcd_remap(blockIdx.x, gridDim.x);
  const int kvh = id % a.kv_heads;
  id /= a.kv_heads;
  const int tile = id % a.row_tiles;
  id /= a.row_tiles;
  const int split = id % a.nsplits, b = id / a.nsplits;
  const Seq sq = sequence(a, b);
  const int rows = min(sq.nq, a.max_q) * a.group;
  const int r0 = tile * kTokenRows;
  if (r0 >= rows) return;

  const int last_q = (int)fast_div((unsigned)(min(r0 + kTokenRows, rows) - 1), a.by_group);
  const int see = a.causal ? max(0, min(sq.len, sq.len - sq.nq + last_q + 1)) : sq.len;
  const int share = ((see + a.nsplits - 1) / a.nsplits + 63) & ~63;
  const int key0 = min(see, split * share), key1 = min(see, key0 + share);

  const int r = min(r0 + col, rows - 1);
  const int qi = (int)fast_div((unsigned)r, a.by_group);
  const int head = kvh * a.group + (r - qi * a.group);
  const int upto = a.causal ? sq.len - sq.nq + qi : sq.len;  // last key this lane's query sees
  const int upto_min = __builtin_amdgcn_readfirstlane(upto);

  const int nc = a.head_dim >> 3, chunk0 = kvh * nc;
  const int64_t width8 = (int64_t)a.kv_heads * nc;
  bf16x8 qf[NS];
  const uint16_t* qp = a.q + (sq.row0 + qi) * a.q_stride + (int64_t)head * a.head_dim;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int ch = quarter * NS + s;
    u32x4 w = {0, 0, 0, 0};
    if (ch < nc) w = *reinterpret_cast<const u32x4*>(qp + 8 * ch);
    qf[s] = __builtin_bit_cast(bf16x8, w);
  }

  // One 64-key tile of this lane: codes and scales of keys 16 k + col.
  struct Tile {
    unsigned kw[4][NS], vw[4][NS];
    unsigned kb[4][ALIGNED ? 1 : NS], vb[4][ALIGNED ? 1 : NS];
    uint64_t seen;
  };
  auto load = [&](int slot, Tile& t) {
    t.seen = __builtin_amdgcn_ballot_w64(slot >= 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int sl = __shfl(slot, 16 * k + col);
      const int64_t at = (int64_t)max(sl, 0) * width8 + chunk0 + quarter * NS;  // slot 0 is always there
      if constexpr (ALIGNED) {
        typedef __attribute__((ext_vector_type(NS))) unsigned words;
        const words kw = *reinterpret_cast<const words*>(a.k_codes + 4 * at);
        const words vw = *reinterpret_cast<const words*>(a.v_codes + 4 * at);
        t.kb[k][0] = a.k_scales[at >> 2];
        t.vb[k][0] = sl >= 0 ? a.v_scales[at >> 2] : 0u;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          t.kw[k][s] = kw[s];
          t.vw[k][s] = sl >= 0 ? vw[s] : 0u;
        }
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const bool in = quarter * NS + s < nc;
          const int64_t c = in ? at + s : 0;
          t.kw[k][s] = in ? *reinterpret_cast<const unsigned*>(a.k_codes + 4 * c) : 0u;
          t.kb[k][s] = in ? a.k_scales[c >> 2] : 0u;
          t.vw[k][s] = in && sl >= 0 ? *reinterpret_cast<const unsigned*>(a.v_codes + 4 * c) : 0u;
          t.vb[k][s] = in && sl >= 0 ? a.v_scales[c >> 2] : 0u;
        }
      }
    }
  };

  f32x4 o[NO];
#pragma unroll
  for (int t = 0; t < NO; ++t) o[t] = f32x4{0, 0, 0, 0};
  float m = -__builtin_inff(), l = 0.0f;
  uint16_t* vs = reinterpret_cast<uint16_t*>(shared) + wv * 32 * VS;

  auto multiply = [&](const Tile& t, int key) {
    f32x4 s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[k] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < NS; ++d)
        s[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_values8(t.kw[k][d], t.kb[k][ALIGNED ? 0 : d]), qf[d], s[k], 0,
                                                       0, 0);
    }
    if (t.seen != ~(uint64_t)0 || upto_min < key + 63) {
      const uint64_t mine = t.seen >> (4 * quarter);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (!((mine >> (16 * k + x)) & 1) || key + 16 * k + 4 * quarter + x > upto) s[k][x] = -__builtin_inff();
    }
    float top = s[0][0];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int x = 0; x < 4; ++x) top = fmaxf(top, s[k][x]);
    if (__builtin_amdgcn_ballot_w64(top > m) != 0) {  // some query has a new maximum
      const unsigned u = __float_as_uint(top);
      const auto h = __builtin_amdgcn_permlane16_swap(u, u, false, false);
      const float mn = fmaxf(m, swap_max32(fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]))));
      const float alpha = mn > m ? __builtin_amdgcn_exp2f((m - mn) * a.c) : 1.0f;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < NO; ++d) o[d] *= alpha;
      m = mn;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m * a.c;
    bf16x8 p[2];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][x], a.c, -base));
        sum += e;
        p[k >> 1][4 * (k & 1) + x] = (__bf16)e;
      }
    l += sum;
    typedef __attribute__((address_space(3))) s16x4 lds4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int d = 0; d < NS; ++d)
          *reinterpret_cast<bf16x8*>(&vs[(16 * k + col) * VS + 8 * (quarter * NS + d)]) =
              mx_values8(t.vw[2 * half + k][d], t.vb[2 * half + k][ALIGNED ? 0 : d]);
      wave_lds_fence();
      const uint16_t* at = vs + (4 * quarter + (col >> 2)) * VS + 4 * (col & 3);
#pragma unroll
      for (int d = 0; d < NO; ++d) {
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 16 * d));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 16 * VS + 16 * d));
        const bf16x8 w = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, p[half], o[d], 0, 0, 0);
      }
      wave_lds_fence();
    }
  };

  // tiles wv, wv + 4, ... of the range: the next tile's codes are in flight during this one's
  // product, and the slots of the one after
  constexpr int kStep = 64 * kTokenWaves;
  int key = key0 + 64 * wv;
  if (key < key1) {
    Tile cur, next;
    load(slot_of(a, b, key + lane, key1), cur);
    int slot = slot_of(a, b, key + kStep + lane, key1);
    for (; key + kStep < key1; key += kStep) {
      load(slot, next);
      slot = slot_of(a, b, key + 2 * kStep + lane, key1);
      multiply(cur, key);
      cur = next;
    }
    multiply(cur, key);
  }

  // join the waves
  l = quarter_sum(l);
  if (quarter == 0) {
    wave_m[wv][col] = m;
    wave_l[wv][col] = l;
  }
  __syncthreads();  // also: every wave is done with its tile of values
  float top = wave_m[0][col];
#pragma unroll
  for (int w = 1; w < kTokenWaves; ++w) top = fmaxf(top, wave_m[w][col]);
  const float mine = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((m - top) * a.c);
  float* os = reinterpret_cast<float*>(shared);
#pragma unroll
  for (int d = 0; d < NO; ++d)
    *reinterpret_cast<f32x4*>(&os[(wv * kTokenRows + col) * OS + 16 * d + 4 * quarter]) = o[d] * mine;
  __syncthreads();
  for (int x = tid; x < kTokenRows * nc; x += 64 * kTokenWaves) {
    const int q = x / nc, ch = x - q * nc;
    if (r0 + q >= rows) break;
    float best = wave_m[0][q];
#pragma unroll
    for (int w = 1; w < kTokenWaves; ++w) best = fmaxf(best, wave_m[w][q]);
    float sum = 0.0f;
    f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kTokenWaves; ++w) {
      sum += wave_m[w][q] == -__builtin_inff() ? 0.0f
                                               : wave_l[w][q] * __builtin_amdgcn_exp2f((wave_m[w][q] - best) * a.c);
      const f32x4* src = reinterpret_cast<const f32x4*>(&os[(w * kTokenRows + q) * OS + 8 * ch]);
      lo += src[0];
      hi += src[1];
    }
    const int qx = (int)fast_div((unsigned)(r0 + q), a.by_group);
    const int h = kvh * a.group + (r0 + q - qx * a.group);
    const int64_t row = sq.row0 + qx;
    const float base = best == -__builtin_inff() ? best : best * a.c;
    if (a.nsplits > 1) {
      const int64_t n = a.q_rows * a.q_heads, at = split * n + row * a.q_heads + h;
      if (ch == 0) {
        float* ml = a.part + (int64_t)a.nsplits * n * a.head_dim + 2 * at;
        ml[0] = base;
        ml[1] = sum;
      }
      f32x4* dst = reinterpret_cast<f32x4*>(a.part + at * a.head_dim + 8 * ch);
      dst[0] = lo;
      dst[1] = hi;
    } else {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (a.lse && ch == 0) a.lse[row * a.q_heads + h] = kLn2 * (base + __builtin_amdgcn_logf(sum));
      bf16x8 w;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        w[c] = (__bf16)(lo[c] * inv);
        w[4 + c] = (__bf16)(hi[c] * inv);
      }
      *reinterpret_cast<u32x4*>(a.out + row * a.out_stride + (int64_t)h * a.head_dim + 8 * ch) =
          __builtin_bit_cast(u32x4, w);
    }
  }
}

// ---------------------------------------------------------------- joining

// One lane per eight channels of a row: the splits' outputs weighted by
// exp2(max_s - max).
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int nc = a.head_dim >> 3;
  const int64_t per = (int64_t)a.max_q * a.q_heads * nc;  // lanes of a sequence
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int b = blockIdx.y;
  if (i >= per) return;
  const Seq sq = sequence(a, b);
  const int ch = (int)(i % nc);
  const int64_t rh = i / nc;
  const int head = (int)(rh % a.q_heads), qi = (int)(rh / a.q_heads);
  if (qi >= sq.nq) return;
  const int64_t n = a.q_rows * a.q_heads, at = (sq.row0 + qi) * a.q_heads + head;
  const float* ml = a.part + (int64_t)a.nsplits * n * a.head_dim;
  float top = -__builtin_inff();
  for (int s = 0; s < a.nsplits; ++s) top = fmaxf(top, ml[2 * (s * n + at)]);
  float sum = 0.0f, o[8] = {};
  for (int s = 0; s < a.nsplits; ++s) {
    const float l = ml[2 * (s * n + at) + 1];
    if (l == 0.0f) continue;
    const float w = __builtin_amdgcn_exp2f(ml[2 * (s * n + at)] - top);
    sum += w * l;
    const f32x4* src = reinterpret_cast<const f32x4*>(a.part + (s * n + at) * a.head_dim + 8 * ch);
    const f32x4 x = src[0], y = src[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[k] += w * x[k];
      o[4 + k] += w * y[k];
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (a.lse && ch == 0) a.lse[at] = kLn2 * (top + __builtin_amdgcn_logf(sum));
  bf16x8 w;
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = (__bf16)(o[k] * inv);
  *reinterpret_cast<u32x4*>(a.out + (sq.row0 + qi) * a.out_stride + (int64_t)head * a.head_dim + 8 * ch) =
      __builtin_bit_cast(u32x4, w);
}

const void* rows_kernel(int d) {
  return d <= 32   ? (const void*)&attn_rows_kernel<32>
         : d <= 64 ? (const void*)&attn_rows_kernel<64>
         : d <= 96 ? (const void*)&attn_rows_kernel<96>
                   : (const void*)&attn_rows_kernel<128>;
}

const void* tokens_kernel(int d) {
  if (d == 32) return (const void*)&attn_tokens_kernel<32, true>;
  if (d == 64) return (const void*)&attn_tokens_kernel<64, true>;
  if (d == 128) return (const void*)&attn_tokens_kernel<128, true>;
  return d < 32   ? (const void*)&attn_tokens_kernel<32, false>
         : d < 64 ? (const void*)&attn_tokens_kernel<64, false>
         : d <= 96 ? (const void*)&attn_tokens_kernel<96, false>
                   : (const void*)&attn_tokens_kernel<128, false>;
}

}  // namespace

// Few rows: up to two 16-row tiles for each sequence and key head.
AttnPlan attn_plan(int64_t batch, int64_t max_q, int64_t q_heads, int64_t kv_heads, int64_t capacity) {
  AttnPlan p;
  const int64_t rows = max_q * (q_heads / kv_heads);
  p.few = rows <= 2 * kTokenRows;
  const int tile = p.few ? kTokenRows : kRowsTile;
  p.row_tiles = (int)((rows + tile - 1) / tile);
  const int64_t tiles = std::max<int64_t>(1, batch * kv_heads * p.row_tiles);
  const int64_t want = (p.few ? 2048 : 512) / tiles, most = capacity / (p.few ? 256 : 128);
  p.nsplits = (int)std::max<int64_t>(1, std::min(want, most));
  return p;
}

int64_t attn_workspace(int64_t q_rows, int64_t q_heads, int64_t head_dim, int nsplits) {
  return nsplits > 1 ? nsplits * q_rows * q_heads * (head_dim + 2) * 4 : 0;
}

hipError_t launch_attn(const AttnArgs& args, hipStream_t stream) {
  AttnArgs a = args;
  a.group = a.q_heads / a.kv_heads;
  a.by_page = make_divisor((unsigned)a.page_size);
  a.by_group = make_divisor((unsigned)a.group);
  a.capacity = a.n_pages > 0 ? a.pages_per_seq * a.page_size : 0;
  a.c = a.scale * kLog2e;
  const AttnPlan p =
      attn_plan(a.batch, a.max_q, a.q_heads, a.kv_heads, (int64_t)a.pages_per_seq * a.page_size);
  a.nsplits = p.nsplits;
  a.row_tiles = p.row_tiles;
  void* kargs[] = {&a};
  const int64_t grid = (int64_t)a.batch * a.kv_heads * a.row_tiles * a.nsplits;
  const hipError_t e =
      hipLaunchKernel(p.few ? tokens_kernel(a.head_dim) : rows_kernel(a.head_dim), dim3((unsigned)grid),
                      dim3(64 * (p.few ? kTokenWaves : kRowsWaves)), kargs, 0, stream);
  if (e != hipSuccess || a.nsplits == 1) return e;
  const int64_t per = (int64_t)a.max_q * a.q_heads * (a.head_dim >> 3);
  return hipLaunchKernel((const void*)&attn_join_kernel, dim3((unsigned)((per + 255) / 256), (unsigned)a.batch),
                         dim3(256), kargs, 0, stream);
}

}  // namespace kq
