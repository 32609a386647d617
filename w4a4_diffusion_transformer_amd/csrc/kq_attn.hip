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
// once when it is stored.  A second bf16 term of p (p - bf16(p), another product)
// would leave o's rounding alone, rms 0.0017 of o against 0.0019 to 0.0020, and
// takes 30-35% longer (4608 rows of 16 heads of 128 over 5120 keys 280 us, 210 so).
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

// The table entry of key `key` of sequence b, as loaded.  Apart from slot_of, so that it can be asked
// for well ahead: without a branch and with nothing that looks at it, the load stays in flight.  Keys
// past the end read the last entry; without a table the word read (the sequence's length) is not used.
__device__ __forceinline__ int page_entry(const AttnArgs& a, int b, int key) {
  const int p = min((int)fast_div((unsigned)key, a.by_page), a.pages_per_seq - 1);
  const int32_t* at = a.table ? a.table + (int64_t)b * a.pages_per_seq + p : a.kv_len + b;
  return *at;
}

// Slot of key `key`, whose table entry is `entry`, or -1 where there is none: past the end, or on a
// page that the cache does not have.
__device__ __forceinline__ int slot_of(const AttnArgs& a, int b, int key, int entry, int end) {
  const int p = (int)fast_div((unsigned)key, a.by_page);
  const int64_t page = a.table ? (int64_t)entry : (int64_t)b * a.pages_per_seq + p;
  const bool there = key < end && page >= 0 && page < a.n_pages;
  return there ? (int)page * a.page_size + (key - p * a.page_size) : -1;
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

// Masks scores: `upto` is the last key of the tile that this lane's query sees; where the tile has keys
// that are not there before that (holes: a page that the cache does not have), bit x of `seen`
// (wave-uniform) says whether key x is.
template <int NK>
__device__ __forceinline__ void mask_scores(f32x16 (&s)[NK], uint64_t seen, bool holes, int upto, int half) {
  const int last = upto - 4 * half;
#pragma unroll
  for (int k = 0; k < NK; ++k)
#pragma unroll
    for (int r = 0; r < 16; ++r)  // key of half 0; half 1 has 4 more
      if (32 * k + 8 * (r >> 2) + (r & 3) > last) s[k][r] = -__builtin_inff();
  if (holes) {
    const uint64_t mine = seen >> (4 * half);
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (!((mine >> (32 * k + 8 * (r >> 2) + (r & 3))) & 1)) s[k][r] = -__builtin_inff();
  }
}

// V^T of one 16-key step as the A operands of O^T's NT tiles: V rows at `v` (the step's first key), row
// stride `stride` elements.
template <int NT>
__device__ __forceinline__ void read_values(const uint16_t* v, int stride, int lane, bf16x8 (&w)[NT]) {
  typedef __attribute__((address_space(3))) s16x4 lds4;
  const int g = lane >> 4, i = lane & 15;
  // 16 lanes: key rows 4 h .. 4 h + 3 (and + 8), columns 16 (g % 2) .. + 15 of each 32-column tile
  const uint16_t* at = v + (4 * (g >> 1) + (i >> 2)) * stride + 16 * (g & 1) + 4 * (i & 3);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 32 * t));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 8 * stride + 32 * t));
    w[t] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// What a workgroup of the many-rows kernel does.  Tiles are ranked by what
// they are likely to cost, for the longest to start first: by the sequence's
// keys (of up to 64 sequences), then by their place in it, last first (with a
// causal mask the last see the most keys).  The first a.whole ranks are
// workgroups of their own, each of the rest (the last, partial round of the
// GPU) is divided into a.nsplits key ranges, whose results are joined.
struct RowsWork {
  int b, kvh, tile;
  int index, split, splits;  // of a divided tile: its number among those, its range, and of how many
};

__device__ __forceinline__ RowsWork rows_work(const AttnArgs& a, int id) {
  RowsWork w;
  w.index = 0;
  w.split = 0;
  w.splits = 1;
  int rank = id;
  if (id >= a.whole) {
    w.index = (id - a.whole) % a.split_tiles;
    w.split = (id - a.whole) / a.split_tiles;
    w.splits = a.nsplits;
    rank = a.whole + w.index;
  }
  const int each = a.row_tiles * a.kv_heads, order = rank / each, rest = rank - order * each;
  w.tile = a.row_tiles - 1 - rest / a.kv_heads;
  w.kvh = rest % a.kv_heads;
  w.b = order;
  if (a.batch > 1 && a.batch <= 64) {  // the order-th sequence by length
    const int i = threadIdx.x & 63, len = i < a.batch ? a.kv_len[i] : 0;
    int longer = 0;
    for (int j = 0; j < a.batch; ++j) {
      const int other = __builtin_amdgcn_readlane(len, j);
      longer += other > len || (other == len && j < i);
    }
    w.b = __builtin_ctzll(__builtin_amdgcn_ballot_w64(i < a.batch && longer == order));
  }
  return w;
}

// ---------------------------------------------------------------- many rows

// A tile of 64 keys and values in LDS, row-major bf16, rows padded so that
// fragment reads (keys) and transposing reads (values) fall on distinct banks,
// and a thread's part in bringing it there: waves 0-3 widen keys, waves 4-7
// values, a thread one quarter of key tid / 4 % 64's channels.
constexpr int kRowsWaves = 8, kRowsTile = 32 * kRowsWaves, kKeys = 64;

template <int DP, bool ALIGNED>
struct KeyTile {
  static constexpr int KS = DP + 8, VS = DP + 16;      // row strides, elements
  static constexpr int kSize = kKeys * (KS + VS);      // elements: keys, then values
  static constexpr int NS = DP / 32, NB = ALIGNED ? 1 : NS;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t width8;
  int chunk0, nc, lkey, lq, at;  // at: the thread's place in a tile
  unsigned word[NS], byte[NB];   // as loaded

  __device__ __forceinline__ void place(const AttnArgs& a, int kvh, int tid, int wv) {
    const bool values = wv >= kRowsWaves / 2;  // uniform
    codes = values ? a.v_codes : a.k_codes;
    scales = values ? a.v_scales : a.k_scales;
    nc = a.head_dim >> 3;
    chunk0 = kvh * nc;
    width8 = (int64_t)a.kv_heads * nc;
    lkey = (tid >> 2) & (kKeys - 1);
    lq = tid & 3;
    at = (values ? kKeys * KS + lkey * VS : lkey * KS) + 8 * NS * lq;
  }

  // slot: of key `lane` of the tile.  A key that is not there reads slot 0 (always there), a quarter's
  // chunks past the head's its first one; nothing looks at the words before stage().
  __device__ __forceinline__ void load(int slot) {
    const int64_t row = (int64_t)max(__shfl(slot, lkey), 0) * width8 + chunk0;
    if constexpr (ALIGNED) {
      typedef __attribute__((ext_vector_type(NS))) unsigned words;
      const int64_t c = row + lq * NS;
      const words x = *reinterpret_cast<const words*>(codes + 4 * c);
      byte[0] = scales[c >> 2];
#pragma unroll
      for (int s = 0; s < NS; ++s) word[s] = x[s];
    } else {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int64_t c = row + (lq * NS + s < nc ? lq * NS + s : 0);
        word[s] = *reinterpret_cast<const unsigned*>(codes + 4 * c);
        byte[s] = scales[c >> 2];
      }
    }
  }

  __device__ __forceinline__ void stage(uint16_t* tile, uint64_t seen) {
    if (seen != ~(uint64_t)0 && !((seen >> lkey) & 1)) {  // a key that is not there: zeros, whatever the slot holds
#pragma unroll
      for (int s = 0; s < NS; ++s) word[s] = 0;
#pragma unroll
      for (int s = 0; s < NB; ++s) byte[s] = 0;
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const bool pad = !ALIGNED && lq * NS + s >= nc;  // chunks past the head's: zeros
      *reinterpret_cast<bf16x8*>(tile + at + 8 * s) = mx_values8(pad ? 0u : word[s], pad ? 0u : byte[ALIGNED ? 0 : s]);
    }
  }
};

// One tile for the 32 rows of a wave: scores, softmax, and P V added to O^T.
template <int DP>
__device__ __forceinline__ void attend_tile(const uint16_t* ks, const bf16x8 (&qf)[DP / 16], uint64_t seen, int key,
                                            int upto, int upto_min, int upto_max, float c, int lane, float& m,
                                            float& l,
                                            f32x16 (&o)[DP / 32]) {
  constexpr int KS = KeyTile<DP, false>::KS, VS = KeyTile<DP, false>::VS;
  const int half = lane >> 5, col = lane & 31;
  const uint16_t* vs = ks + kKeys * KS;
  f32x16 s[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int x = 0; x < 16; ++x) s[k][x] = 0.0f;
  // the wave in its products goes before the one in its softmax on the same SIMD: 1-3%
  __builtin_amdgcn_s_setprio(1);
  // fragments two steps ahead of their products; at 64 channels and less the registers of four waves a
  // SIMD are worth more (329 us against 383 for 2 x 4096 rows of 32 heads over 4096 keys)
  constexpr int ND = DP / 16, kAhead = DP >= 96 ? 2 : 1;
  bf16x8 kf[kAhead][2];
  auto read_keys = [&](int d) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      kf[d % kAhead][k] = *reinterpret_cast<const bf16x8*>(&ks[(32 * k + col) * KS + 16 * d + 8 * half]);
  };
  if constexpr (kAhead > 1) {
    read_keys(0);
    read_keys(1);
  }
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    if constexpr (kAhead == 1) {
      read_keys(d);
    } else {
      __builtin_amdgcn_sched_barrier(0);
    }
    const bf16x8 now[2] = {kf[d % kAhead][0], kf[d % kAhead][1]};
    if constexpr (kAhead > 1) {
      if (d + kAhead < ND) read_keys(d + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) s[k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now[k], qf[d], s[k], 0, 0, 0);
  }
  // a hole: some key under the highest that is there, or under the last that a query sees, is not
  const bool holes = (seen & (seen + 1)) != 0 || (seen != ~(uint64_t)0 && upto_max >= key + __builtin_popcountll(seen));
  if (holes || upto_min < key + kKeys - 1) mask_scores<2>(s, seen, holes, upto - key, half);
  bf16x8 p[4], w[2][DP / 32];
  __builtin_amdgcn_s_setprio(0);
  read_values<DP / 32>(vs, VS, lane, w[0]);  // a step's values are read while the one before is multiplied
  softmax_step<2, DP / 32>(s, c, m, l, o, p);
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if (x < 3) read_values<DP / 32>(vs + 16 * (x + 1) * VS, VS, lane, w[(x + 1) & 1]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < DP / 32; ++t) o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[x & 1][t], p[x], o[t], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  }
  __builtin_amdgcn_s_setprio(0);
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint64_t hi = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(v >> 32));
  return (hi << 32) | (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)v);
}

// Four values of O^T from register r on, scaled, in bf16.
__device__ __forceinline__ u32x2 pack4(const f32x16& o, int r, float inv) {
  typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
  const bf16x4 x = {(__bf16)(o[r] * inv), (__bf16)(o[r + 1] * inv), (__bf16)(o[r + 2] * inv), (__bf16)(o[r + 3] * inv)};
  return __builtin_bit_cast(u32x2, x);
}

// A workgroup owns 256 rows, 32 to each of its eight waves, over the same
// keys; tiles are widened once for all of them.  Two LDS buffers: the codes of
// tile t + 1 are loaded before tile t is multiplied and widened after it, the
// table entries of tile t + 2 asked for before those loads.  What bounds it is
// issue: a wave's exponentials and its products take turns, and two waves a
// SIMD (their O and S fill the registers) overlap them in part: 4608 rows of 16
// heads of 128 over 5120 keys 206 us, 0.94 PFLOP/s.  (The next tile's scores
// computed between a tile's exponentials by one wave: 232 us.)
template <int DP, bool ALIGNED>
__global__ __launch_bounds__(64 * kRowsWaves) __attribute__((amdgpu_waves_per_eu(DP <= 64 ? 4 : 2, DP <= 64 ? 4 : 2)))
void attn_rows_kernel(AttnArgs a) {
  using T = KeyTile<DP, ALIGNED>;
  constexpr int NT = DP / 32, ND = DP / 16, OS = DP + 8;  // OS: row stride of the outputs in LDS, elements
  static_assert(kRowsTile * OS <= 2 * T::kSize, "the outputs fit the tiles");
  __shared__ __attribute__((aligned(16))) uint16_t tiles[2 * T::kSize];

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const RowsWork w = rows_work(a, blockIdx.x);
  const Seq sq = sequence(a, w.b);
  const int rows = min(sq.nq, a.max_q) * a.group;
  const int r0 = w.tile * kRowsTile;
  if (r0 >= rows) return;

  // keys of this workgroup: what its last query sees, this range's share of it
  const int last_q = (int)fast_div((unsigned)(min(r0 + kRowsTile, rows) - 1), a.by_group);
  const int see = a.causal ? max(0, min(sq.len, sq.len - sq.nq + last_q + 1)) : sq.len;
  const int share = ((see + w.splits - 1) / w.splits + kKeys - 1) & ~(kKeys - 1);
  const int key0 = min(see, w.split * share), key1 = min(see, key0 + share);

  const int r = r0 + 32 * wv + col;
  const bool live = r < rows;
  const int qi = (int)fast_div((unsigned)min(r, rows - 1), a.by_group);
  const int head = w.kvh * a.group + (min(r, rows - 1) - qi * a.group);
  const int64_t row = sq.row0 + qi;
  const int upto = a.causal ? sq.len - sq.nq + qi : sq.len - 1;  // last key this query sees
  const int upto_min = __builtin_amdgcn_readfirstlane(upto);  // rows ascend, lane 0 has the first query
  const int upto_max = __builtin_amdgcn_readlane(upto, 31);

  bf16x8 qf[ND];
  const uint16_t* qp = a.q + row * a.q_stride + (int64_t)head * a.head_dim;
#pragma unroll
  for (int s = 0; s < ND; ++s) {
    const int d = 16 * s + 8 * half;
    u32x4 x = {0, 0, 0, 0};
    if (live && d < a.head_dim) x = *reinterpret_cast<const u32x4*>(qp + d);
    qf[s] = __builtin_bit_cast(bf16x8, x);
  }

  T part;
  part.place(a, w.kvh, tid, wv);
  f32x16 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int x = 0; x < 16; ++x) o[t][x] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;

  if (key0 < key1) {
    int slot = slot_of(a, w.b, key0 + lane, page_entry(a, w.b, key0 + lane), key1);
    int entry = page_entry(a, w.b, key0 + kKeys + lane);
    uint64_t seen = __builtin_amdgcn_ballot_w64(slot >= 0), seen_next = 0;
    part.load(slot);
    part.stage(tiles, seen);
    __syncthreads();
    int buf = 0;
    for (int key = key0; key < key1; key += kKeys, buf ^= 1) {
      const bool more = key + kKeys < key1;  // uniform
      if (more) {
        slot = slot_of(a, w.b, key + kKeys + lane, entry, key1);
        seen_next = __builtin_amdgcn_ballot_w64(slot >= 0);
        entry = page_entry(a, w.b, key + 2 * kKeys + lane);
        part.load(slot);
      }
      if (seen != 0 && key <= upto_max)
        attend_tile<DP>(tiles + buf * T::kSize, qf, seen, key, upto, upto_min, upto_max, a.c, lane, m, l, o);
      if (more) {
        part.stage(tiles + (buf ^ 1) * T::kSize, seen_next);
        __syncthreads();
        seen = seen_next;
      }
    }
  }
  l = swap_sum32(l);
  const float base = m == -__builtin_inff() ? m : m * a.c;

  if (w.splits > 1) {  // this range's unnormalised output, maximum (in log2 units) and sum
    const int64_t n = (int64_t)a.split_tiles * w.splits * kRowsTile;
    const int64_t at = ((int64_t)w.index * w.splits + w.split) * kRowsTile + 32 * wv + col;
    if (!live) return;
    if (half == 0) {
      float* ml = a.part + n * a.head_dim + 2 * at;
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

  if (a.lse && half == 0 && live) a.lse[row * a.q_heads + head] = kLn2 * (base + __builtin_amdgcn_logf(l));
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // an empty row: zeros
  // through LDS, so that a wave stores whole rows
  __syncthreads();  // every wave is done with the tiles
  uint16_t* os = tiles + 32 * wv * OS;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      *reinterpret_cast<u32x2*>(&os[col * OS + 32 * t + 8 * g + 4 * half]) = pack4(o[t], 4 * g, inv);
    }
  wave_lds_fence();
  constexpr int LPR = DP / 8, RPI = 64 / LPR;  // lanes of a row, rows of an instruction
  const int ch = lane % LPR, nc = a.head_dim >> 3;
#pragma unroll
  for (int k = 0; k < (32 + RPI - 1) / RPI; ++k) {
    const int x = k * RPI + lane / LPR, y = r0 + 32 * wv + x;  // row of the wave, packed row
    if (lane >= LPR * RPI || x >= 32 || y >= rows || ch >= nc) continue;
    const int q = (int)fast_div((unsigned)y, a.by_group), h = w.kvh * a.group + (y - q * a.group);
    *reinterpret_cast<u32x4*>(a.out + (sq.row0 + q) * a.out_stride + (int64_t)h * a.head_dim + 8 * ch) =
        *reinterpret_cast<const u32x4*>(&os[x * OS + 8 * ch]);
  }
}

// ---------------------------------------------------------------- many rows, few keys

// Cross attention to a short text: all keys and values of a sequence and head
// fit in LDS, so a workgroup widens them once and its waves then work through
// 32-row groups of their own with no barrier: wave w takes groups w, w + W, ...
// of the workgroup's.  What bounds it is latency along a group's chain of
// products and exponentials: as many waves as registers allow.  (Staged again
// for every 256 rows, the 1152-wide transformer's 8 x 4096 rows over up to 300
// keys took 106 us, most of it the start and end of workgroups; 72 so, of
// which the outputs' stores, beside no other work at the end of a group, are
// some 20.)
constexpr int resident_tiles(int dp) { return dp <= 64 ? 8 : dp <= 96 ? 5 : 4; }      // of 64 keys, as LDS allows
constexpr int resident_waves(int dp) { return dp <= 64 ? 16 : dp <= 96 ? 12 : 8; }  // as registers allow

template <int DP, bool ALIGNED>
__global__ __launch_bounds__(64 * resident_waves(DP))
    __attribute__((amdgpu_waves_per_eu(resident_waves(DP) / 4, resident_waves(DP) / 4)))
void attn_resident_kernel(AttnArgs a) {
  using T = KeyTile<DP, ALIGNED>;
  constexpr int NT = DP / 32, ND = DP / 16, NBUF = resident_tiles(DP);
  __shared__ __attribute__((aligned(16))) uint16_t tiles[NBUF * T::kSize];
  __shared__ uint64_t tile_seen[NBUF];

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  // XCD i has every head of the row tiles i, i + 8, ...: heads next to each other share cache lines of the
  // codes and, where their rows are not whole lines, of the queries and the outputs (8 x 4096 rows of 16 heads
  // over up to 300 keys: of 72 channels 76.1 us, dealt out singly 78.7; of 64 70.9 and 72.7; 24 heads of 128 level;
  // 4 x 4096 rows of 96 51.8 and 50.4)
  int id = blockIdx.x;
  if (a.by_xcd) {
    const int unit = id / (8 * a.kv_heads) * 8 + (id & 7);
    id = unit * a.kv_heads + (id >> 3) % a.kv_heads;
  }
  const RowsWork w = rows_work(a, id);
  const Seq sq = sequence(a, w.b);
  const int rows = min(sq.nq, a.max_q) * a.group;
  const int r0 = w.tile * 32 * a.run_groups;
  if (r0 >= rows) return;
  const int groups = min(a.run_groups, (rows - r0 + 31) >> 5);

  // every tile's table entries, then codes, in flight at once
  const int nt = (sq.len + kKeys - 1) / kKeys;  // at most NBUF: the capacity is
  if (wv < kRowsWaves) {
    int entry[NBUF];
#pragma unroll
    for (int t = 0; t < NBUF; ++t) entry[t] = page_entry(a, w.b, t * kKeys + lane);
    T parts[NBUF];
    uint64_t seen[NBUF];
#pragma unroll
    for (int t = 0; t < NBUF; ++t)
      if (t < nt) {
        const int slot = slot_of(a, w.b, t * kKeys + lane, entry[t], sq.len);
        seen[t] = __builtin_amdgcn_ballot_w64(slot >= 0);
        parts[t].place(a, w.kvh, tid, wv);
        parts[t].load(slot);
      }
#pragma unroll
    for (int t = 0; t < NBUF; ++t)
      if (t < nt) {
        if (tid == 0) tile_seen[t] = seen[t];
        parts[t].stage(tiles + t * T::kSize, seen[t]);
      }
  }
  __syncthreads();

  for (int g = wv; g < groups; g += resident_waves(DP)) {
    const int r = r0 + 32 * g + col;
    const bool live = r < rows;
    const int qi = (int)fast_div((unsigned)min(r, rows - 1), a.by_group);
    const int head = w.kvh * a.group + (min(r, rows - 1) - qi * a.group);
    const int64_t row = sq.row0 + qi;
    const int upto = a.causal ? sq.len - sq.nq + qi : sq.len - 1;  // last key this query sees
    const int upto_min = __builtin_amdgcn_readfirstlane(upto);
    const int upto_max = __builtin_amdgcn_readlane(upto, 31);
    bf16x8 qf[ND];
    const uint16_t* qp = a.q + row * a.q_stride + (int64_t)head * a.head_dim;
#pragma unroll
    for (int s = 0; s < ND; ++s) {
      const int d = 16 * s + 8 * half;
      // chunks past the head's read its first one: their keys are zeros
      qf[s] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(qp + (d < a.head_dim ? d : 0)));
    }
    f32x16 o[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[t][x] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;
    for (int t = 0; t < nt; ++t) {
      if (t * kKeys > upto_max) break;
      attend_tile<DP>(tiles + t * T::kSize, qf, uniform64(tile_seen[t]), t * kKeys, upto, upto_min, upto_max, a.c,
                      lane, m, l, o);
    }
    l = swap_sum32(l);
    if (a.lse && half == 0 && live)
      a.lse[row * a.q_heads + head] = kLn2 * ((m == -__builtin_inff() ? m : m * a.c) + __builtin_amdgcn_logf(l));
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // an empty row: zeros
    // O^T holds a row's channels 8 g + 4 h + 0 .. 3 in half h: one exchange between the halves for each
    // pair of g makes them 16 bytes, channels 16 p + 8 h + 0 .. 7
    uint16_t* dst = a.out + row * a.out_stride + (int64_t)head * a.head_dim + 8 * half;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const u32x2 e = pack4(o[t], 8 * p, inv), f = pack4(o[t], 8 * p + 4, inv);
        const auto x = __builtin_amdgcn_permlane32_swap(e[0], f[0], false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(e[1], f[1], false, false);
        if (live && 32 * t + 16 * p + 8 * half < a.head_dim)
          *reinterpret_cast<u32x4*>(dst + 32 * t + 16 * p) = u32x4{x[0], y[0], x[1], y[1]};
      }
  }
}

// ---------------------------------------------------------------- few rows

// A workgroup owns up to 16 rows of one or two key heads; its four (or eight) waves take
// tiles of keys in turn (64 of one head, 32 of two), each with its own loads,
// softmax and O, and join at the end.  What bounds it is reading the cache:
//  - Every code is read once into registers, the next tile's while this one
//    is multiplied, and nothing looks at a loaded word before its use: a
//    select or a branch on it would wait there.  Table entries are asked for
//    two tiles ahead.
//  - Adjacent lanes read a key's part of the row (at head_dim 128 a lane reads
//    one MX block: 16 bytes and a scale byte), since loads are merged among
//    adjacent lanes only: in the operand order of v_mfma_f32_16x16x32_bf16
//    (lane l: key l % 16, the l / 16-th quarter of the channels) every lane
//    was an access of its own, 64 an instruction, and the address units, busy
//    80% of the time, were the bound (32 sequences of 8192 keys, 8 heads of
//    128: 97 us; 87 so).
//  - With two heads those reads are whole 128-byte lines: a compute unit has
//    about as many requests in flight either way, so twice the bytes (75 us,
//    3.9 TB/s; 256 sequences of 2048: 128 us, 4.5 TB/s, of the 5.1 to 5.9 that
//    a plain read of as much reaches).  Between 104 and 120 channels two
//    heads' tiles do not fit the registers (36 spilled, 491 us against 412
//    with one for 32 sequences of 8192 keys, 20 heads of 112).
// Keys change lanes as codes through LDS, values as bf16 for their
// transposition (32 keys at a time), both in wave-private memory, so no wave
// waits for another.  Key order within a 32-key step of the second product:
// index j of quarter g is key 4 g + j (j < 4) or 16 + 4 g + j - 4, the order
// S^T has.
constexpr int kTokenRows = 16, kTokenWaves = 4, kWideWaves = 8;
constexpr int64_t kTwoHeadKeys = int64_t(1) << 20;  // keys times heads from which a workgroup takes two heads

// Keys of one workgroup of a sequence that sees `see`: the smallest share
// (in tiles of 64) by which the batch's keys are at most a.chunks pieces, the
// workgroups of a group of heads that the GPU holds at once; so a ragged batch
// of up to 512 workgroups, undivided, is divided into equal pieces, in one
// round, whatever room its cache has.  More where the sequence has fewer ranges than that takes.  The same for
// every workgroup of the sequence.
__device__ __forceinline__ int token_share(const AttnArgs& a, int see, int unit, int lane) {
  int share = (see + a.nsplits - 1) / a.nsplits;
  if (a.nsplits > 1) {
    auto total = [&](auto&& of) {  // sum over the batch, 512 sequences at most: with 2^21 tiles each 2^30 in all
      unsigned n = 0;
      for (int i = lane; i < a.batch; i += 64)
        n += of(min((unsigned)(max(0, min(a.kv_len[i], a.capacity)) + 63) >> 6, 1u << 21));
#pragma unroll
      for (int x = 32; x; x >>= 1) n += __shfl_xor(n, x);
      return n;
    };
    const unsigned tiles = total([](unsigned t) { return t; }), most = (unsigned)a.chunks;
    const unsigned spare = (unsigned)max(a.chunks - a.batch, (a.chunks + 1) / 2);
    unsigned lo = max(1u, (tiles + most - 1) / most), hi = max(lo, (tiles + spare - 1) / spare);
#pragma unroll 1
    for (int it = 0; it < 8 && lo < hi; ++it) {
      const unsigned mid = (lo + hi) >> 1;
      const float inv = 1.0f / (float)mid;  // pieces need not be counted exactly
      if (total([&](unsigned t) { return (unsigned)ceilf((float)t * inv); }) <= most)
        hi = mid;
      else
        lo = mid + 1;
    }
    share = max(share, (int)min(hi, 1u << 24) * 64);
  }
  share = __builtin_amdgcn_readfirstlane(share);
  return (int)min(((int64_t)share + unit - 1) / unit * unit, (int64_t)1 << 30);
}

template <int DP, bool ALIGNED, int HEADS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void attn_tokens_kernel(AttnArgs a) {
  constexpr int NS = DP / 32, NO = DP / 16, NB = ALIGNED ? 1 : NS;
  constexpr int KEYS = 64 / HEADS, KT = KEYS / 16;  // keys of a wave's tile, and in operand tiles of 16
  constexpr int LANES = 4 * HEADS, STEP = 64 / LANES;  // lanes that read one key, keys that one load reads
  constexpr int VS = HEADS * DP + 16, OS = DP + 4;     // LDS row strides: values (elements), outputs (floats)
  constexpr int kVBytes = WAVES * 32 * VS * 2, kOBytes = WAVES * HEADS * kTokenRows * OS * 4;
  __shared__ __attribute__((aligned(16))) uint8_t shared[kVBytes > kOBytes ? kVBytes : kOBytes];
  __shared__ float wave_m[WAVES][HEADS][kTokenRows], wave_l[WAVES][HEADS][kTokenRows];

  const int tid = threadIdx.x, lane = tid & 63, quarter = lane >> 4, col = lane & 15;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroups are dealt to the eight XCDs in turn: the head groups of one sequence and range follow one
  // another on one XCD, sequences and ranges go round them (each range of a sequence on another); later
  // ranges, which a short sequence does not have, come last, so that the workgroups that do work are
  // spread evenly.
  const int head_groups = a.kv_heads / HEADS, turn = blockIdx.x >> 3;
  int id = turn / head_groups * 8 + (blockIdx.x & 7);
  const int units = a.batch * a.row_tiles, split = id / units;
  if (split >= a.nsplits) return;
  const int kvh0 = turn % head_groups * HEADS;
  id = (id % units + 3 * split) % units;
  const int tile = id % a.row_tiles, b = id / a.row_tiles;
  const Seq sq = sequence(a, b);
  const int rows = min(sq.nq, a.max_q) * a.group;
  const int r0 = tile * kTokenRows;
  if (r0 >= rows) return;

  const int last_q = (int)fast_div((unsigned)(min(r0 + kTokenRows, rows) - 1), a.by_group);
  const int see = a.causal ? max(0, min(sq.len, sq.len - sq.nq + last_q + 1)) : sq.len;
  const int share = token_share(a, see, KEYS * WAVES, lane);
  const int key0 = (int)min((int64_t)see, (int64_t)split * share), key1 = min(see, key0 + share);

  const int r = min(r0 + col, rows - 1);
  const int qi = (int)fast_div((unsigned)r, a.by_group);
  const int head = kvh0 * a.group + (r - qi * a.group);
  const int upto = a.causal ? sq.len - sq.nq + qi : sq.len;  // last key this lane's query sees
  const int upto_min = __builtin_amdgcn_readfirstlane(upto);

  const int nc = a.head_dim >> 3, chunk0 = kvh0 * nc;
  const int64_t width8 = (int64_t)a.kv_heads * nc;
  bf16x8 qf[HEADS][NS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    const uint16_t* qp = a.q + (sq.row0 + qi) * a.q_stride + (int64_t)(head + h * a.group) * a.head_dim;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int ch = quarter * NS + s;
      u32x4 w = {0, 0, 0, 0};
      if (ch < nc) w = *reinterpret_cast<const u32x4*>(qp + 8 * ch);
      qf[h][s] = __builtin_bit_cast(bf16x8, w);
    }
  }

  // One tile as it is loaded: codes and scales of keys STEP k + lane / LANES, head and quarter
  // lane % LANES.  Nothing may look at them before their use (a select here would wait for the loads): a
  // key that is not there reads slot 0 (always there) and is dealt with in multiply(); a quarter's chunks
  // past the head's read its first one (their queries are zero, and their channels of O are not stored).
  struct Tile {
    unsigned kw[4][NS], vw[4][NS];
    unsigned kb[4][NB], vb[4][NB];
    unsigned long long seen;
  };
  const int lkey = lane / LANES, lc = lane % LANES, lq = lc & 3;
  const int chunk = chunk0 + (lc >> 2) * nc;  // of the lane's head
  auto load = [&](int slot, Tile& t) {
    t.seen = __builtin_amdgcn_ballot_w64(slot >= 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = (int64_t)max(__shfl(slot, STEP * k + lkey), 0) * width8 + chunk;
      if constexpr (ALIGNED) {
        typedef __attribute__((ext_vector_type(NS))) unsigned words;
        const int64_t c = at + lq * NS;
        const words kw = *reinterpret_cast<const words*>(a.k_codes + 4 * c);
        const words vw = *reinterpret_cast<const words*>(a.v_codes + 4 * c);
        t.kb[k][0] = a.k_scales[c >> 2];
        t.vb[k][0] = a.v_scales[c >> 2];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          t.kw[k][s] = kw[s];
          t.vw[k][s] = vw[s];
        }
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const int64_t c = at + (lq * NS + s < nc ? lq * NS + s : 0);
          t.kw[k][s] = *reinterpret_cast<const unsigned*>(a.k_codes + 4 * c);
          t.kb[k][s] = a.k_scales[c >> 2];
          t.vw[k][s] = *reinterpret_cast<const unsigned*>(a.v_codes + 4 * c);
          t.vb[k][s] = a.v_scales[c >> 2];
        }
      }
    }
  };

  f32x4 o[HEADS][NO];
  float m[HEADS], l[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    m[h] = -__builtin_inff();
    l[h] = 0.0f;
#pragma unroll
    for (int t = 0; t < NO; ++t) o[h][t] = f32x4{0, 0, 0, 0};
  }
  uint16_t* vs = reinterpret_cast<uint16_t*>(shared) + wv * 32 * VS;

  auto multiply = [&](Tile& t, int key) {
    constexpr unsigned long long kAll = HEADS == 1 ? ~0ull : (1ull << (KEYS & 63)) - 1;
    const unsigned long long seen = t.seen & kAll;
    if (seen != kAll) {  // values that are not there: zeros, whatever the slot holds
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (!((seen >> (STEP * k + lkey)) & 1)) {
#pragma unroll
          for (int s = 0; s < NS; ++s) t.vw[k][s] = 0;
#pragma unroll
          for (int s = 0; s < NB; ++s) t.vb[k][s] = 0;
        }
    }
    // keys from the lanes that loaded them to the operand's: codes through LDS (pieces swizzled against
    // bank conflicts), scale bytes, four to a register, by one permute
    unsigned scales[HEADS][NB];
    unsigned* kx = reinterpret_cast<unsigned*>(vs);
    auto swizzle = [](int k) { return HEADS == 1 ? (k >> 1) & 3 : k & (LANES - 1); };
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      const unsigned w = t.kb[0][x] | (t.kb[1][x] << 8) | (t.kb[2][x] << 16) | (t.kb[3][x] << 24);
#pragma unroll
      for (int h = 0; h < HEADS; ++h)
        scales[h][x] = (unsigned)__shfl((int)w, col % STEP * LANES + 4 * h + quarter);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int d = 0; d < NS; ++d)
        kx[((STEP * k + lkey) * LANES + (lc ^ swizzle(STEP * k + lkey))) * NS + d] = t.kw[k][d];
    wave_lds_fence();
    f32x4 s[HEADS][KT];
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        // key 16 k + col was byte (16 k + col) / STEP of its lane
        const unsigned shift = 8 * ((16 / STEP) * k + col / STEP);
        s[h][k] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < NS; ++d)
          s[h][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              mx_values8(kx[((16 * k + col) * LANES + ((4 * h + quarter) ^ swizzle(16 * k + col))) * NS + d],
                         (scales[h][ALIGNED ? 0 : d] >> shift) & 0xFF),
              qf[h][d], s[h][k], 0, 0, 0);
      }
    wave_lds_fence();
    if (seen != kAll || upto_min < key + KEYS - 1) {
      const unsigned long long mine = seen >> (4 * quarter);
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (!((mine >> (16 * k + x)) & 1) || key + 16 * k + 4 * quarter + x > upto) {
#pragma unroll
            for (int h = 0; h < HEADS; ++h) s[h][k][x] = -__builtin_inff();
          }
    }
    bf16x8 p[HEADS][KT / 2];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      float top = s[h][0][0];
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) top = fmaxf(top, s[h][k][x]);
      if (__builtin_amdgcn_ballot_w64(top > m[h]) != 0) {  // some query has a new maximum
        const unsigned u = __float_as_uint(top);
        const auto y = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const float mn = fmaxf(m[h], swap_max32(fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]))));
        const float alpha = mn > m[h] ? __builtin_amdgcn_exp2f((m[h] - mn) * a.c) : 1.0f;
        l[h] *= alpha;
#pragma unroll
        for (int d = 0; d < NO; ++d) o[h][d] *= alpha;
        m[h] = mn;
      }
      const float base = m[h] == -__builtin_inff() ? 0.0f : m[h] * a.c;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[h][k][x], a.c, -base));
          sum += e;
          p[h][k >> 1][4 * (k & 1) + x] = (__bf16)e;
        }
      l[h] += sum;
    }
    typedef __attribute__((address_space(3))) s16x4 lds4;
#pragma unroll
    for (int part = 0; part < KT / 2; ++part) {  // 32 keys
#pragma unroll
      for (int k = 0; k < 32 / STEP; ++k)
#pragma unroll
        for (int d = 0; d < NS; ++d)
          *reinterpret_cast<bf16x8*>(&vs[(STEP * k + lkey) * VS + (lc >> 2) * DP + 8 * (lq * NS + d)]) =
              mx_values8(t.vw[32 / STEP * part + k][d], t.vb[32 / STEP * part + k][ALIGNED ? 0 : d]);
      wave_lds_fence();
#pragma unroll
      for (int h = 0; h < HEADS; ++h) {
        const uint16_t* at = vs + (4 * quarter + (col >> 2)) * VS + h * DP + 4 * (col & 3);
#pragma unroll
        for (int d = 0; d < NO; ++d) {
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 16 * d));
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 16 * VS + 16 * d));
          const bf16x8 w = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
          o[h][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, p[h][part], o[h][d], 0, 0, 0);
        }
      }
      wave_lds_fence();
    }
  };

  // tiles wv, wv + 4, ... of the range: the next tile's codes are in flight during this one's
  // product, and the slots of the one after, asked for before those codes (loads return in order:
  // behind them, waiting for a slot would wait for the codes too)
  constexpr int kStep = KEYS * WAVES;
  int key = key0 + KEYS * wv;
  if (key < key1) {
    Tile even, odd;
    auto entry = [&](int k) { return page_entry(a, b, k + lane % KEYS); };
    auto slot = [&](int k, int e) { return slot_of(a, b, k + lane % KEYS, e, key1); };
    int e0 = entry(key), e1 = entry(key + kStep);
    load(slot(key, e0), even);
    for (;; key += 2 * kStep) {
      e0 = entry(key + 2 * kStep);
      load(slot(key + kStep, e1), odd);
      multiply(even, key);
      if (key + kStep >= key1) break;
      e1 = entry(key + 3 * kStep);
      load(slot(key + 2 * kStep, e0), even);
      multiply(odd, key + kStep);
      if (key + 2 * kStep >= key1) break;
    }
  }

  // join the waves
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    const float sum = quarter_sum(l[h]);
    if (quarter == 0) {
      wave_m[wv][h][col] = m[h];
      wave_l[wv][h][col] = sum;
    }
  }
  __syncthreads();  // also: every wave is done with its tile of values
  float* os = reinterpret_cast<float*>(shared);
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    float top = wave_m[0][h][col];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) top = fmaxf(top, wave_m[w][h][col]);
    const float mine = m[h] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((m[h] - top) * a.c);
#pragma unroll
    for (int d = 0; d < NO; ++d)
      *reinterpret_cast<f32x4*>(&os[((wv * HEADS + h) * kTokenRows + col) * OS + 16 * d + 4 * quarter]) = o[h][d] * mine;
  }
  __syncthreads();
  for (int x = tid; x < HEADS * kTokenRows * nc; x += 64 * WAVES) {
    const int hq = x / nc, ch = x - hq * nc, hw = hq / kTokenRows, q = hq % kTokenRows;
    if (r0 + q >= rows) continue;
    float best = wave_m[0][hw][q];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) best = fmaxf(best, wave_m[w][hw][q]);
    float sum = 0.0f;
    f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float wm = wave_m[w][hw][q], wl = wave_l[w][hw][q];
      // a wave that saw no key is known by its sum: one whose scores are all NaN keeps the maximum -inf too
      sum += wl == 0.0f ? 0.0f : wl * __builtin_amdgcn_exp2f((wm - best) * a.c);
      const f32x4* src = reinterpret_cast<const f32x4*>(&os[((w * HEADS + hw) * kTokenRows + q) * OS + 8 * ch]);
      lo += src[0];
      hi += src[1];
    }
    const int qx = (int)fast_div((unsigned)(r0 + q), a.by_group);
    const int h = (kvh0 + hw) * a.group + (r0 + q - qx * a.group);
    const int64_t row = sq.row0 + qx;
    const float base = best == -__builtin_inff() ? best : best * a.c;
    if (a.nsplits > 1) {
      const int64_t n = a.q_rows * a.q_heads, at = split * n + row * a.q_heads + h;
      if (ch == 0) {
        float* ml = a.part + (int64_t)a.nsplits * n * a.head_dim + 2 * at;
        ml[0] = base;
        ml[1] = sum;
      }
      if (sum == 0.0f) continue;  // the join reads no output of an empty range
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

// The ranges' outputs weighted by exp2(max_s - max).  Sixteen lanes hold a
// row's channels, eight each; `slices` such groups share a row's ranges (one
// lane group reading 64 of them in turn took longer than the attention), and
// meet in LDS in slice order.
constexpr int kJoinThreads = 256;

template <bool FEW>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a, int slices) {
  __shared__ float part[kJoinThreads][11];  // maximum, sum, eight channels, and a pad against bank conflicts
  const int tid = threadIdx.x, lane = tid & 15, group = tid >> 4, slice = group % slices;
  const int64_t i = (int64_t)blockIdx.x * (kJoinThreads / 16 / slices) + group / slices;
  // the row's place in the output, and its partial results: the first one, and how far to the next
  int b, qi, head;
  bool live;
  int64_t first, next, total;
  if constexpr (FEW) {  // i: query and head of sequence blockIdx.y; results by range, row and head
    b = blockIdx.y;
    qi = (int)(i / a.q_heads);
    head = (int)(i - (int64_t)qi * a.q_heads);
    live = i < (int64_t)a.max_q * a.q_heads;
  } else {  // i: row of the divided tiles; results by tile, range and row
    const int index = (int)(i / kRowsTile), lr = (int)(i % kRowsTile);
    const RowsWork w = rows_work(a, a.whole + min(index, a.split_tiles - 1));
    const int r = w.tile * kRowsTile + lr;
    b = w.b;
    qi = (int)fast_div((unsigned)r, a.by_group);
    head = w.kvh * a.group + (r - qi * a.group);
    live = index < a.split_tiles && qi < a.max_q;
    first = (int64_t)index * a.nsplits * kRowsTile + lr;
    next = kRowsTile;
    total = (int64_t)a.split_tiles * a.nsplits * kRowsTile;
  }
  const Seq sq = sequence(a, b);
  live = live && qi < sq.nq && 8 * lane < a.head_dim;
  const int64_t at = (sq.row0 + qi) * a.q_heads + head;
  if constexpr (FEW) {
    first = at;
    next = a.q_rows * a.q_heads;
    total = a.nsplits * next;
  }
  const float* ml = a.part + total * a.head_dim;
  float top = -__builtin_inff(), sum = 0.0f, o[8] = {};
  if (live)
#pragma unroll 4
    for (int s = slice; s < a.nsplits; s += slices) {
      const int64_t x0 = first + s * next;
      const float ms = ml[2 * x0], ls = ml[2 * x0 + 1];
      const f32x4* src = reinterpret_cast<const f32x4*>(a.part + x0 * a.head_dim + 8 * lane);
      const f32x4 x = src[0], y = src[1];
      const bool there = ls != 0.0f;  // an empty range: its output was not written (loaded all the same, not to wait here)
      const float t = there ? fmaxf(top, ms) : top;
      const float keep = top == t ? 1.0f : __builtin_amdgcn_exp2f(top - t), w = there ? __builtin_amdgcn_exp2f(ms - t) : 0.0f;
      top = t;
      sum = sum * keep + w * ls;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[k] = o[k] * keep + (there ? w * x[k] : 0.0f);
        o[4 + k] = o[4 + k] * keep + (there ? w * y[k] : 0.0f);
      }
    }
  if (slices > 1) {
    part[tid][0] = top;
    part[tid][1] = sum;
#pragma unroll
    for (int k = 0; k < 8; ++k) part[tid][2 + k] = o[k];
    __syncthreads();
    if (slice != 0) return;
    for (int s = 1; s < slices; ++s) top = fmaxf(top, part[tid + 16 * s][0]);
    const float own = sum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(part[tid][0] - top);
    sum *= own;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] *= own;
    for (int s = 1; s < slices; ++s) {
      const float* p = part[tid + 16 * s];
      if (p[1] == 0.0f) continue;
      const float w = __builtin_amdgcn_exp2f(p[0] - top);
      sum += w * p[1];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] += w * p[2 + k];
    }
  }
  if (!live) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (a.lse && lane == 0) a.lse[at] = kLn2 * (top + __builtin_amdgcn_logf(sum));
  bf16x8 w;
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = (__bf16)(o[k] * inv);
  *reinterpret_cast<u32x4*>(a.out + (sq.row0 + qi) * a.out_stride + (int64_t)head * a.head_dim + 8 * lane) =
      __builtin_bit_cast(u32x4, w);
}

const void* rows_kernel(int d) {
  if (d == 32) return (const void*)&attn_rows_kernel<32, true>;
  if (d == 64) return (const void*)&attn_rows_kernel<64, true>;
  if (d == 128) return (const void*)&attn_rows_kernel<128, true>;
  return d < 32   ? (const void*)&attn_rows_kernel<32, false>
         : d < 64 ? (const void*)&attn_rows_kernel<64, false>
         : d <= 96 ? (const void*)&attn_rows_kernel<96, false>
                   : (const void*)&attn_rows_kernel<128, false>;
}

const void* resident_kernel(int d) {
  if (d == 32) return (const void*)&attn_resident_kernel<32, true>;
  if (d == 64) return (const void*)&attn_resident_kernel<64, true>;
  if (d == 128) return (const void*)&attn_resident_kernel<128, true>;
  return d < 32   ? (const void*)&attn_resident_kernel<32, false>
         : d < 64 ? (const void*)&attn_resident_kernel<64, false>
         : d <= 96 ? (const void*)&attn_resident_kernel<96, false>
                   : (const void*)&attn_resident_kernel<128, false>;
}

template <int HEADS, int WAVES>
const void* tokens_kernel(int d) {
  if (d == 32) return (const void*)&attn_tokens_kernel<32, true, HEADS, WAVES>;
  if (d == 64) return (const void*)&attn_tokens_kernel<64, true, HEADS, WAVES>;
  if (d == 128) return (const void*)&attn_tokens_kernel<128, true, HEADS, WAVES>;
  if (d < 32) return (const void*)&attn_tokens_kernel<32, false, HEADS, WAVES>;
  if (d < 64) return (const void*)&attn_tokens_kernel<64, false, HEADS, WAVES>;
  // two heads of 104 to 120 channels do not fit the registers
  if constexpr (HEADS == 1)
    if (d > 96) return (const void*)&attn_tokens_kernel<128, false, HEADS, WAVES>;
  return (const void*)&attn_tokens_kernel<96, false, HEADS, WAVES>;
}

}  // namespace

// Few rows: up to two 16-row tiles for each sequence and key head.  Their
// workgroups take two key heads where the call reads enough keys (the two
// read the same cache lines together), else one, so that a short context is
// spread over waves.  Many: 256-row tiles, or row tiles of a size chosen below
// where the keys fit LDS.
AttnPlan attn_plan(int64_t batch, int64_t max_q, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                   int64_t capacity) {
  AttnPlan p{};
  const int64_t rows = max_q * (q_heads / kv_heads);
  p.few = rows <= 2 * kTokenRows;
  const int tile = p.few ? kTokenRows : kRowsTile;
  p.row_tiles = (int)((rows + tile - 1) / tile);
  p.wg_heads = 1;
  if (p.few) {
    const int64_t tiles = batch * kv_heads * p.row_tiles;
    p.wg_heads = kv_heads % 2 == 0 && (head_dim <= 96 || head_dim == 128) && tiles * capacity >= kTwoHeadKeys ? 2 : 1;
    const int64_t wgs = tiles / p.wg_heads, unit = 64 / p.wg_heads * kTokenWaves;
    // Ranges of a sequence: up to one workgroup a compute unit as long as a wave has a tile, up to the two
    // that fit while it has four; none below eight tiles a wave, where the join and its launch cost as much
    // (1023 keys of one sequence 10.6 us whole, 11.4 in four ranges, called from Python 9.7 and 13.6; of 32
    // sequences 14 whole, 20 in two; 2048 keys of one 17 whole, 11.2 in eight).  Twice as many may be
    // launched, for the longest sequences of a ragged batch.  Above 512 workgroups, so above 512 sequences,
    // nothing is divided.
    const int64_t steps = capacity / unit;
    const int64_t each = steps < 8 ? 1 : std::max(std::min(256 / wgs, steps), std::min(512 / wgs, steps / 4));
    p.nsplits = steps < 8 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>({2 * each, steps, 64}));
    // Eight waves where that many keys are not divided and the GPU has room: 1023 keys of one sequence, 32 heads
    // over 8, 10.6 us and 11.6 (called from Python 9.7 and 11.0); at a workgroup for every compute unit 32
    // sequences take 14.6 and 14.3.
    p.wide = p.nsplits == 1 && p.wg_heads == 1 && wgs <= 128 && capacity > 64 * kTokenWaves;
    p.chunks = (int)(std::max<int64_t>(1, each) * batch);
  } else if (capacity <= kKeys * resident_tiles((int)head_dim)) {
    // One workgroup fits a compute unit.  Of the row tiles that fill one to four rounds of workgroups, the
    // number whose rounds take the least time, in units of what `waves` groups of 32 rows take together:
    // kStage of it for the keys, and for a last part of the groups less than its share of the waves saves,
    // since each then has more of its SIMD.  Against runs of `waves` groups, several where that leaves 384
    // workgroups: 4 x 4096 rows of 16 heads of 96 over 300 keys 46.4 us and 62.2, 300 rows of one sequence
    // 11.4 and 17.3, 2 x 4608 rows of 24 heads of 128 over 256 keys 47.6 and 52.6.
    constexpr double kStage = 0.35, kAlone = 0.4;
    const int64_t waves = resident_waves((int)head_dim), seqs = batch * kv_heads, groups = (rows + 31) / 32;
    double least = 0;
    for (int64_t round = (seqs + 255) / 256, end = round + 4; round < end; ++round) {
      const int64_t n = std::max<int64_t>(1, std::min(groups, 256 * round / seqs)), each = (groups + n - 1) / n, rest = each % waves;
      const double time = round * (kStage + each / waves + (rest ? kAlone + (1 - kAlone) * rest / waves : 0));
      if (p.run_groups == 0 || time < least) p.run_groups = (int)each, least = time;
    }
    p.row_tiles = (int)((groups + p.run_groups - 1) / p.run_groups);
    p.nsplits = 1;
    p.whole = (int)(seqs * p.row_tiles);
    p.by_xcd = batch * p.row_tiles % 8 == 0;
  } else {
    const int64_t tiles = batch * kv_heads * p.row_tiles, slots = 256;  // one workgroup a compute unit
    const int64_t rest = tiles % slots;
    p.nsplits = rest == 0 ? 1 : (int)std::max<int64_t>(1, std::min(slots / rest, capacity / (2 * kKeys)));
    p.split_tiles = p.nsplits > 1 ? (int)rest : 0;
    p.whole = (int)(tiles - p.split_tiles);
  }
  return p;
}

int64_t attn_workspace(int64_t q_rows, int64_t q_heads, int64_t head_dim, const AttnPlan& p) {
  if (p.nsplits <= 1) return 0;
  return p.nsplits * (p.few ? q_rows * q_heads : (int64_t)p.split_tiles * kRowsTile) * (head_dim + 2) * 4;
}

AttnLaunch attn_launch(int64_t batch, int64_t kv_heads, int64_t head_dim, const AttnPlan& p) {
  AttnLaunch l{};
  l.grid = p.few ? (batch * p.row_tiles * p.nsplits + 7) / 8 * 8 * (kv_heads / p.wg_heads)
                 : p.whole + (int64_t)p.split_tiles * p.nsplits;
  l.threads = 64 * (p.run_groups ? resident_waves((int)head_dim) : p.wide ? kWideWaves : p.few ? kTokenWaves : kRowsWaves);
  return l;
}

hipError_t launch_attn(const AttnArgs& args, hipStream_t stream) {
  AttnArgs a = args;
  a.group = a.q_heads / a.kv_heads;
  a.by_page = make_divisor((unsigned)a.page_size);
  a.by_group = make_divisor((unsigned)a.group);
  a.capacity = a.n_pages > 0 ? a.pages_per_seq * a.page_size : 0;
  if (a.pages_per_seq == 0) a.table = nullptr;  // no entry that page_entry could read
  a.c = a.scale * kLog2e;
  const AttnPlan p =
      attn_plan(a.batch, a.max_q, a.q_heads, a.kv_heads, a.head_dim, (int64_t)a.pages_per_seq * a.page_size);
  a.nsplits = p.nsplits;
  a.chunks = p.chunks;
  a.whole = p.whole;
  a.split_tiles = p.split_tiles;
  a.run_groups = p.run_groups;
  a.by_xcd = p.by_xcd;
  a.row_tiles = p.row_tiles;
  void* kargs[] = {&a};
  const AttnLaunch l = attn_launch(a.batch, a.kv_heads, a.head_dim, p);
  const hipError_t e =
      hipLaunchKernel(p.run_groups      ? resident_kernel(a.head_dim)
                      : !p.few          ? rows_kernel(a.head_dim)
                      : p.wg_heads == 2 ? tokens_kernel<2, kTokenWaves>(a.head_dim)
                      : p.wide          ? tokens_kernel<1, kWideWaves>(a.head_dim)
                                        : tokens_kernel<1, kTokenWaves>(a.head_dim),
                      dim3((unsigned)l.grid), dim3(l.threads), kargs, 0, stream);
  if (e != hipSuccess || a.nsplits == 1) return e;
  int slices = 1;
  // two ranges a lane (few rows) or four, all in flight: 16384 keys of one sequence 17.0 us, 18.0 one by one
  while (slices < 16 && (p.few ? 2 : 4) * slices < a.nsplits) slices *= 2;
  const int64_t per = kJoinThreads / 16 / slices;
  const int64_t pairs = p.few ? (int64_t)a.max_q * a.q_heads : (int64_t)a.split_tiles * kRowsTile;
  void* jargs[] = {&a, &slices};
  return hipLaunchKernel(p.few ? (const void*)&attn_join_kernel<true> : (const void*)&attn_join_kernel<false>,
                         dim3((unsigned)((pairs + per - 1) / per), p.few ? (unsigned)a.batch : 1u), dim3(kJoinThreads),
                         jargs, 0, stream);
}

}  // namespace kq
