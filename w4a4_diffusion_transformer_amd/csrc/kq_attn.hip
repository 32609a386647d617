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

}  // namespace

int attn_splits(int64_t batch, int64_t max_q, int64_t q_heads, int64_t kv_heads, int64_t capacity) {
  const int64_t tiles = batch * kv_heads * ((max_q * (q_heads / kv_heads) + kRowsTile - 1) / kRowsTile);
  const int64_t want = tiles > 0 ? 512 / tiles : 1, most = capacity / 128;
  return (int)std::max<int64_t>(1, std::min(want, most));
}

int64_t attn_workspace(int64_t q_rows, int64_t q_heads, int64_t head_dim, int nsplits) {
  return nsplits > 1 ? nsplits * q_rows * q_heads * (head_dim + 2) * 4 : 0;
}

hipError_t launch_attn(const AttnArgs& args, int nsplits, hipStream_t stream) {
  AttnArgs a = args;
  a.group = a.q_heads / a.kv_heads;
  a.by_page = make_divisor((unsigned)a.page_size);
  a.by_group = make_divisor((unsigned)a.group);
  a.capacity = a.n_pages > 0 ? a.pages_per_seq * a.page_size : 0;
  a.c = a.scale * kLog2e;
  a.nsplits = nsplits;
  a.row_tiles = (int)(((int64_t)a.max_q * a.group + kRowsTile - 1) / kRowsTile);
  void* kargs[] = {&a};
  const int64_t grid = (int64_t)a.batch * a.kv_heads * a.row_tiles * a.nsplits;
  const hipError_t e = hipLaunchKernel(rows_kernel(a.head_dim), dim3((unsigned)grid), dim3(64 * kRowsWaves), kargs, 0, stream);
  if (e != hipSuccess || a.nsplits == 1) return e;
  const int64_t per = (int64_t)a.max_q * a.q_heads * (a.head_dim >> 3);
  return hipLaunchKernel((const void*)&attn_join_kernel, dim3((unsigned)((per + 255) / 256), (unsigned)a.batch),
                         dim3(256), kargs, 0, stream);
}

}  // namespace kq
