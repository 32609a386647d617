// Internal launch interface between the C ABI layer and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kq {

enum { KSRC_PARAMS = 0, KSRC_SPLIT = 1 };

// Tile decomposition of the MFMA kernels: a workgroup of eight waves owns a
// column group of 8 blocks (512 B of each bf16 row; each wave one block,
// whose K operands stay in its registers) and processes tiles of 32 rows.
// The grid has two parts.  The first w1 = ngroups * nchunks workgroups fill
// the GPU once: workgroup (group g, chunk c) takes row tiles c, c + nchunks,
// ... below r1.  The rest take the tiles from r1 on, n2 consecutive tiles
// each; the hardware dispatcher starts them on whichever compute units
// finish their first-part work first, which evens out the finish times.
struct MfmaArgs {
  const uint16_t* X;
  int T, d, nb;
  const float* P;  // [nb][15] or one set (pstride 0)
  int pstride;
  const uint16_t* Kbf;  // [nb][3][32][32] transposed split
  int kstride;          // 3072 or 0
  uint8_t* codes;
  uint8_t* scales;
  float* Y;  // diagnostic output or nullptr
  // AdaLN producer step (the MOD kernels): row (mean, rstd) pairs or nullptr,
  // per-sample fp32 scale and shift [samples][d] or nullptr, rows per sample
  const float* stats;
  const float* mscale;
  const float* mshift;
  int tps;
  int ngroups, nchunks;
  int w1, r1, n2;  // second part of the grid: see above
  // requested grid shape: size of the second part (percent of the tiles,
  // tiles per workgroup) and workgroups per CU the first part is sized for;
  // -1: the built-in rule.  The results do not depend on it, only the time.
  int req_tail_pct = -1, req_n2 = -1, req_wg_per_cu = -1;
};

// Row-segment decomposition of the vector-ALU kernels: a workgroup of four
// waves owns a column group of 16 blocks (1 KB of each bf16 row); each lane
// owns one fixed 16-byte piece (8 channels) of it, so every wave instruction
// reads 1 KB and writes 256 code bytes and 16 scale bytes, all contiguous.
// Rows go in blocks of four (one per wave); workgroup (group g, chunk c)
// takes row blocks c, c + nchunks, c + 2 nchunks, ...
struct QuadArgs {
  const uint16_t* X;
  int T, d, nb;
  const float* P;
  int pstride;
  const float* m;  // channel multipliers (SmoothQuant front-end)
  uint8_t* codes;
  uint8_t* scales;
  float* Y;
  int ngroups, nchunks;
};

// Block-per-lane decomposition of the vector-ALU kernels: X as a flat
// sequence of 64-byte blocks, a wave per unit of 64 consecutive blocks (one
// per lane, staged through a wave-private LDS region), each wave visiting
// units a whole number of rows apart so that each lane keeps one block
// column.  Set by launch_flat: nblocks, xbytes, units, phases, chunks.
struct FlatArgs {
  const uint16_t* X;
  int T, nb;
  const float* P;
  int pstride;
  const float* m;  // channel multipliers (SmoothQuant front-end)
  uint8_t* codes;
  uint8_t* scales;
  float* Y;
  // FRONT_ADALN: per-row (mean, rstd) [T][2] (null: 0, 1), (1 + scale) and shift vectors
  // [samples][d] (null: scale 0, shift -0), rows per sample (>= T: one sample)
  const float* stats = nullptr;
  const float* mscale = nullptr;
  const float* mshift = nullptr;
  int64_t tps = 0;
  int64_t nblocks, xbytes, units;
  int phases, chunks;
  int rows_step;      // set by launch_flat: rows between a lane's consecutive blocks
  int req_waves = 0;  // requested total waves (tuning; 0: one resident round)
  int hlog = 5;       // FRONT_HADAMARD_WIDE: log2 of the Hadamard block (6 .. 9)
  float hscale = 0.0f;  // and 1 / sqrt(block) in fp32
};

// Compute units of the current device (cached per device).
int cu_count();
// Workgroups of `fn` (block_threads threads, no dynamic LDS) resident per
// compute unit, from the occupancy calculator, cached per kernel and device;
// capped by the KQ_WG_PER_CU tuning override when set.
int resident_per_cu(const void* fn, int block_threads);
// Row chunks so that ngroups x nchunks workgroups fill the machine exactly
// once (no second, partial round), with at least one row tile per chunk.
int chunks_one_round(const void* fn, int block_threads, int ngroups, int ntiles, int wg_per_cu_cap = 0);

hipError_t launch_mfma(int ksrc, bool store_y, bool mod, const MfmaArgs& args, hipStream_t stream);
hipError_t launch_quad(int front, bool store_y, const QuadArgs& args, hipStream_t stream);
hipError_t launch_flat(int front, bool store_y, const FlatArgs& args, hipStream_t stream);
// Division of 31-bit numbers by a run-time constant (kq_mxval.hpp, fast_div).
struct Divisor {
  uint32_t m;
  int shift;
};

inline Divisor make_divisor(unsigned d) {
  int l = 0;
  while ((1u << l) < d) ++l;
  return Divisor{(uint32_t)(((uint64_t)1 << (31 + l)) / d + 1), 31 + l};  // m <= 2^32 - 2^8 for d <= 2^24
}

// What kq_gemm_mx_ex does to each fp32 sum: (residual + gate[sample] * act(sum + bias)); null: left out.
struct Epilogue {
  bool on = false;  // any of it
  int act = 0;      // kq_act
  const float* bias = nullptr;
  const float* gate = nullptr;  // [samples][N]
  Divisor by_rows{};            // rows of a sample
  const uint16_t* residual = nullptr;
};

// W4A4 GEMM: Y [M][N] = deq(A) deq(B)^T, A [M][K] and B [N][K] in MXFP4
// (codes [rows][K/2], E8M0 scales [rows][K/32]); either output may be null.
struct GemmArgs {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  int M, N, K;
  float* y_f32;
  uint16_t* y_bf16;
  Epilogue epi;
  int full_tiles;  // set by launch_gemm: tiles computed whole; the rest in two halves
  int tile_mi;     // set by launch_gemm: rows of a tile / 64
};

// MXFP4 key/value cache, write or read: rows of 8 * chunks channels, slots
// [tokens], pools of n_slots rows.  Strides in elements.
struct CacheArgs {
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* k_out;
  uint16_t* v_out;
  int64_t k_stride, v_stride;
  const int32_t* slots;
  int64_t tokens;
  int n_slots;
  int chunks;
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  Divisor by_chunks;  // set by launch_cache
};

// Rows of heads, normalised and turned (kq_rope.hip).  Strides in elements.
struct RopePart {  // queries (or any rows), keys or values of a call; heads 0: none
  const uint16_t* x;
  int64_t x_stride;
  uint16_t* out;  // rows, or
  int64_t out_stride;
  uint8_t* codes;  // the pools of a cache (null: rows)
  uint8_t* scales;
  const float* weight;  // of the norm, [head_dim] (null: 1)
  int heads;
  bool turn;  // false: taken as they are (values)
  // set by launch_rope: tokens and heads of a wave, waves of a wave's tokens, waves in all
  int tokens, per, chunks;
  int64_t waves;
};

struct RopeArgs {
  RopePart part[3];
  int64_t tokens;
  int head_dim;
  bool norm;
  double eps;
  const int32_t* positions;  // [tokens][n_axes]
  const double* freqs;       // [pairs]
  int n_axes;                // 0: nothing turns
  int axis_end[4];           // the pair after an axis' last; `pairs` for the last axis and past it
  int pairs;
  bool halves;
  const int32_t* slots;
  int n_slots;
  // set by launch_rope
  int64_t waves, first_wave;
  Divisor by_value_chunks;  // pieces of a row of values
  double inv_dim;
};

// The residual stream between two blocks (kq_norm.hip).  Strides in elements; norms 0 none, 1 RMS, 2 layer.
struct NormArgs {
  const uint16_t* x;
  const uint16_t* y;  // null: x is the stream already
  uint16_t* x_out;
  int64_t x_stride, y_stride, x_out_stride;
  int64_t tokens;
  int d;
  int post, pre;
  const float* post_w;
  const float* gate;  // [samples][d]
  double residual_scale;
  const float* pre_w;
  const float* mod_scale;  // [samples][d]
  const float* mod_shift;
  int64_t sample_rows;  // rows of a sample
  Divisor by_sample;
  double eps;
  bool next;    // any of the outputs below
  uint16_t* h;  // may be null, as the others
  int64_t h_stride;
  uint8_t* codes;
  uint8_t* scales;
  float* stats;
  // set by launch_residual_norm: consecutive rows of a workgroup
  int64_t group_rows;
  double inv_d;
};

// Attention over the cache: see kq_attn.hip.  Strides in elements.
struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride, q_rows;
  const int32_t* q_start;  // [batch + 1], or null: max_q rows per sequence
  int batch, max_q;
  const uint8_t* k_codes;
  const uint8_t* k_scales;
  const uint8_t* v_codes;
  const uint8_t* v_scales;
  int n_pages;
  const int32_t* table;  // [batch][pages_per_seq], or null: pages in order
  int pages_per_seq, page_size;
  const int32_t* kv_len;
  int q_heads, kv_heads, head_dim;
  float scale;
  int causal;
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  float* part;  // workspace of a split launch
  // set by the launch
  Divisor by_page, by_group;
  int capacity, group, row_tiles, nsplits, chunks, whole, split_tiles, run_groups;
  bool by_xcd;
  float c;  // scale * log2(e)
};

// How a call is divided: the kernel for few rows or the one for many, tiles of rows, and ranges of keys (more than
// one: partial results in a workspace, joined by a second launch).
struct AttnPlan {
  bool few;
  int row_tiles, nsplits;
  int wg_heads;  // key heads of a workgroup
  bool wide;     // few: workgroups of eight waves, not four
  int chunks;    // few: key ranges of the whole batch, for each group of heads
  int whole, split_tiles;  // many: tiles that are not divided, and the others
  int run_groups;          // many, with all keys in LDS: 32-row groups of a workgroup (its row tile); else 0
  bool by_xcd;             // of those: every head of a row tile on one XCD (row tiles of the batch: a multiple of 8)
};

// batch and max_q at least 1.
AttnPlan attn_plan(int64_t batch, int64_t max_q, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                   int64_t capacity);
// The first launch of a call so divided.
struct AttnLaunch {
  int64_t grid;
  int threads;
};
AttnLaunch attn_launch(int64_t batch, int64_t kv_heads, int64_t head_dim, const AttnPlan& plan);
int64_t attn_workspace(int64_t q_rows, int64_t q_heads, int64_t head_dim, const AttnPlan& plan);
hipError_t launch_attn(const AttnArgs& args, hipStream_t stream);

hipError_t launch_cache(bool write, bool both, const CacheArgs& args, hipStream_t stream);
hipError_t launch_rope(const RopeArgs& args, hipStream_t stream);
hipError_t launch_residual_norm(const NormArgs& args, hipStream_t stream);
hipError_t launch_gemm(const GemmArgs& args, hipStream_t stream);
// The same for few rows (kq_gemm_rows.hip).
hipError_t launch_gemm_rows(const GemmArgs& args, hipStream_t stream);
hipError_t launch_row_stats(const uint16_t* X, int T, int d, double eps, float* stats, hipStream_t stream);
hipError_t launch_build(const float* P, int nb, float* K32, uint16_t* Kbf, int n_split, int inverse_t,
                        hipStream_t stream);
hipError_t launch_build16(const float* P16, int nb, float* K32, uint16_t* Kbf, int n_split, hipStream_t stream);

}  // namespace kq
