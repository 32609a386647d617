// MXFP4 key/value cache: rows quantized as they are written to their slots,
// and slots read back as the bf16 values they stand for.
//
// A cache is four pools (codes and scales of keys and of values) whose row s
// is slot s in the quantizer's own output format: codes [slots][W/2], E8M0
// scales [slots][W/32], W = kv_heads * head_dim.  Both directions are
// streams with one gather: the slot of a row is looked up, everything else
// is contiguous.
//
// Mathematics.  Writing: byte = max(floor(log2 amax) - 2 + 127, 0) over each
// 32 channels and code = E2M1(x / 2^(byte - 127)), the shared epilogue of the
// quantizers.  Reading: E2M1(code) * 2^(byte - 127), which bf16 holds exactly
// (two significant bits, fp32's exponent range) for every byte the library
// writes (0 .. 252: checked on MI355X for all 16 codes of each), so nothing is
// rounded.
//
// Layout.  The rows of one tensor are a flat sequence of 8-channel chunks (16
// bytes of bf16, 4 of codes); a lane takes one chunk, four lanes a block.  A
// wave instruction then moves 1 KB of bf16 and 256 bytes of codes, both
// contiguous within a row whatever its width, and a workgroup's first chunk
// gives its first row by one scalar division.
//
// What bounds it: HBM.  40961 rows of 8 heads of 128 written and read back
// take 74.5 us (5.1 TB/s, the rate of a copy).  Few rows: the launch, 2.6 us.
#include "kq_device.hpp"
#include "kq_internal.h"
#include "kq_mxval.hpp"

namespace kq {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;  // chunks per lane, all in flight at once

// One workgroup moves kThreads * kUnits consecutive chunks of one tensor
// (blockIdx.y: 0 keys, 1 values).  Calls body(k, row, chunk, live) per unit.
template <class Body>
__device__ __forceinline__ void for_chunks(const CacheArgs& a, Body&& body) {
  const int64_t base = (int64_t)blockIdx.x * (kThreads * kUnits);
  const int64_t row0 = base / a.chunks;
  const unsigned first = (unsigned)(base - row0 * a.chunks) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const unsigned i = first + (unsigned)(k * kThreads);
    const unsigned r = fast_div(i, a.by_chunks);
    const int64_t row = row0 + r;
    body(k, row, (int)(i - r * (unsigned)a.chunks), row < a.tokens);
  }
}

__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheArgs a) {
  const int which = blockIdx.y;
  const uint16_t* x = which ? a.v : a.k;
  const int64_t stride = which ? a.v_stride : a.k_stride;
  uint8_t* codes = which ? a.v_codes : a.k_codes;
  uint8_t* scales = which ? a.v_scales : a.k_scales;
  u32x4 in[kUnits];
  int slot[kUnits];
  for_chunks(a, [&](int k, int64_t row, int chunk, bool live) {
    in[k] = u32x4{0, 0, 0, 0};
    slot[k] = -1;
    if (live) {
      in[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + row * stride + 8 * chunk));
      slot[k] = a.slots[row];
    }
  });
  for_chunks(a, [&](int k, int64_t, int chunk, bool) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[2 * j] = bf16_lo(in[k][j]);
      y[2 * j + 1] = bf16_hi(in[k][j]);
    }
    const unsigned byte = e8m0_byte(block_amax<LAYOUT_QUAD>(y));  // the four lanes of a block share a row
    const unsigned word = pack_fp4(y, byte);
    if ((unsigned)slot[k] < (unsigned)a.n_slots) {  // a token without a slot writes nothing
      *reinterpret_cast<unsigned*>(codes + (int64_t)slot[k] * (4 * a.chunks) + 4 * chunk) = word;
      if ((chunk & 3) == 0) scales[(int64_t)slot[k] * (a.chunks >> 2) + (chunk >> 2)] = (uint8_t)byte;
    }
  });
}

__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheArgs a) {
  const int which = blockIdx.y;
  uint16_t* x = which ? a.v_out : a.k_out;
  const int64_t stride = which ? a.v_stride : a.k_stride;
  const uint8_t* codes = which ? a.v_codes : a.k_codes;
  const uint8_t* scales = which ? a.v_scales : a.k_scales;
  unsigned word[kUnits], byte[kUnits];
  for_chunks(a, [&](int k, int64_t row, int chunk, bool live) {
    word[k] = 0;
    byte[k] = 0;
    const int slot = live ? a.slots[row] : -1;
    if ((unsigned)slot < (unsigned)a.n_slots) {  // a token without a slot reads as zeros
      word[k] = *reinterpret_cast<const unsigned*>(codes + (int64_t)slot * (4 * a.chunks) + 4 * chunk);
      byte[k] = scales[(int64_t)slot * (a.chunks >> 2) + (chunk >> 2)];
    }
  });
  for_chunks(a, [&](int k, int64_t row, int chunk, bool live) {
    if (live) {
      const u32x4 v = __builtin_bit_cast(u32x4, mx_values8(word[k], byte[k]));
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(x + row * stride + 8 * chunk));
    }
  });
}

}  // namespace

hipError_t launch_cache(bool write, bool both, const CacheArgs& args, hipStream_t stream) {
  CacheArgs a = args;
  a.by_chunks = make_divisor((unsigned)a.chunks);
  const int64_t n = a.tokens * a.chunks, per = kThreads * kUnits;
  const dim3 grid((unsigned)((n + per - 1) / per), both ? 2 : 1);
  void* kargs[] = {&a};
  return hipLaunchKernel(write ? (const void*)&cache_write_kernel : (const void*)&cache_read_kernel, grid,
                         dim3(kThreads), kargs, 0, stream);
}

}  // namespace kq
