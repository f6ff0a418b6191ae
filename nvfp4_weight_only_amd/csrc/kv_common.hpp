// What the kernels around a paged FP4 cache of keys and values share: the cache
// and the batch as the kernels see them, the place of a row's token, the codes'
// decoding and the rotation's angles.
//
// Cache: pages of block_size tokens; codes [num_blocks, block_size, heads,
// head_dim / 2], scales [num_blocks, block_size, heads, head_dim / G] (G = 16
// with E4M3 scales and one FP32 tensor scale, or 32 with UE8M0 scales).
// Batch: rows row_start[s] .. row_start[s + 1] - 1 are the last tokens of
// sequence s, whose tokens 0 .. seq_lens[s] - 1 are in the pages block_table[s, *]
// (without row_start, row s is the last token of sequence s).  All of it is device
// data, so every index made from it is checked where it is used.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace nvfp4 {

struct KvCache {
  bool mx;
  int64_t num_blocks, block_size, heads, head_dim;
  uint8_t* codes[2];  // keys, values
  uint8_t* scales[2];
  const float* tscale[2];
};

struct KvBatch {
  const int32_t* block_table;  // [seqs, max_blocks]
  int64_t max_blocks;
  const int32_t* seq_lens;   // [seqs]
  const int32_t* row_start;  // [seqs + 1], or null
  int64_t seqs;
  int64_t rows;
};

// First head_dim elements of a head that are rotated, and how.
struct RopeArgs {
  const double* freqs;  // [rot / 2], radians a token
  int64_t rot;          // a multiple of 16; 0: no rotation
  float amplitude;
  int interleaved;
};

// n / d for 0 <= n < 2^31 by the high half of one product: m = ceil(2^(31 + lg) / d)
// with lg = ceil(log2 d) fits 32 bits and overshoots 2^(31 + lg) / d by less than 1, so
// n m / 2^(31 + lg) overshoots n / d by less than n / 2^(31 + lg) <= 1 / d, which does not
// reach the next integer.
struct FastDiv {
  uint32_t m, lg;
  int32_t d;
};
inline FastDiv make_fastdiv(int64_t d) {
  uint32_t lg = 0;
  while (((int64_t)1 << lg) < d) ++lg;
  const uint64_t one = (uint64_t)1 << (31 + lg);
  return {(uint32_t)((one + (uint64_t)d - 1) / (uint64_t)d), lg, (int32_t)d};
}
__device__ __forceinline__ int32_t fastdiv(int32_t n, const FastDiv& f) {
  return (int32_t)(__umulhi((uint32_t)n << 1, f.m) >> f.lg);
}

// a / b for 0 <= a < 2^52, 0 < b < 2^52: the FP64 quotient, put right by its remainder
// (a 64-bit integer division takes some 150 instructions).
__device__ __forceinline__ int64_t div_i64(int64_t a, int64_t b) {
  int64_t q = (int64_t)((double)a / (double)b);
  const int64_t r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}

// Rows of sequence s inside [0, rows), and where its last token ends:
// row r is token end - (last - r).
struct SeqRows {
  int64_t first, count;  // rows to compute
  int64_t shift;         // row r is token r + shift
  int64_t len;           // tokens of the cache: min(seq_lens, max_blocks * block_size), at least 0
};
__device__ __forceinline__ SeqRows seq_rows(const KvBatch& b, int64_t cap, int64_t s) {
  const int64_t a = b.row_start ? (int64_t)b.row_start[s] : s, e = b.row_start ? (int64_t)b.row_start[s + 1] : s + 1;
  const int64_t n = b.seq_lens[s];
  SeqRows r;
  r.first = a < 0 ? 0 : a;
  const int64_t last = e > b.rows ? b.rows : e;
  r.count = last > r.first ? last - r.first : 0;
  r.shift = n - e;
  r.len = n < 0 ? 0 : (n > cap ? cap : n);
  return r;
}

// The last sequence that starts at or before row r (any sequence if none does), by a
// wavefront: 64 starts at a time; starts do not fall, so those at or before r come first.
__device__ __forceinline__ int64_t find_sequence(const KvBatch& b, int64_t r, int lane) {
  int64_t lo = 0, hi = b.seqs;  // sequences lo .. hi - 1 may hold r
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64, at = lo + lane * step;
    const bool le = at < hi && (int64_t)b.row_start[at] <= r;
    const int n = __popcll(__ballot(le));
    if (n == 0) break;
    lo += (int64_t)(n - 1) * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// Angles.  Radians in FP64: at position 10^6 an angle in FP32 would be off by
// 0.06.  Reduced by multiples of pi / 2 in two parts (the first difference is exact,
// the second rounded once, so what is left is off by less than 2^-53 for |angle| up
// to 2^31), then the Taylor series, whose first term left out is below 2^-63 on
// [-pi/4, pi/4].  FP64 runs at FP32's rate here.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void sincos_f64(double x, double* sn, double* cs) {
  const double n = __builtin_rint(x * 0.63661977236758134308);  // 2 / pi
  double r = fma(-n, 1.5707963267948965580, x);                 // pi / 2 = its FP64 value
  r = fma(-n, 6.1232339957367658861e-17, r);                    //   + the rest's FP64 value
  const double z = r * r;
  double s = 1.0 / 355687428096000.0;  // 1 / 17!
  s = fma(-z, s, 1.0 / 1307674368000.0);
  s = fma(-z, s, 1.0 / 6227020800.0);
  s = fma(-z, s, 1.0 / 39916800.0);
  s = fma(-z, s, 1.0 / 362880.0);
  s = fma(-z, s, 1.0 / 5040.0);
  s = fma(-z, s, 1.0 / 120.0);
  s = fma(-z, s, 1.0 / 6.0);
  s = fma(-z * s, r, r);
  double c = 1.0 / 6402373705728000.0;  // 1 / 18!
  c = fma(-z, c, 1.0 / 20922789888000.0);
  c = fma(-z, c, 1.0 / 87178291200.0);
  c = fma(-z, c, 1.0 / 479001600.0);
  c = fma(-z, c, 1.0 / 3628800.0);
  c = fma(-z, c, 1.0 / 40320.0);
  c = fma(-z, c, 1.0 / 720.0);
  c = fma(-z, c, 1.0 / 24.0);
  c = fma(-z, c, 0.5);
  c = fma(-z, c, 1.0);
  const int q = (int)(int64_t)n;  // the quarter turn, by its last two bits
  const double a = q & 1 ? c : s, b = q & 1 ? s : c;
  *sn = q & 2 ? -a : a;
  *cs = (q + 1) & 2 ? -b : b;
}

// ---------------------------------------------------------------------------
// 16-bit inputs and outputs.
// ---------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ float half_to_f32(uint32_t b) {
  if constexpr (BF16) return bf16_to_f32(b);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

// Two floats rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t f32x2_to_half(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  if constexpr (BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

}  // namespace nvfp4
