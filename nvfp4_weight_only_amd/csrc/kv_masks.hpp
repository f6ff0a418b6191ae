// Which tokens a row of attention sees by its place, apart from the kernels so that a
// program on the host runs the same code at the ends of the range
// (tests/sanitize/kv_masks_driver.cpp).  A row at position pos sees token t if t <= pos and,
// with a window, t > pos - window.  pos is at least -2^23 (rows before token 0), a token at
// least 0 and at most 64 behind a sequence's last row, window at most 2^31 - 1: differences
// of positions and tokens fit 32 bits, those of a hidden token and a window may not.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define NVFP4_MASK __host__ __device__ inline __attribute__((always_inline))
#else
#define NVFP4_MASK inline
#endif

namespace nvfp4 {

// Bits 0 .. n - 1.
NVFP4_MASK uint32_t low_bits(int32_t n) { return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u); }

// Of the 32 tokens from t0 on, those that a row at position pos sees by its place.
NVFP4_MASK uint32_t seen_bits(int32_t pos, int32_t window, int32_t t0) {
  const int32_t to = pos - t0 + 1;  // tokens up to the row's
  return low_bits(to) & ~(window > 0 && to > window ? low_bits(to - window) : 0u);
}

NVFP4_MASK bool sees(int32_t pos, int32_t window, int32_t t) { return t <= pos && (window == 0 || pos - t < window); }

// The first token that a row at position pos sees.
NVFP4_MASK int32_t first_seen(int32_t pos, int32_t window) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// Where the tokens start that some row of a tile sees, the first of which is at pos (tile tokens at a time, a power of
// two): not behind their end, so that places computed from it stay in range.
NVFP4_MASK int32_t first_tile(int64_t pos, int32_t window, int32_t tile, int32_t end) {
  if (window == 0 || pos < window) return 0;
  const int64_t first = pos - window + 1;
  return (int32_t)(first < end ? first : end) & ~(tile - 1);
}

}  // namespace nvfp4
