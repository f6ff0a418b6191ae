// Which tokens a row of attention sees (csrc/kv_masks.hpp), against 64-bit arithmetic, at the ends of the range that
// the kernels use it in.  Built with AddressSanitizer and UndefinedBehaviorSanitizer.
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "kv_masks.hpp"

static long g_checks = 0;

static void check(bool ok, const char* what, long pos, long window, long t) {
  ++g_checks;
  if (ok) return;
  fprintf(stderr, "%s: pos %ld, window %ld, token %ld\n", what, pos, window, t);
  exit(1);
}

int main() {
  const int64_t kMost = INT32_MAX, kTokens = kMost - 4096;
  const int64_t places[] = {-(1 << 23), -1000, -33, -1, 0, 1, 31, 32, 63, 64, 1000, 70001, 1 << 30, kTokens - 64, kTokens - 1,
                            kMost - 1};
  const int64_t windows[] = {0, 1, 2, 31, 32, 33, 64, 4096, 1 << 30, kTokens, kMost - 31, kMost - 1, kMost};
  for (int64_t pos : places)
    for (int64_t window : windows) {
      const auto want = [&](int64_t t) { return t <= pos && (window == 0 || t > pos - window); };
      for (int64_t near : {pos, pos - window, (int64_t)0, pos + 64, pos - (1 << 23)})
        for (int64_t t0 = (near & ~(int64_t)31) - 64; t0 <= near + 64; t0 += 32) {
          if (t0 < 0 || t0 > kTokens || t0 > (pos < 0 ? (1 << 23) : pos) + 64) continue;  // at most 64 behind a last row
          const uint32_t bits = nvfp4::seen_bits((int32_t)pos, (int32_t)window, (int32_t)t0);
          for (int i = 0; i < 32; ++i) {
            check(((bits >> i) & 1u) == (want(t0 + i) ? 1u : 0u), "seen_bits", pos, window, t0 + i);
            check(nvfp4::sees((int32_t)pos, (int32_t)window, (int32_t)(t0 + i)) == want(t0 + i), "sees", pos, window, t0 + i);
          }
        }
      const int64_t first = window > 0 && pos - window + 1 > 0 ? pos - window + 1 : 0;
      check(nvfp4::first_seen((int32_t)pos, (int32_t)window) == first, "first_seen", pos, window, first);
      for (int64_t end : {(int64_t)0, (int64_t)1, (int64_t)100, (int64_t)4096, kTokens, pos + 1})
        for (int tile : {32, 64}) {
          if (end < 0 || end > kTokens) continue;
          const int64_t lo = nvfp4::first_tile(pos, (int32_t)window, tile, (int32_t)end);
          check(lo >= 0 && lo % tile == 0 && lo <= end && lo <= first, "first_tile's range", pos, window, lo);
          check(first >= end || first - lo < tile, "first_tile", pos, window, lo);
        }
    }
  printf("%ld checks\n", g_checks);
  return 0;
}
