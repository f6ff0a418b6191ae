// Host-side sweep of the entry points around a paged FP4 cache with invalid, boundary
// and overflowing arguments, for a build whose host code is compiled with
// AddressSanitizer and UndefinedBehaviorSanitizer.  Pointers are fake addresses that must
// never be dereferenced; with a GPU present the sweep does not run.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "nvfp4.h"

namespace {

const int64_t kSizes[] = {-1, 0, 1, 8, 16, 64, 96, 128, 4096, (int64_t)1 << 19, (int64_t)1 << 31,
                          (int64_t)1 << 40, INT64_MAX / 16, INT64_MAX - 1, INT64_MAX};

template <typename T>
T* fake(uint64_t n, uint64_t off = 0) {
  return reinterpret_cast<T*>(n * 0x100000000000ull + off);
}

long g_calls = 0;

void note(nvfp4_status st) {
  ++g_calls;
  if (st < NVFP4_OK || st > NVFP4_ERR_ALIAS) {
    fprintf(stderr, "status out of range: %d\n", (int)st);
    __builtin_trap();
  }
}

}  // namespace

int main() {
  int devices = 0;
  if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {
    printf("GPU present: sweep skipped\n");
    return 0;
  }
  for (uint64_t o : {(uint64_t)0, (uint64_t)8})
    for (int64_t a : kSizes)
      for (int64_t b : kSizes) {
        const nvfp4_rope_spec rope = {fake<double>(9), a, 1.0f, 0}, rope64 = {fake<double>(9, o), 64, 1.0f, 1};
        for (double base : {1e4, 0.0, (double)NAN})
          note(nvfp4_rope_frequencies(3, a, base, 2.0, (double)b, 1.0, 32.0, fake<double>(1, o), nullptr));
        note(nvfp4_rope(1, fake<uint16_t>(1), 8, 4, b, a, b, fake<int32_t>(2), &rope, 0, fake<uint16_t>(3, o), a, b,
                        nullptr));
        for (int64_t c : kSizes) {
          note(nvfp4_rope(0, fake<uint16_t>(1, o), a, b, 64, c, 64, fake<int32_t>(2), &rope64, 1, fake<uint16_t>(3), 64 * 64,
                          c, nullptr));
          (void)nvfp4_kv_attention_workspace_bytes(a, 128, b, c, 8);
          (void)nvfp4_kv_attention_workspace_bytes(8, a, 40, b, c);
          for (int format = -1; format < 3; ++format) {
            const nvfp4_kv_cache sizes = {format, a, b, c, 128, fake<uint8_t>(4), fake<uint8_t>(5), fake<float>(6),
                                          fake<uint8_t>(7, o), fake<uint8_t>(8), fake<float>(10)};
            const nvfp4_kv_cache plain = {format, 64, 16, 8, 128, fake<uint8_t>(4), fake<uint8_t>(5), fake<float>(6),
                                          fake<uint8_t>(7), fake<uint8_t>(8, o), fake<float>(10)};
            for (const nvfp4_kv_cache* cache : {&sizes, &plain}) {
              note(nvfp4_kv_append(cache, 1, fake<uint16_t>(1), fake<uint16_t>(2), a, b, 128, 1024, c, fake<int32_t>(11), b,
                                   fake<int32_t>(12), fake<int32_t>(13), c, &rope64, fake<int32_t>(14, o), nullptr));
              note(nvfp4_kv_append(cache, 0, fake<uint16_t>(1), fake<uint16_t>(2), 4, 2048, 128, 2048, 128, fake<int32_t>(11),
                                   a, fake<int32_t>(12), fake<int32_t>(13), b, &rope, nullptr, nullptr));
              for (int64_t wsb : {(int64_t)-1, (int64_t)0, INT64_MAX})
                note(nvfp4_kv_attention(cache, 1, fake<uint16_t>(1), a, 40, b, 128, fake<int32_t>(11), c, fake<int32_t>(12),
                                        fake<int32_t>(13), b, 0.1f, c, fake<uint16_t>(2), fake<void>(3), wsb, nullptr));
              note(nvfp4_kv_attention(cache, 0, fake<uint16_t>(1), 8, a, 128, b, fake<int32_t>(11), 4, fake<int32_t>(12),
                                      nullptr, 8, 0.1f, 0, fake<uint16_t>(2), fake<void>(3, o), INT64_MAX, nullptr));
            }
          }
        }
      }
  printf("%ld calls\n", g_calls);
  return 0;
}
