// Host-side sweep of the E4M3 entry points with invalid, boundary and
// overflowing arguments, for a build whose host code is compiled with
// AddressSanitizer and UndefinedBehaviorSanitizer.  Pointers are fake addresses
// that must never be dereferenced; with a GPU present the sweep does not run.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "nvfp4.h"

namespace {

const int64_t kSizes[] = {-1, 0, 1, 8, 16, 127, 128, 144, 4096, 17408, (int64_t)1 << 23, (int64_t)1 << 31,
                          (int64_t)1 << 40, INT64_MAX / 16, INT64_MAX - 1, INT64_MAX};
const int kNumSizes = sizeof(kSizes) / sizeof(kSizes[0]);

template <typename T>
T* fake(uint64_t base, uint64_t off = 0) {
  return reinterpret_cast<T*>(base + off);
}

const uint64_t A = 0x100000000000ull, B = 0x200000000000ull, C = 0x300000000000ull, D = 0x400000000000ull,
               E = 0x500000000000ull, F = 0x600000000000ull, G = 0x700000000000ull;

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
  const float eps[] = {1e-6f, 0.0f, -1.0f, NAN, INFINITY};
  for (int offs = 0; offs < 3; ++offs) {
    const uint64_t o = offs == 0 ? 0 : (offs == 1 ? 8 : 16);
    for (int i = 0; i < kNumSizes; ++i)
      for (int j = 0; j < kNumSizes; ++j) {
        const int64_t a = kSizes[i], b = kSizes[j];
        for (float e : eps) {
          note(nvfp4_rmsnorm_fp8(fake<uint16_t>(A), fake<uint16_t>(B), fake<uint16_t>(C, o), e, a, b,
                                 fake<uint16_t>(B, o), fake<uint8_t>(D), fake<float>(E), nullptr));
          note(nvfp4_rmsnorm_fp8(fake<uint16_t>(A, o), nullptr, fake<uint16_t>(C), e, a, b, nullptr, fake<uint8_t>(D),
                                 fake<float>(E), nullptr));
        }
        note(nvfp4_silu_mul_fp8(fake<uint16_t>(A, o), a, b, fake<uint8_t>(D), fake<float>(E), nullptr));
        for (int l = 0; l < kNumSizes; ++l) {
          const int64_t c = kSizes[l];
          for (int64_t rows : {(int64_t)1, (int64_t)128, (int64_t)0})
            note(nvfp4_fp8_quantize(fake<uint16_t>(A), a, b, c, rows, fake<uint8_t>(D, o), fake<float>(E), nullptr));
          (void)nvfp4_fp8_linear_workspace_bytes(a, b, c);
          (void)nvfp4_fp8_linear_grouped_workspace_bytes(a, b, c);
          for (int64_t wsb : {(int64_t)-1, (int64_t)0, (int64_t)1 << 30})
            note(nvfp4_fp8_linear(fake<uint8_t>(A), fake<float>(B, o), a, b, c, fake<uint8_t>(C), fake<float>(D),
                                  fake<uint16_t>(E), fake<void>(F, o), wsb, nullptr));
          // (t_count, topk, experts) = (a, b, c), and (experts, n, k) = (a, b, c).
          note(nvfp4_fp8_linear_grouped(fake<uint8_t>(A), fake<float>(B), a, b, fake<int32_t>(G, o), c, 256, 512,
                                        fake<uint8_t>(C), fake<float>(D), fake<uint16_t>(E), fake<void>(F),
                                        INT64_MAX, nullptr));
          note(nvfp4_fp8_linear_grouped(fake<uint8_t>(A), fake<float>(B), 64, 4, fake<int32_t>(G), a, b, c,
                                        fake<uint8_t>(C, o), fake<float>(D), fake<uint16_t>(E), fake<void>(F),
                                        (int64_t)1 << 30, nullptr));
        }
      }
  }
  printf("%ld calls\n", g_calls);
  return 0;
}
