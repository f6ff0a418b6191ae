// E4M3 tensors with one FP32 scale per block of 1 x 128 (activations) or
// 128 x 128 (weights): the quantizer, and the two producers of a layer's 8-bit
// operands, the RMS norm (with the residual's addition) and silu(gate) * up.
//
// For a block with values v (the last block of an axis may be short):
//   amax = max |v|,  scale = fl32(amax / 448),
//   code = the E4M3 value nearest to 448 v / amax, ties to the even code.
// amax = 0 gives scale 0 and codes 0; a block with a value that is not finite
// gives scale NaN and codes 0x7F (NaN), so the fault reaches the output.
//
// The quotient is rounded once: q = a * rcp(b) and one residual step
// q + (a - q b) rcp(b) give the FP32 nearest to a / b, so a quotient that is a
// tie of the E4M3 grid comes out exactly.  For BF16 inputs a = 448 v and b =
// amax have at most 11 and 8 significant bits, so any other quotient is at
// least 2^-14 (relative) away from a tie and stays on its side.  A power of
// two keeps a and b inside FP32's normal range.
//
// Lanes: one 16-byte load (8 BF16 values) per piece; 16 consecutive lanes hold
// a block of 128, so its maximum is four DPP row rotations.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u, kNanBits = 0x7FC00000u;

template <int R>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 | R, 0xF, 0xF, true);
}

// Maximum over each aligned group of 16 lanes, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  uint32_t o = row_ror<8>(v);
  v = o > v ? o : v;
  o = row_ror<4>(v);
  v = o > v ? o : v;
  o = row_ror<2>(v);
  v = o > v ? o : v;
  o = row_ror<1>(v);
  return o > v ? o : v;
}

template <int R>
__device__ __forceinline__ uint64_t row_max64_step(uint64_t v) {
  const uint64_t o = (uint64_t)row_ror<R>((uint32_t)(v >> 32)) << 32 | row_ror<R>((uint32_t)v);
  return o > v ? o : v;
}
__device__ __forceinline__ uint64_t row_max64(uint64_t v) {
  return row_max64_step<1>(row_max64_step<2>(row_max64_step<4>(row_max64_step<8>(v))));
}

__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8]) {
  v[0] = bf16_lo(p.x), v[1] = bf16_hi(p.x), v[2] = bf16_lo(p.y), v[3] = bf16_hi(p.y);
  v[4] = bf16_lo(p.z), v[5] = bf16_hi(p.z), v[6] = bf16_lo(p.w), v[7] = bf16_hi(p.w);
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// Bits of max |v|: as integers the bits of non-negative floats order like their
// values, with infinity and the NaNs above every finite one.
__device__ __forceinline__ uint32_t max8(const float (&v)[8]) {
  uint32_t m = abs_bits(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = abs_bits(v[i]) > m ? abs_bits(v[i]) : m;
  return m;
}

// The block's constants: code = E4M3(v * c / b).
struct Encoder {
  float c, b, r;
  uint32_t amax;
};

__device__ __forceinline__ Encoder encoder(uint32_t amax) {
  const float p = amax >= 0x71800000u ? 0x1p-64f : (amax < 0x21800000u ? 0x1p64f : 1.0f);  // 2^100, 2^-60
  Encoder e;
  e.amax = amax;
  e.c = 448.0f * p;
  e.b = __uint_as_float(amax) * p;
  e.r = __builtin_amdgcn_rcpf(e.b);
  return e;
}

__device__ __forceinline__ float quotient(const Encoder& e, float v) {
  const float a = v * e.c, q = a * e.r;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, e.b, a), e.r, q), v);  // -0 stays -0
}

// 8 values -> 8 codes.
__device__ __forceinline__ uint2 encode8(const Encoder& e, const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(e, v[4 * h]), quotient(e, v[4 * h + 1]), 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(e, v[4 * h + 2]), quotient(e, v[4 * h + 3]), p, true);
    w[h] = e.amax == 0 ? 0u : (e.amax >= kInfBits ? 0x7F7F7F7Fu : (uint32_t)p);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float block_scale(uint32_t amax) {
  return amax >= kInfBits ? __uint_as_float(kNanBits) : __uint_as_float(amax) / 448.0f;
}

// ---------------------------------------------------------------------------
// Blocks of 1 x 128 along the rows of a [rows, k] tensor: thread t of the grid
// takes block t / 16 (and U - 1 more, a workgroup's 16 apart), piece t % 16 of
// it, and goes on a grid further while there are blocks.
// SILU: the tensor is silu(g) * u of a [rows, 2 k] tensor of g and u halves.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;

// g / (1 + exp(-g)) * u through z = exp(-|g| / 2) <= 1, which cannot overflow: d = 1 +
// z^2, and g u / d or (g z) (u z) / d by the sign of g.  Neither factor leaves FP32's
// normal range before the product does, down to g = -174, below which z is taken as 0.
// log2(e) = hi + lo with 16 bits in hi, so that |g| hi is exact for a BF16 g and exp2's
// argument has no rounding; z (1 - |g| lo ln 2 / 2) is exp(-|g| / 2) to second order.
// The quotient n / d is corrected once (d is in [1, 2]).  The result is within 6
// 2^-24 of it (all BF16 gates, four ups).  A gate that is not finite gives NaN.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float ag = __builtin_fabsf(g);
  const float z0 = __builtin_amdgcn_exp2f(-(ag * 0x1.7154000000000p-1f));
  const float z = __builtin_fmaf(z0, ag * -(0x1.480fb50c621ccp-19f), z0), d = __builtin_fmaf(z, z, 1.0f);
  const float f = g >= 0.0f ? 1.0f : z, r = __builtin_amdgcn_rcpf(d), n = g * f, q = n * r;
  return __builtin_fmaf(__builtin_fmaf(-q, d, n), r, q) * (u * f);
}

// NEAR: a workgroup's U * 16 blocks lie in two rows (kb >= 16 U, k < 2^28), so the
// row and the addresses come from one scalar division and 32-bit offsets.  The
// general form divides in every lane (on [2048, 2 x 17408], silu: 42.5 us
// against 41.0 with two blocks a thread, 39.8 with four).
template <bool SILU, int U, bool NEAR>
__global__ void __launch_bounds__(kThreads) fp8_rows_kernel(const uint16_t* __restrict__ x, int64_t blocks, uint32_t kb,
                                                            int64_t k, uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
  constexpr int step = kThreads / 16;
  const uint32_t piece = threadIdx.x & 15;
  const int64_t xrow = SILU ? 2 * k : k;
  // The same trip count in every lane of a row of 16 (and no lane leaves early).
  for (int64_t first = (int64_t)blockIdx.x * (U * step); first < blocks; first += (int64_t)gridDim.x * (U * step)) {
    const int64_t r0 = NEAR ? first / kb : 0;
    const uint32_t c0 = NEAR ? (uint32_t)(first - r0 * kb) : 0;
    const uint16_t* const xb = x + r0 * xrow;
    uint8_t* const cb = codes + r0 * k;
    uint4 d[U], d2[U];
    typename std::conditional<NEAR, uint32_t, int64_t>::type out[U];
    bool in[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t blk = first + i * step + (threadIdx.x >> 4);
      if constexpr (NEAR) {
        const uint32_t c = c0 + i * step + (threadIdx.x >> 4), next = c >= kb;
        const uint32_t col = (c - (next ? kb : 0u)) * 128 + piece * 8;
        in[i] = blk < blocks && col < (uint32_t)k;
        out[i] = (next ? (uint32_t)k : 0u) + col;
        d[i] = d2[i] = make_uint4(0, 0, 0, 0);
        if (in[i]) {
          const uint16_t* src = xb + (next ? (uint32_t)xrow : 0u) + col;
          d[i] = ld_stream16(src);
          if constexpr (SILU) d2[i] = ld_stream16(src + k);
        }
      } else {
        const int64_t row = blk / kb, col = (blk - row * kb) * 128 + piece * 8;
        in[i] = blk < blocks && col < k;
        out[i] = row * k + col;
        d[i] = d2[i] = make_uint4(0, 0, 0, 0);
        if (in[i]) {
          const uint16_t* src = xb + row * xrow + col;
          d[i] = ld_stream16(src);
          if constexpr (SILU) d2[i] = ld_stream16(src + k);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float v[8];
      unpack8(d[i], v);
      if constexpr (SILU) {
        float u[8];
        unpack8(d2[i], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = silu_mul(v[j], u[j]);
      }
      const uint32_t amax = row_max(max8(v));
      const uint2 c = encode8(encoder(amax), v);
      if (in[i]) *reinterpret_cast<uint2*>(cb + out[i]) = c;
      const int64_t blk = first + i * step + (threadIdx.x >> 4);
      if (piece == 0 && blk < blocks) scales[blk] = block_scale(amax);
    }
  }
}

// ---------------------------------------------------------------------------
// Blocks of 128 x 128: one workgroup each, 8 rows' pieces per thread (thread t:
// piece t % 16 of rows t / 16, t / 16 + 16, ...).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) fp8_tiles_kernel(const uint16_t* __restrict__ w, int64_t n, int64_t k,
                                                             int64_t nb, int64_t kb, int64_t blocks,
                                                             uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ uint32_t wmax[kThreads / 64];
  const int64_t id = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
  if (id >= blocks) return;
  const int64_t bk = id % kb, rest = id / kb, bn = rest % nb, base = rest / nb * n * k;
  const int64_t col = bk * 128 + (threadIdx.x & 15) * 8, row0 = bn * 128 + (threadIdx.x >> 4);
  uint4 d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 16 * i;
    d[i] = row < n && col < k ? ld_stream16(w + base + row * k + col) : make_uint4(0, 0, 0, 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8(d[i], v);
    const uint32_t o = max8(v);
    m = o > m ? o : m;
  }
  m = wave_max_u32(m);
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
  __syncthreads();
  m = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) m = wmax[i] > m ? wmax[i] : m;
  const Encoder e = encoder(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 16 * i;
    float v[8];
    unpack8(d[i], v);
    const uint2 c = encode8(e, v);
    if (row < n && col < k) *reinterpret_cast<uint2*>(codes + base + row * k + col) = c;
  }
  if (threadIdx.x == 0) scales[id] = block_scale(m);
}

// ---------------------------------------------------------------------------
// RMS norm: h = BF16(x + r) (h = x without a residual), stored;
//   v_i = h_i g_i / sqrt(mean_j h_j^2 + eps), quantized in blocks of 1 x 128.
// The row's factor cancels in the codes' quotients, so they are taken from the
// products h_i g_i (16 significant bits, exact in FP32; in FP64 where they leave its
// range) and only the scale carries the factor: the codes do not depend on how the
// statistics rounded.
// h is rounded before the norm reads it, so that the norm and the next layer's
// residual see the same values.
// One workgroup per row, P pieces of 8 elements per thread in registers; the
// sum of squares in FP32.  A row whose sum is not finite gives NaN scales and
// NaN codes.
// ---------------------------------------------------------------------------
// BF16(x + r) of 8 elements.
__device__ __forceinline__ uint4 add8(const uint4& x, const uint4& r) {
  float a[8], b[8];
  unpack8(x, a);
  unpack8(r, b);
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bf16x2_t s = {(__bf16)(a[2 * j] + b[2 * j]), (__bf16)(a[2 * j + 1] + b[2 * j + 1])};
    o[j] = __builtin_bit_cast(uint32_t, s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float sum_squares(const uint4& h) {
  float v[8], s = 0.0f;
  unpack8(h, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) s = __builtin_fmaf(v[j], v[j], s);
  return s;
}

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ float wg_sum(float s) {
  __shared__ float part[16];
  s = wave_sum(s);
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = part[0];
  for (int i = 1; i < waves; ++i) s += part[i];
  return s;
}

// Eight elements of a row to codes and scale.  Returns whether norm_store_far has to
// do it again: a product h g or the block's largest v is no FP32 number, or products
// below FP32's normal range may count.  With a maximum of at least 2^-100 they do
// not: they have code 0 whatever their lost bits.
__device__ __forceinline__ bool norm_store(const uint4& h, const uint16_t* __restrict__ weight, int64_t col, bool in,
                                           float rstd, bool finite, int64_t row, int64_t k, int64_t kb,
                                           uint8_t* __restrict__ codes, float* __restrict__ scales) {
  float v[8], g[8];
  unpack8(h, v);
  const uint4 gw = in ? *reinterpret_cast<const uint4*>(weight + col) : make_uint4(0, 0, 0, 0);
  unpack8(gw, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= g[j];
  uint32_t amax = row_max(max8(v));
  amax = finite ? amax : kNanBits;
  const float top = __uint_as_float(amax) * rstd;
  const uint2 c = encode8(encoder(amax), v);
  if (in) *reinterpret_cast<uint2*>(codes + row * k + col) = c;
  if ((threadIdx.x & 15) == 0 && in) scales[row * kb + col / 128] = block_scale(__float_as_uint(top));
  return finite && (amax < 0x0D800000u || __float_as_uint(top) >= kInfBits) &&
         ((h.x | h.y | h.z | h.w) & 0x7FFF7FFFu) != 0;
}

// The same in FP64: products exact, quotients rounded once, the range of v FP32's.
__device__ __forceinline__ void norm_store_far(const uint4& h, const uint16_t* __restrict__ weight, int64_t col, bool in,
                                               float rstd, int64_t row, int64_t k, int64_t kb,
                                               uint8_t* __restrict__ codes, float* __restrict__ scales) {
  float a[8], g[8];
  unpack8(h, a);
  unpack8(in ? *reinterpret_cast<const uint4*>(weight + col) : make_uint4(0, 0, 0, 0), g);
  uint64_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint64_t o = __builtin_bit_cast(uint64_t, __builtin_fabs((double)a[j] * (double)g[j]));
    m = o > m ? o : m;
  }
  m = row_max64(m);
  const double amax = __builtin_bit_cast(double, m);
  const float top = (float)(amax * (double)rstd);
  const bool finite = __float_as_uint(top) < kInfBits;
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = m == 0 ? 0.0f : (float)((double)a[j] * (double)g[j] * 448.0 / amax);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], p, true);
    w[i] = finite ? (uint32_t)p : 0x7F7F7F7Fu;
  }
  if (in) *reinterpret_cast<uint2*>(codes + row * k + col) = make_uint2(w[0], w[1]);
  if ((threadIdx.x & 15) == 0 && in) scales[row * kb + col / 128] = block_scale(__float_as_uint(top));
}

// The wavefront's pieces (n of them, step elements apart) again in FP64.  They are
// read again, each by the thread that stored it, and not kept in registers: in line,
// 2048 x 5120 took 18.1 us instead of 17.2.
template <bool RES>
__device__ __forceinline__ void norm_row_far(const uint16_t* x, const uint16_t* __restrict__ weight, float rstd, int64_t row,
                                             int64_t k, int64_t kb, int64_t step, int64_t n, const uint16_t* h,
                                             uint8_t* __restrict__ codes, float* __restrict__ scales) {
#pragma unroll 1
  for (int64_t i = 0; i < n; ++i) {
    const int64_t col = i * step + 8 * threadIdx.x;
    const bool in = col < k;
    const uint4 v = in ? *reinterpret_cast<const uint4*>((RES ? h : x) + row * k + col) : make_uint4(0, 0, 0, 0);
    norm_store_far(v, weight, col, in, rstd, row, k, kb, codes, scales);
  }
}

template <int P, bool RES>
__global__ void __launch_bounds__(1024) rmsnorm_fp8_kernel(const uint16_t* __restrict__ x, const uint16_t* residual,
                                                           const uint16_t* __restrict__ weight, float eps, int64_t rows,
                                                           int64_t k, uint16_t* h_out, uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales) {
  const int64_t row = blockIdx.x + (int64_t)blockIdx.y * gridDim.x, kb = (k + 127) / 128;
  if (row >= rows) return;
  uint4 h[P], r[RES ? P : 1];
  float ss = 0.0f;
  // Every load before the first store: h_out may be the residual itself.
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int64_t col = 8 * ((int64_t)i * blockDim.x + threadIdx.x);
    h[i] = col < k ? ld_stream16(x + row * k + col) : make_uint4(0, 0, 0, 0);
    if constexpr (RES)
      r[i] = col < k ? ld_stream16(residual + row * k + col) : make_uint4(0, 0, 0, 0);
  }
  if constexpr (RES) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int64_t col = 8 * ((int64_t)i * blockDim.x + threadIdx.x);
      h[i] = add8(h[i], r[i]);
      if (col < k) *reinterpret_cast<uint4*>(h_out + row * k + col) = h[i];
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) ss += sum_squares(h[i]);
  ss = wg_sum(ss);
  const float rstd = 1.0f / __builtin_sqrtf(ss / (float)k + eps);
  const bool finite = (__float_as_uint(ss) & kInfBits) != kInfBits;
  bool far = false;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int64_t col = 8 * ((int64_t)i * blockDim.x + threadIdx.x);
    far |= norm_store(h[i], weight, col, col < k, rstd, finite, row, k, kb, codes, scales);
  }
  if (__builtin_amdgcn_ballot_w64(far) != 0)
    norm_row_far<RES>(x, weight, rstd, row, k, kb, 8 * (int64_t)blockDim.x, P, h_out, codes, scales);
}

// Rows longer than the registers of one workgroup hold: two passes, the second
// reads h (or x) again.
template <bool RES>
__global__ void __launch_bounds__(1024) rmsnorm_fp8_long_kernel(const uint16_t* __restrict__ x,
                                                                const uint16_t* residual,
                                                                const uint16_t* __restrict__ weight, float eps,
                                                                int64_t rows, int64_t k, uint16_t* h_out,
                                                                uint8_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
  const int64_t row = blockIdx.x + (int64_t)blockIdx.y * gridDim.x, kb = (k + 127) / 128;
  if (row >= rows) return;
  float ss = 0.0f;
  for (int64_t col = 8 * threadIdx.x; col < k; col += 8 * 1024) {
    uint4 h = *reinterpret_cast<const uint4*>(x + row * k + col);
    if constexpr (RES) {
      h = add8(h, *reinterpret_cast<const uint4*>(residual + row * k + col));
      *reinterpret_cast<uint4*>(h_out + row * k + col) = h;
    }
    ss += sum_squares(h);
  }
  ss = wg_sum(ss);
  const float rstd = 1.0f / __builtin_sqrtf(ss / (float)k + eps);
  const bool finite = (__float_as_uint(ss) & kInfBits) != kInfBits;
  // Each thread reads back the pieces that it stored itself.
  bool far = false;
  for (int64_t c0 = 0; c0 < k; c0 += 8 * 1024) {
    const int64_t col = c0 + 8 * threadIdx.x;
    const bool in = col < k;
    const uint4 h = in ? *reinterpret_cast<const uint4*>((RES ? h_out : x) + row * k + col) : make_uint4(0, 0, 0, 0);
    far |= norm_store(h, weight, col, in, rstd, finite, row, k, kb, codes, scales);
  }
  if (__builtin_amdgcn_ballot_w64(far) != 0)
    norm_row_far<RES>(x, weight, rstd, row, k, kb, 8 * 1024, (k + 8 * 1024 - 1) / (8 * 1024), h_out, codes, scales);
}

}  // namespace

// A launch has at most 2^32 threads along x: more workgroups go to y (the last
// row of the grid may hold spare ones).
static dim3 grid2(int64_t wgs) {
  constexpr int64_t kX = 1 << 20;
  return wgs <= kX ? dim3((unsigned)wgs) : dim3((unsigned)kX, (unsigned)((wgs + kX - 1) / kX));
}

template <bool SILU, int U>
static void launch_rows(const uint16_t* x, int64_t blocks, int64_t kb, int64_t k, uint8_t* codes, float* scales,
                        hipStream_t s) {
  const int64_t wgs = (blocks + 16 * U - 1) / (16 * U);
  const dim3 grid((unsigned)(wgs < (1 << 22) ? wgs : 1 << 22));
  if (kb >= 16 * U && k < ((int64_t)1 << 28))
    fp8_rows_kernel<SILU, U, true><<<grid, kThreads, 0, s>>>(x, blocks, (uint32_t)kb, k, codes, scales);
  else if constexpr (U != 2)  // two blocks a thread only for kb of 32 to 63
    fp8_rows_kernel<SILU, U, false><<<grid, kThreads, 0, s>>>(x, blocks, (uint32_t)kb, k, codes, scales);
}

// Blocks per thread: one for few blocks (latency), else as many as keep a
// workgroup within two rows ([2048, 2 x 17408] silu, us: 1 block 47.3, 2 41.0, 4
// 39.8).
template <bool SILU>
static void launch_rows_any(const uint16_t* x, int64_t rows, int64_t k, uint8_t* codes, float* scales, hipStream_t s) {
  const int64_t kb = (k + 127) / 128, blocks = rows * kb;
  if (blocks <= 32768 || (kb >= 16 && kb < 32)) launch_rows<SILU, 1>(x, blocks, kb, k, codes, scales, s);
  else if (kb >= 32 && kb < 64) launch_rows<SILU, 2>(x, blocks, kb, k, codes, scales, s);
  else launch_rows<SILU, 4>(x, blocks, kb, k, codes, scales, s);
}

void launch_fp8_quantize_rows(const uint16_t* x, int64_t rows, int64_t k, uint8_t* codes, float* scales,
                              hipStream_t s) {
  launch_rows_any<false>(x, rows, k, codes, scales, s);
}

void launch_fp8_quantize_tiles(const uint16_t* w, int64_t count, int64_t n, int64_t k, uint8_t* codes, float* scales,
                               hipStream_t s) {
  const int64_t nb = (n + 127) / 128, kb = (k + 127) / 128, blocks = count * nb * kb;
  fp8_tiles_kernel<<<grid2(blocks), kThreads, 0, s>>>(w, n, k, nb, kb, blocks, codes, scales);
}

void launch_silu_mul_fp8(const uint16_t* gate_up, int64_t rows, int64_t n, uint8_t* codes, float* scales,
                         hipStream_t s) {
  launch_rows_any<true>(gate_up, rows, n, codes, scales, s);
}

template <bool RES>
static void launch_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, int64_t rows,
                        int64_t k, uint16_t* h, uint8_t* codes, float* scales, hipStream_t s) {
  const int64_t pieces = (k + 127) / 128 * 16;
  const dim3 grid = grid2(rows);
  const auto threads = [&](int64_t p) { return dim3((unsigned)(((pieces + p - 1) / p + 63) / 64 * 64)); };
  // Pieces per thread: one for few rows (8 x 5120: 3.5 us against 4.2 with three),
  // three for many (2048 x 5120: 16.7 us against 19.3, 17.2, 17.4 with 1, 2, 4).
  if (pieces <= 1024 && rows <= 512)
    rmsnorm_fp8_kernel<1, RES><<<grid, threads(1), 0, s>>>(x, residual, weight, eps, rows, k, h, codes, scales);
  else if (pieces <= 3 * 1024)
    rmsnorm_fp8_kernel<3, RES><<<grid, threads(3), 0, s>>>(x, residual, weight, eps, rows, k, h, codes, scales);
  else if (pieces <= 4 * 1024)
    rmsnorm_fp8_kernel<4, RES><<<grid, threads(4), 0, s>>>(x, residual, weight, eps, rows, k, h, codes, scales);
  else
    rmsnorm_fp8_long_kernel<RES><<<grid, 1024, 0, s>>>(x, residual, weight, eps, rows, k, h, codes, scales);
}

void launch_rmsnorm_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, int64_t rows,
                        int64_t k, uint16_t* residual_out, uint8_t* codes, float* scales, hipStream_t s) {
  if (residual) launch_norm<true>(x, residual, weight, eps, rows, k, residual_out, codes, scales, s);
  else launch_norm<false>(x, residual, weight, eps, rows, k, residual_out, codes, scales, s);
}

}  // namespace nvfp4
