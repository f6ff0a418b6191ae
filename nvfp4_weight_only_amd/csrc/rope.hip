// Rotary positions: the first `rot` elements of every head turned by an angle that
// grows with the row's position,
//   (x1, x2) -> a (x1 cos t - x2 sin t, x2 cos t + x1 sin t),  t = position * freqs[i],
// for the pairs (i, i + rot / 2) or, interleaved, (2 i, 2 i + 1), i < rot / 2; the
// inverse turns by -t.  Elements behind the first `rot` are copied.
//
// Bound by memory: each element is read and written once.  A row's rot / 2 angles are
// the same for all its heads, so a workgroup takes whole rows, computes their sines
// and cosines once into LDS (FP64 angles, kv_common.hpp; FP32 factors) and streams the
// heads past them, 16 elements a thread at a time: the two 8-element pieces that hold
// 8 pairs.  Products in FP32, one rounding to 16 bits.
//
// Measured: 8192 rows of 40 heads of 128 31 us, 5.3 TB/s (a large copy reaches 5.1);
// 8 rows 3.6 us, a dependent chain of position, angle, sine and store.
#include "kv_common.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeAngles = 2048;  // in LDS at a time

struct RopeKernelArgs {
  const uint16_t* x;
  uint16_t* out;
  int64_t rows;
  int32_t heads, head_dim, rot;
  int64_t xr, xh, yr, yh;  // strides of rows and heads, in elements
  const int32_t* positions;
  const double* freqs;
  float amplitude, sign;  // sign -1: inverse
  int32_t rows_wg;        // rows a workgroup takes
  int32_t items;          // 16-element items of a head: rot / 16 rotated, then copied pieces of 8
};

template <bool BF16>
__device__ __forceinline__ uint4 rope_pack(const float (&v)[8]) {
  return make_uint4(f32x2_to_half<BF16>(v[0], v[1]), f32x2_to_half<BF16>(v[2], v[3]),
                    f32x2_to_half<BF16>(v[4], v[5]), f32x2_to_half<BF16>(v[6], v[7]));
}
template <bool BF16>
__device__ __forceinline__ void rope_unpack(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = half_to_f32<BF16>(w[i] & 0xFFFFu);
    v[2 * i + 1] = half_to_f32<BF16>(w[i] >> 16);
  }
}

template <bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeKernelArgs a) {
  __shared__ float2 turn[kRopeAngles];  // (cos, sin) times the amplitude
  const int tid = threadIdx.x, half = a.rot / 2;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_wg;
  const int nrows = (int)(a.rows - r0 < a.rows_wg ? a.rows - r0 : a.rows_wg);
  for (int i = tid; i < nrows * half; i += kRopeThreads) {
    const int r = i / half, f = i - r * half;
    double sn, cs;
    sincos_f64((double)a.positions[r0 + r] * a.freqs[f], &sn, &cs);
    turn[i] = make_float2((float)cs * a.amplitude, (float)sn * a.amplitude * a.sign);
  }
  __syncthreads();
  const int rotated = a.rot / 16, per_row = a.heads * a.items;
  for (int i = tid; i < nrows * per_row; i += kRopeThreads) {
    const int r = i / per_row, j = i - r * per_row, h = j / a.items, p = j - h * a.items;
    const uint16_t* x = a.x + (r0 + r) * a.xr + h * a.xh;
    uint16_t* y = a.out + (r0 + r) * a.yr + h * a.yh;
    if (p >= rotated) {
      const int e = a.rot + (p - rotated) * 8;
      *reinterpret_cast<uint4*>(y + e) = *reinterpret_cast<const uint4*>(x + e);
      continue;
    }
    const int e1 = INTERLEAVED ? 16 * p : 8 * p, e2 = INTERLEAVED ? e1 + 8 : e1 + half;
    float u[8], v[8], s[8], t[8];
    rope_unpack<BF16>(*reinterpret_cast<const uint4*>(x + e1), u);
    rope_unpack<BF16>(*reinterpret_cast<const uint4*>(x + e2), v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 cs = turn[r * half + 8 * p + k];
      if constexpr (INTERLEAVED) {
        const float a1 = k < 4 ? u[2 * (k & 3)] : v[2 * (k & 3)], a2 = k < 4 ? u[2 * (k & 3) + 1] : v[2 * (k & 3) + 1];
        (k < 4 ? s : t)[2 * (k & 3)] = a1 * cs.x - a2 * cs.y;
        (k < 4 ? s : t)[2 * (k & 3) + 1] = a2 * cs.x + a1 * cs.y;
      } else {
        s[k] = u[k] * cs.x - v[k] * cs.y;
        t[k] = v[k] * cs.x + u[k] * cs.y;
      }
    }
    *reinterpret_cast<uint4*>(y + e1) = rope_pack<BF16>(s);
    *reinterpret_cast<uint4*>(y + e2) = rope_pack<BF16>(t);
  }
}

// Angular frequencies, base^(-2 i / rot) changed for contexts longer than the
// one trained on (factor times as long):
//   linear      / factor                      (positions interpolated)
//   base        base * factor^(rot / (rot - 2)) for base: the slowest is slowed by factor, the fastest kept
//   ramp        kept where a wavelength fits `high` times into the original length, / factor where it fits
//               less than `low` times, in between a mean whose weight runs linearly over the index i
//   wavelength  the same bounds, the weight running linearly over original / wavelength
__global__ void __launch_bounds__(64) rope_frequencies_kernel(int scaling, int64_t rot, double base, double factor,
                                                              double original, double low, double high,
                                                              double* freqs) {
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= rot / 2) return;
  const double two_pi = 6.283185307179586477;
  if (scaling == 2) base *= pow(factor, (double)rot / (double)(rot - 2));
  const double f = pow(base, -2.0 * (double)i / (double)rot);
  double slow = 0.0;  // weight of f / factor
  if (scaling == 1) slow = 1.0;
  if (scaling == 3) {
    // The index whose wavelength fits `turns` times into the original length.
    const auto index = [&](double turns) { return (double)rot * log(original / (turns * two_pi)) / (2.0 * log(base)); };
    const double first = fmax(floor(index(high)), 0.0);
    const double last = fmin(ceil(index(low)), (double)(rot - 1));
    slow = fmin(fmax(((double)i - first) / fmax(last - first, 0.001), 0.0), 1.0);
  }
  if (scaling == 4) {
    const double turns = original * f / two_pi;
    slow = fmin(fmax((high - turns) / (high - low), 0.0), 1.0);
  }
  freqs[i] = scaling == 1 ? f / factor : f * (1.0 - slow) + f / factor * slow;
}

}  // namespace

void launch_rope(bool bf16, const uint16_t* x, int64_t rows, int64_t heads, int64_t head_dim, int64_t x_row,
                 int64_t x_head, const int32_t* positions, const RopeArgs& rope, bool inverse, uint16_t* out,
                 int64_t out_row, int64_t out_head, hipStream_t s) {
  RopeKernelArgs a;
  a.x = x;
  a.out = out;
  a.rows = rows;
  a.heads = (int32_t)heads;
  a.head_dim = (int32_t)head_dim;
  a.rot = (int32_t)rope.rot;
  a.xr = x_row;
  a.xh = x_head;
  a.yr = out_row;
  a.yh = out_head;
  a.positions = positions;
  a.freqs = rope.freqs;
  a.amplitude = rope.amplitude;
  a.sign = inverse ? -1.0f : 1.0f;
  // In place the elements behind the rotated ones stay where they are.
  a.items = (int32_t)(rope.rot / 16 + (x == out ? 0 : (head_dim - rope.rot) / 8));
  const int64_t per_row = heads * a.items;
  int64_t n = (1024 + per_row - 1) / per_row;
  const int64_t fit = kRopeAngles / (rope.rot / 2);
  n = n < fit ? n : fit;
  while (n > 1 && (rows + n - 1) / n < 1024) --n;
  a.rows_wg = (int32_t)n;
  const dim3 grid((unsigned)((rows + n - 1) / n));
  if (bf16) {
    if (rope.interleaved) rope_kernel<true, true><<<grid, kRopeThreads, 0, s>>>(a);
    else rope_kernel<true, false><<<grid, kRopeThreads, 0, s>>>(a);
  } else {
    if (rope.interleaved) rope_kernel<false, true><<<grid, kRopeThreads, 0, s>>>(a);
    else rope_kernel<false, false><<<grid, kRopeThreads, 0, s>>>(a);
  }
}

void launch_rope_frequencies(int scaling, int64_t rot, double base, double factor, double original, double low,
                             double high, double* freqs, hipStream_t s) {
  rope_frequencies_kernel<<<dim3((unsigned)((rot / 2 + 63) / 64)), 64, 0, s>>>(scaling, rot, base, factor, original,
                                                                               low, high, freqs);
}

}  // namespace nvfp4
