// The parts of attention over a paged FP4 cache that its kernels share: arguments,
// the loads and the decoding of cache rows, the partial results and their join.
//
// For a row at position p of its sequence and a query head with key/value head h,
//   o = tscale_v sum_t w_t v_t / sum_t w_t,  w_t = exp(scale tscale_k q . k_t),
// over the tokens t <= p (and t > p - window) that are in the cache, k and v without
// their tensor scales.  The sums run over tiles of tokens with the running maximum m,
// the sum l of 2^(s - m) and the unnormalized output, all in FP32; parts of the tokens
// that different wavefronts or workgroups took are joined by their m, l and output.
//
// What the matrix cores multiply.  NVFP4: E2M1 * E4M3 has at most 6 significant bits
// and lies in [2^-10, 2688], so keys and values are exact in FP16, where a pair of
// codes takes one conversion and one packed product.  The query's row is divided by the
// power of two of its largest element, so that any BF16 or FP16 row fits FP16 (what
// lies 2^14 below the largest loses bits, less than 2^-25 of the largest) and the products'
// range hangs on the keys alone.  MXFP4: E2M1 * 2^(byte - 127) needs BF16's range and is
// exact there, in one conversion a pair (bytes 253 and 254, whose blocks pass FP32's range,
// count as NaN).  A BF16 query is exact too; an FP16 one is split into two BF16 terms.
//
// Weights are two terms of the matrix type, 22 bits (FP16) or 16 (BF16), so that their
// rounding stays far below the output's: with one, the distance from the exact result grew
// by a quarter to a third for FP16 outputs of NVFP4 and BF16 ones of MXFP4 (9 streams with a
// chunk of 256 rows: 2.67e-4 instead of 2.07e-4, 2.12e-3 instead of 1.66e-3 of the
// outputs' norm).  The second term takes 1.5 of 36 us at 16 streams of up to 8192 tokens,
// where memory bounds, and 80 of 410 at 2048 rows behind 6144 (MXFP4, BF16), where products
// do; so many rows of NVFP4 with BF16 outputs keep one, 11 bits under an output of 8 (1.669e-3
// and 1.660e-3).
#pragma once

#include "kv_common.hpp"
#include "kv_masks.hpp"

namespace nvfp4 {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));

// MXFP4 scale bytes from here on count as NaN: 6 * 2^(253 - 127) is beyond FP32.
constexpr uint32_t kMxNan = 253;

// Weights are 2^(s - m + bias) with m at most kSlack (log2 units) below the running
// maximum.  FP16: bias 7, so up to 2^15, its last power of two: a weight 2^21 below the
// largest is still a normal number, and below that it is off by at most 2^-32 of the
// largest (without the bias by 2^-25, which 10^5 small weights add up to something seen).
// BF16 has FP32's range: bias -8, so up to 1, as a softmax's own, and the sum over n tokens
// of MXFP4 values v stays in range while n |v| is below 2^128 (a lower bias would allow more
// and lose small weights instead).  Sums keep the bias; it cancels in the quotient.
//
// From kFar on FP32's step is half a unit and more: there a step of 8, the bias beside the
// maximum and the product with the row's factor would each be rounded by so much that weights
// pass 2^15 (scores of 2^24 and more gave infinite weights in FP16).  A wavefront with such a
// maximum takes the differences from it first, rounded products on both sides, which are at
// most 0, and scales again whenever it grows (looking for it takes 1.4 % of the time of 2048
// rows behind 6144 tokens).
constexpr float kSlack = 8.0f;
constexpr float kFar = 4194304.0f;  // 2^22
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar && m > -__builtin_inff(); }
// A score's difference from a maximum that no score passes; NaN stays.
__device__ __forceinline__ float below(float score, float m) {
  const float x = score - (m == -__builtin_inff() ? 0.0f : m);
  return x > 0.0f ? 0.0f : x;
}
template <bool MX>
constexpr float weight_bias() {
  return MX ? -kSlack : 7.0f;
}

struct AttendArgs {
  KvCache c;
  KvBatch b;
  FastDiv page, group, unit;  // block_size, g, tokens of a unit
  int64_t cap;  // max_blocks * block_size
  const uint16_t* q;
  int64_t q_row, q_head;
  uint16_t* out;  // [rows, q_heads, head_dim]
  int32_t q_heads, g;  // g = q_heads / heads
  float scale;
  int32_t window;  // 0: none
  int32_t hw, tw, hgroups;  // heads and token slices of a workgroup, groups of heads
  int32_t nwg;              // workgroups of a group of heads
  int32_t least;            // units of a workgroup, where there are few
  float* part;              // partial results
  int64_t* prefix;          // [seqs + 1] units before each sequence
};

// Many rows a sequence (kv_attend_many.hip): one workgroup a CU.
constexpr int kManyWorkgroups = 256;
int64_t kv_attend_many_workspace_bytes(int64_t head_dim, int64_t g, int64_t rows, int64_t seqs);
void launch_kv_attend_many(const AttendArgs& a, bool bf16, void* workspace, hipStream_t s);

// Terms of the matrix type that a query and a weight take, by format and query type; MANY: the kernel for many rows.
template <bool MX, bool BF16, bool MANY>
struct AttendTerms {
  static constexpr int kQuery = MX && !BF16 ? 2 : 1;
  static constexpr int kWeight = MANY && !MX && BF16 ? 1 : 2;
};

// D = A B + C on 16 x 16 x 32 (A: 16 tokens or dims; B: 16 rows of queries).
template <bool MX>
__device__ __forceinline__ f32x4_t mfma16(const u32x4v_t& a, const u32x4v_t& b, const f32x4_t& c) {
  if constexpr (MX)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

// Two floats as the matrix type.
template <bool MX>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return f32x2_to_half<MX>(a, b);
}
// What the first term left out, as the matrix type.
template <bool MX>
__device__ __forceinline__ uint32_t pack2_rest(float a, float b, uint32_t first) {
  if constexpr (MX) return f32x2_to_half<true>(a - bf16_to_f32(first & 0xFFFFu), b - __uint_as_float(first & 0xFFFF0000u));
  const f16x2_t f = __builtin_bit_cast(f16x2_t, first);  // one mixed product and sum each
  return f32x2_to_half<false>(__builtin_fmaf((float)f[0], -1.0f, a), __builtin_fmaf((float)f[1], -1.0f, b));
}

// Scale bytes that a lane needs of a row whose quarter (NS pieces of 8 elements) it holds, and where they are.
template <bool MX, int NS>
struct ScaleBytes {
  static constexpr int kRow = MX ? NS : 2 * NS;  // bytes of a row: head_dim = 32 NS
  static constexpr int kShift = MX ? 2 : 1;      // log2 pieces a block
  // Blocks that NS pieces from quarter * NS on touch at most.
  static constexpr int kLoad = MX ? (NS <= 2 || NS == 4 ? 1 : 2) : (NS == 3 ? 2 : NS / 2);
  static __device__ __forceinline__ int base(int quarter) {
    const int b = (quarter * NS) >> kShift;
    return b + kLoad > kRow ? kRow - kLoad : b;
  }
  // Bytes of all quarters side by side: a quarter's start is at a multiple of kLoad.
  static constexpr bool kEven = 4 * kLoad == kRow;
  // Byte of piece c in the loaded word.
  static __device__ __forceinline__ int index(int quarter, int c) {
    if constexpr ((NS * 1) % (1 << kShift) == 0 || (MX && NS == 2)) return MX && NS == 2 ? 0 : c >> kShift;
    else return ((quarter * NS + c) >> kShift) - base(quarter);
  }
  static __device__ __forceinline__ uint32_t load(const uint8_t* p) {
    if constexpr (kLoad == 1) return *p;
    if constexpr (kLoad == 2) return (uint32_t)p[0] | (uint32_t)p[1] << 8;
    if constexpr (kLoad == 3) return (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16;
    return *reinterpret_cast<const uint32_t*>(p);
  }
};
// With an even number of bytes the row's offset is even, and the load is one.
template <>
__device__ __forceinline__ uint32_t ScaleBytes<false, 4>::load(const uint8_t* p) {
  return *reinterpret_cast<const uint16_t*>(p);
}
template <>
__device__ __forceinline__ uint32_t ScaleBytes<true, 8>::load(const uint8_t* p) {
  return *reinterpret_cast<const uint16_t*>(p);
}

// Whether a block with this scale byte holds values that are not finite.
template <bool MX>
__device__ __forceinline__ bool scale_nonfinite(uint32_t byte) {
  return MX ? byte >= kMxNan : (byte & 0x7Fu) == 0x7Fu;
}

// The scale bytes with those of NaN blocks set to 0.
template <bool MX>
__device__ __forceinline__ uint32_t drop_nan(uint32_t word) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (scale_nonfinite<MX>((word >> (8 * i)) & 0xFFu)) word &= ~(0xFFu << (8 * i));
  return word;
}

// 8 codes times their block's scale in the matrix type, natural order.
__device__ __forceinline__ u32x4v_t decode8_nv(uint32_t w, f16x2_t s) {
  const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s;
  const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s;
  const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s;
  const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s;
  return u32x4v_t{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                  __builtin_bit_cast(uint32_t, d)};
}
// The conversion multiplies by the scale's exponent alone: byte 0 is 2^-127, 255 NaN.
__device__ __forceinline__ u32x4v_t decode8_mx(uint32_t w, float s) {
  return u32x4v_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
}

// A lane's quarter of a cache row: NS pieces of 8.
template <bool MX, int NS>
__device__ __forceinline__ void decode_quarter(const uint32_t (&w)[NS], uint32_t sw, int quarter, u32x4v_t (&out)[NS]) {
  using B = ScaleBytes<MX, NS>;
  if constexpr (MX) {
#pragma unroll
    for (int c = 0; c < NS; ++c) {
      const uint32_t byte = (sw >> (8 * B::index(quarter, c))) & 0xFFu;
      out[c] = decode8_mx(w[c], __uint_as_float((byte >= kMxNan ? 255u : byte) << 23));
    }
  } else {
    const f16x2_t s01 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, false);
    f16x2_t s23 = s01;
    if constexpr (B::kLoad > 2) s23 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, true);
#pragma unroll
    for (int c = 0; c < NS; ++c) {
      const int i = B::index(quarter, c);
      const f16x2_t pair = i >= 2 ? s23 : s01;
      const _Float16 s = i & 1 ? pair[1] : pair[0];
      out[c] = decode8_nv(w[c], f16x2_t{s, s});
    }
  }
}

// A row of queries' scale: s = factor * (the product of the matrix type's values) in
// units of log2; the query's elements times `mul`, which brings the largest to 1 .. 2.
// The factor in FP64, since the product of two scales and the row's power of two can leave
// FP32's range on the way where the scores do not.
struct RowScale {
  float factor, mul;
};
__device__ __forceinline__ RowScale row_scale(float amax, float scale, float ts) {
  const double c = (double)scale * (double)ts * 1.4426950408889634074;  // log2 e
  double f = fabs(c);
  RowScale r;
  r.mul = c < 0.0 ? -1.0f : 1.0f;
  const uint32_t e = __float_as_uint(amax) >> 23;  // amax >= 0
  if (amax > 0.0f && e < 255u) {
    const int n = (int)e - 127;  // FP32 subnormals (e = 0) by 2^-127
    f = __builtin_amdgcn_ldexp(f, n);
    r.mul = __builtin_amdgcn_ldexpf(r.mul, -n);
  }
  // With an infinity in the query every score is one or NaN, and the softmax NaN, also where all are -inf, which would
  // count as masked.
  if (e == 255u) r.mul = __builtin_nanf("");
  // A factor beyond FP32 makes scores of any keys but tiny ones overflow or lie far beyond exp2's range from each other.
  constexpr double kMax = 3.4028234663852886e38;
  r.factor = f > kMax && f < __builtin_inf() ? (float)kMax : (float)f;
  // A factor of 0 goes to the query, so that a masked score, -inf, times the factor stays -inf.
  if (r.factor == 0.0f) {
    r.factor = 1.0f;
    r.mul = 0.0f;
  }
  return r;
}

// What a sequence takes: tiles of rows times units of tokens.
struct SeqWork {
  int32_t first, packed;  // first row, rows times g
  int32_t pos;            // token of the first row (negative: it sees nothing)
  int32_t lo, hi;         // tokens that some row sees: lo a multiple of 32
  int32_t rtiles, ttiles;
};
template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int32_t s) {
  const SeqRows r = seq_rows(a.b, a.cap, s);
  SeqWork w;
  w.first = (int32_t)r.first;
  w.packed = (int32_t)r.count * a.g;
  const int64_t p0 = r.first + r.shift, p1 = p0 + r.count;
  w.pos = p0 < -a.b.rows ? -(int32_t)a.b.rows : (int32_t)p0;  // every row of such a sequence is below token 0
  w.hi = (int32_t)(p1 < 0 ? 0 : (p1 < r.len ? p1 : r.len));
  w.lo = first_tile(p0, a.window, 32, w.hi);
  w.rtiles = (w.packed + ROWS - 1) / ROWS;
  // A sequence whose rows see nothing still has its zeros to write.
  w.ttiles = w.hi > w.lo ? fastdiv(w.hi - w.lo + a.unit.d - 1, a.unit) : 1;
  return w;
}

// Workgroups that share `total` units: workgroup w of n takes units
// w total / n up to (w + 1) total / n.
__device__ __forceinline__ int32_t sharing(const AttendArgs& a, int64_t total) {
  return total < (int64_t)a.nwg * a.least ? ((int32_t)total + a.least - 1) / a.least : a.nwg;
}

// Outputs from sums over tokens and the weights' sum (0: the row sees nothing).  The tensor scale last: its quotient by
// the sum would lose bits below FP32's range where the outputs do not.
__device__ __forceinline__ f32x4_t finish(const f32x4_t& v, float sum, float ts) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  return v * inv * (sum == 0.0f ? 0.0f : ts);
}

// 4 outputs of a row.
template <bool BF16>
__device__ __forceinline__ void store_out4(uint16_t* p, const f32x4_t& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(f32x2_to_half<BF16>(v[0], v[1]), f32x2_to_half<BF16>(v[2], v[3]));
}

}  // namespace nvfp4
