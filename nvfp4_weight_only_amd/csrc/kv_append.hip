// Appending rows to a paged FP4 cache of keys and values, the keys turned by
// their position on the way (kv_common.hpp has the cache, the batch and the angles).
//
// Row r of sequence s goes to token t = seq_lens[s] - (row_start[s + 1] - r): page
// block_table[s, t / block_size], slot t % block_size.  Per block of G elements:
//   NVFP4  scale = the E4M3 value nearest to amax / (6 tscale), at most 448,
//          code = sign, E2M1 magnitude nearest to |x| / (scale tscale), at most 6;
//   MXFP4  scale byte = clamp(floor(log2 amax) - 2 + 127, 0, 254),
//          code = sign, E2M1 magnitude nearest to |x| / 2^(byte - 127), at most 6;
// ties to the even code, on the exact quotients.  The rotated key is computed in FP64
// and rounded to FP32 once, so that its codes do not hang on the rounding of an
// intermediate 16-bit key.  A block with a value that is not finite gets a NaN scale
// (0x7F, 0xFF) and codes 0.
//
// A thread makes the codes of 8 elements (16 bytes in, 4 bytes out), 2 or 4
// neighbouring threads a block; for a rotated key it also loads the piece that holds
// the other half of its pairs, which a neighbour of the same workgroup loads too.
#include "kv_common.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 8;       // rows of a workgroup at most
constexpr int kAppendAngles = 1024;  // in LDS at a time

struct AppendArgs {
  KvCache c;
  KvBatch b;
  FastDiv page;
  int64_t cap;  // max_blocks * block_size
  const uint16_t* x[2];
  int64_t row_stride[2], head_stride[2];
  RopeArgs rope;
  const int32_t* positions;  // or null: the token's place
  int32_t pieces;            // 8-element pieces of a head
  int32_t rows_wg;
};

// FP32 value on the same side of every FP32 value as the exact quotient that q
// approximates to 2^-51: quotients here are of at most 24 by 28 significant bits, so
// one that is no FP32 value of few bits is at least 2^-32 away from it.  q is rounded
// to 2^-41, which makes such a value exact again, then to odd: what is cut off leaves
// its trace in the last bit.
__device__ __forceinline__ float quotient_f32(double q) {
  const uint64_t b = (__builtin_bit_cast(uint64_t, q) + 0x800u) & ~(uint64_t)0xFFFu;
  float f = (float)__builtin_bit_cast(double, b & ~(uint64_t)0x1FFFFFFFu);
  f = __builtin_amdgcn_fmed3f(f, -0x1p100f, 0x1p100f);  // an infinity is no quotient's neighbour
  return __uint_as_float(__float_as_uint(f) | ((uint32_t)b & 0x1FFFFFFFu ? 1u : 0u));
}

// 1 / d for a normal d > 0, to 2^-51.
__device__ __forceinline__ double recip_f64(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = fma(fma(-d, y, 1.0), y, y);
  return fma(fma(-d, y, 1.0), y, y);
}

// Codes of 8 values that the 2 (NVFP4) or 4 (MXFP4) threads of a block hold together.
template <bool MX>
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], float ts, uint32_t* scale_code) {
  uint32_t amax = 0;  // magnitude bits: NaN above infinity above every number
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < (MX ? 4 : 2); d <<= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, d, 64));
  if (amax >= 0x7F800000u) {
    *scale_code = MX ? 0xFFu : 0x7Fu;
    return 0;
  }
  float q[8];
  if constexpr (MX) {
    // floor(log2 amax) of a normal amax is its exponent field - 127.
    const int ef = (int)(amax >> 23), e = ef <= 2 ? 0 : ef - 2;
    *scale_code = (uint32_t)e;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __builtin_amdgcn_ldexpf(v[i], 127 - e);
  } else {
    const double t = (double)ts;
    const float r = quotient_f32((double)__uint_as_float(amax) * recip_f64(6.0 * t));
    const uint32_t sc = amax ? (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fminf(r, 448.0f), 0.0f, 0, false) & 0xFFu : 0u;
    *scale_code = sc;
    const double k = sc ? recip_f64((double)e4m3_to_f32(sc) * t) : 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quotient_f32((double)v[i] * k);
  }
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, q[0], q[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
}

template <bool BF16>
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = half_to_f32<BF16>(w[i] & 0xFFFFu);
    v[2 * i + 1] = half_to_f32<BF16>(w[i] >> 16);
  }
}

// Workgroup b: rows b * rows_wg and on.  First its rows' places, by a wavefront that
// looks for the last sequence that starts at or before the row; then the angles; then
// the codes.
template <bool MX, bool BF16>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(AppendArgs a) {
  __shared__ double2 turn[kAppendAngles];
  __shared__ int64_t place[kAppendRows];  // row of [num_blocks * block_size], or -1
  __shared__ int32_t token[kAppendRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_wg;
  const int nrows = (int)(a.b.rows - r0 < a.rows_wg ? a.b.rows - r0 : a.rows_wg);
  for (int i = wave; i < nrows; i += kAppendThreads / 64) {
    const int64_t r = r0 + i;
    int64_t s = r;
    if (a.b.row_start) s = find_sequence(a.b, r, lane);
    int64_t at = -1, t = -1;
    if (s < a.b.seqs) {
      const SeqRows q = seq_rows(a.b, a.cap, s);
      t = r + q.shift;
      if (r >= q.first && r < q.first + q.count && t >= 0 && t < q.len) {
        const int32_t page = fastdiv((int32_t)t, a.page);
        const int64_t id = a.b.block_table[s * a.b.max_blocks + page];
        if (id >= 0 && id < a.c.num_blocks) at = id * a.c.block_size + (t - (int64_t)page * a.c.block_size);
      }
    }
    if (lane == 0) {
      place[i] = at;
      token[i] = (int32_t)t;
    }
  }
  __syncthreads();
  const int half = (int)a.rope.rot / 2;
  for (int i = tid; i < nrows * half; i += kAppendThreads) {
    const int r = i / half, f = i - r * half;
    if (place[r] < 0) continue;
    const int32_t pos = a.positions ? a.positions[r0 + r] : token[r];
    double sn, cs;
    sincos_f64((double)pos * a.rope.freqs[f], &sn, &cs);
    turn[i] = make_double2(cs * (double)a.rope.amplitude, sn * (double)a.rope.amplitude);
  }
  __syncthreads();
  const int per_head = a.pieces, per_tensor = (int)a.c.heads * per_head, per_row = 2 * per_tensor;
  const int group = MX ? 32 : 16;
  for (int i = tid; i < nrows * per_row; i += kAppendThreads) {
    const int r = i / per_row, j = i - r * per_row, which = j >= per_tensor ? 1 : 0, k = j - which * per_tensor;
    const int h = k / per_head, p = k - h * per_head;
    const int64_t at = place[r];
    if (at < 0) continue;  // all threads of a block together
    const uint16_t* x = a.x[which] + (r0 + r) * a.row_stride[which] + h * a.head_stride[which];
    float v[8];
    load8<BF16>(x + 8 * p, v);
    if (which == 0 && 8 * p < (int)a.rope.rot) {
      const double2* cs = turn + r * half;
      if (a.rope.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double2 t = cs[4 * p + e];
          const double x1 = v[2 * e], x2 = v[2 * e + 1];
          v[2 * e] = (float)(x1 * t.x - x2 * t.y);
          v[2 * e + 1] = (float)(x2 * t.x + x1 * t.y);
        }
      } else {
        const bool first = 8 * p < half;
        float w[8];
        load8<BF16>(x + (first ? 8 * p + half : 8 * p - half), w);
        const int f = first ? 8 * p : 8 * p - half;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double2 t = cs[f + e];
          const double other = (double)w[e] * t.y;
          v[e] = (float)(first ? (double)v[e] * t.x - other : (double)v[e] * t.x + other);
        }
      }
    }
    uint32_t sc;
    const uint32_t codes = encode8<MX>(v, MX ? 1.0f : *a.c.tscale[which], &sc);
    const int64_t row = at * a.c.heads + h;
    reinterpret_cast<uint32_t*>(a.c.codes[which] + row * (a.c.head_dim / 2))[p] = codes;
    if ((8 * p) % group == 0) a.c.scales[which][row * (a.c.head_dim / group) + 8 * p / group] = (uint8_t)sc;
  }
}

}  // namespace

void launch_kv_append(const KvCache& c, const KvBatch& b, bool bf16, const uint16_t* k, const uint16_t* v,
                      int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head, const RopeArgs& rope,
                      const int32_t* positions, hipStream_t s) {
  AppendArgs a;
  a.c = c;
  a.b = b;
  a.page = make_fastdiv(c.block_size);
  a.cap = b.max_blocks * c.block_size;
  a.x[0] = k;
  a.x[1] = v;
  a.row_stride[0] = k_row;
  a.row_stride[1] = v_row;
  a.head_stride[0] = k_head;
  a.head_stride[1] = v_head;
  a.rope = rope;
  a.positions = positions;
  a.pieces = (int32_t)(c.head_dim / 8);
  const int64_t per_row = 2 * c.heads * a.pieces;
  int64_t n = (1024 + per_row - 1) / per_row;
  n = n < kAppendRows ? n : kAppendRows;
  if (rope.rot > 0 && n > 2 * kAppendAngles / rope.rot) n = 2 * kAppendAngles / rope.rot;
  while (n > 1 && (b.rows + n - 1) / n < 1024) --n;
  a.rows_wg = (int32_t)n;
  const dim3 grid((unsigned)((b.rows + n - 1) / n));
  if (c.mx) {
    if (bf16) kv_append_kernel<true, true><<<grid, kAppendThreads, 0, s>>>(a);
    else kv_append_kernel<true, false><<<grid, kAppendThreads, 0, s>>>(a);
  } else {
    if (bf16) kv_append_kernel<false, true><<<grid, kAppendThreads, 0, s>>>(a);
    else kv_append_kernel<false, false><<<grid, kAppendThreads, 0, s>>>(a);
  }
}

}  // namespace nvfp4
