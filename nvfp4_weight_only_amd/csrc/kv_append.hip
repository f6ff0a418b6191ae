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
//
// Measured: 2048 rows of 8 heads of 128 (NVFP4) 7.0 us, 16384 (MXFP4) 25 us, 3.4 TB/s.
// Bound by a workgroup's chain of dependent loads (start, length, page, frequency), which
// its row loads overlap, and by vector instructions (40 % of the clocks at 16384 rows): 4
// pieces a thread, 120 registers, 4 wavefronts a SIMD.  With 2 pieces 45 us, with 8 28;
// held to 96 registers 26, to 80 36 (spills).
#include "kv_common.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

constexpr int kAppendThreads = 256;  // at most
constexpr int kAppendRows = 32;      // rows of a workgroup at most
constexpr int kAppendAngles = 1024;  // in LDS at a time
constexpr int kAppendItems = 4;      // pieces of 8 elements a thread loads at a time, of as many rows

struct AppendArgs {
  KvCache c;
  KvBatch b;
  FastDiv page, row_items, head_items, half;  // divisors: block_size, pieces of a row of heads, of a head, angles
  int64_t cap;  // max_blocks * block_size
  const uint16_t* x[2];
  int64_t row_stride[2], head_stride[2];
  RopeArgs rope;
  const int32_t* positions;  // or null: the token's place
  int32_t pieces;            // 8-element pieces of a head
  int32_t rows_wg;           // rows of a workgroup, at most kAppendItems * rows_at_once,
  int32_t rows_at_once;      // and of them side by side
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

__device__ __forceinline__ uint32_t fp4x8(const float (&q)[8]) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, q[0], q[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
}

// The value of the lane whose number differs in bit 0 (1).
__device__ __forceinline__ uint32_t neighbour1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // quad_perm 1 0 3 2
}
__device__ __forceinline__ uint32_t neighbour2(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // quad_perm 2 3 0 1
}

// Codes of 8 values that the 2 (NVFP4) or 4 (MXFP4) threads of a block hold together.
// ts: the tensor scale, r6 = 1 / (6 ts).
//
// The FP32 quotient is off by less than 2^-21 of itself: by the reciprocal of d = scale
// * ts (an ulp, and half a one for d's rounding) and by the product.
// - few_bits: values of at most 11 significant bits, ts of at most 8.  Then a value and
//   a tie's (3 bits times 4 of the scale times ts) are apart by 2^-16 of themselves or
//   equal, and rounding the quotient to 2^-18 puts it on the right side, or on the tie.
//   A tensor scale that is a power of two makes such ties common: one value in 60.
// - Otherwise the quotient is taken once 2^-20 larger and once 2^-20 smaller: where both
//   give the same codes, so does the exact one.  One value in 10^5 of ordinary data lies
//   nearer to a tie; its 8 are done again in FP64, as are scales out of FP32's middle.
template <bool MX>
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], double ts, double r6, bool few_bits, uint32_t* scale_code) {
  uint32_t amax = 0;  // magnitude bits: NaN above infinity above every number
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  amax = max(amax, neighbour1(amax));
  if (MX) amax = max(amax, neighbour2(amax));
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
    return fp4x8(q);
  } else {
    const float top = __uint_as_float(amax), r = quotient_f32((double)top * r6);
    const uint32_t sc = amax ? (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fminf(r, 448.0f), 0.0f, 0, false) & 0xFFu : 0u;
    *scale_code = sc;
    const double d = (double)__builtin_amdgcn_cvt_f32_fp8((int)sc, 0) * ts;
    const float d32 = (float)d, k = __builtin_amdgcn_rcpf(d32);
    uint32_t low = 0, high = 1;
    if (d32 > 0x1p-100f && d32 < 0x1p100f && top * k < 0x1p100f) {
      if (few_bits) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __uint_as_float((__float_as_uint(v[i] * k) + 0x10u) & ~0x1Fu);
        low = high = fp4x8(q);
      } else {
        const float k_low = k * (1.0f - 0x1p-20f), k_high = k * (1.0f + 0x1p-20f);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = v[i] * k_low;
        low = fp4x8(q);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = v[i] * k_high;
        high = fp4x8(q);
      }
    }
    if (low != high) {
      const double kd = sc ? recip_f64(d) : 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = quotient_f32((double)v[i] * kd);
      low = fp4x8(q);
    }
    return low;
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = half_to_f32<BF16>(w[i] & 0xFFFFu);
    v[2 * i + 1] = half_to_f32<BF16>(w[i] >> 16);
  }
}

// Workgroup (b, which): rows b * rows_wg and on of the keys (0) or the values (1).  Its
// first loads start at once; then come the rows' places, by a wavefront that looks for
// the last sequence that starts at or before the row; then the angles; then the codes.
// A thread keeps its piece of a head and goes from row to row: next to the arithmetic on
// 8 elements, divisions and 64-bit products for every piece took a quarter of the time.
template <bool MX, bool BF16>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(AppendArgs a) {
  // A hole behind every 8 angles: lanes read 8 angles apart, and 128-byte steps share their LDS banks.
  __shared__ double2 turn[kAppendAngles / 8 * 9];
  __shared__ int64_t place[kAppendRows];  // first code byte of the row, or -1
  __shared__ int32_t token[kAppendRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x, which = blockIdx.y;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_wg;
  const int nrows = (int)(a.b.rows - r0 < a.rows_wg ? a.b.rows - r0 : a.rows_wg);
  const int rot = which == 0 ? (int)a.rope.rot : 0, half = rot / 2;
  const int per_row = (int)a.c.heads * a.pieces;
  const int64_t row_bytes = a.c.heads * a.c.head_dim / 2, step = a.rows_at_once * a.row_stride[which];
  const uint16_t* x = a.x[which] + r0 * a.row_stride[which];

  // The thread's row of those side by side, head and piece.
  int first_row, slot, h, piece;
  const uint16_t* px;
  bool turned, first;
  uint4 raw[kAppendItems], pair[kAppendItems];  // 8 elements, and the other halves of their pairs
  const auto take = [&](int from) {
    first_row = fastdiv(tid, a.row_items);
    slot = from + tid - first_row * per_row;
    if (a.rows_at_once == 1) first_row = 0, slot = from + tid;
    if (first_row >= a.rows_at_once || slot >= per_row) first_row = nrows;
    h = fastdiv(slot, a.head_items);
    piece = slot - h * a.pieces;
    px = x + first_row * a.row_stride[which] + h * a.head_stride[which] + 8 * piece;
    turned = 8 * piece < rot;
    first = 8 * piece < half;
  };
  const auto load = [&] {
#pragma unroll
    for (int u = 0; u < kAppendItems; ++u) {
      if (first_row + u * a.rows_at_once >= nrows) break;
      raw[u] = *reinterpret_cast<const uint4*>(px);
      if (turned && !a.rope.interleaved) pair[u] = *reinterpret_cast<const uint4*>(first ? px + half : px - half);
      px += step;
    }
  };
  take(0);
  load();
  // The thread's first angle: its frequency is on the way as well.
  int ar = fastdiv(tid, a.half), af = tid - ar * half;
  double freq = tid < nrows * half ? a.rope.freqs[af] : 0.0;
  if (wave == 0) {
    const int64_t r = r0 + lane;
    int64_t s = r, at = -1, t = -1;
    if (a.b.row_start) {
      // The sequence of the first row, then of the first row that is in a later one.
      s = find_sequence(a.b, r0, lane);
      for (;;) {
        const bool later = lane < nrows && s + 1 < a.b.seqs && (int64_t)a.b.row_start[s + 1] <= r;
        const uint64_t m = __ballot(later);
        if (!m) break;
        const int l = __ffsll((unsigned long long)m) - 1;
        const int64_t next = find_sequence(a.b, r0 + l, lane);
        if (lane >= l) s = next;
        if (__ballot(lane == l && later && next + 1 < a.b.seqs && (int64_t)a.b.row_start[next + 1] <= r)) break;
      }
    }
    if (lane < nrows && s < a.b.seqs) {
      const SeqRows q = seq_rows(a.b, a.cap, s);
      t = r + q.shift;
      if (r >= q.first && r < q.first + q.count && t >= 0 && t < q.len) {
        const int32_t page = fastdiv((int32_t)t, a.page);
        const int64_t id = a.b.block_table[s * a.b.max_blocks + page];
        if (id >= 0 && id < a.c.num_blocks)
          at = (id * a.c.block_size + (t - (int64_t)page * a.c.block_size)) * row_bytes;
      }
    }
    if (lane < nrows) {
      place[lane] = at;
      token[lane] = (int32_t)t;
    }
  }
  __syncthreads();
  for (int i = tid; i < nrows * half; i += threads) {
    if (i != tid) ar = fastdiv(i, a.half), af = i - ar * half, freq = a.rope.freqs[af];
    if (place[ar] < 0) continue;
    const int32_t pos = a.positions ? a.positions[r0 + ar] : token[ar];
    double sn, cs;
    sincos_f64((double)pos * freq, &sn, &cs);
    turn[i + i / 8] = make_double2(cs * (double)a.rope.amplitude, sn * (double)a.rope.amplitude);
  }
  __syncthreads();
  const float tscale = MX ? 1.0f : *a.c.tscale[which];
  const bool short_ts = (__float_as_uint(tscale) & 0xFFFFu) == 0;
  const double ts = (double)tscale, r6 = MX ? 1.0 : recip_f64(6.0 * ts);
  for (int from = 0; from < per_row; from += threads) {
    if (from > 0) {
      take(from);
      load();
    }
    uint8_t* codes = a.c.codes[which] + h * (int)(a.c.head_dim / 2) + 4 * piece;
    uint8_t* scales = a.c.scales[which] + slot / (MX ? 4 : 2);
    const bool scale_mine = slot % (MX ? 4 : 2) == 0;
    const int angle = 9 * (a.rope.interleaved ? 0 : first ? piece : piece - half / 8);
    const uint32_t minus = first ? 0x80008000u : 0u;
#pragma unroll
    for (int u = 0; u < kAppendItems; ++u) {
      const int r = first_row + u * a.rows_at_once;
      if (r >= nrows) break;
      const int64_t at = place[r];
      if (at < 0) continue;  // all threads of a block together
      float v[8];
      unpack8<BF16>(raw[u], v);
      if (turned) {
        const double2* cs = turn + r * (half / 8 * 9) + angle;
        if (a.rope.interleaved) {
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const double2 t = cs[4 * piece + piece / 2 + n];
            const double x1 = v[2 * n], x2 = v[2 * n + 1];
            v[2 * n] = (float)fma(-x2, t.y, x1 * t.x);
            v[2 * n + 1] = (float)fma(x1, t.y, x2 * t.x);
          }
        } else {
          float w[8];
          unpack8<BF16>(make_uint4(pair[u].x ^ minus, pair[u].y ^ minus, pair[u].z ^ minus, pair[u].w ^ minus), w);
#pragma unroll
          for (int n = 0; n < 8; ++n) v[n] = (float)fma((double)w[n], cs[n].y, (double)v[n] * cs[n].x);
        }
      }
      uint32_t sc;
      *reinterpret_cast<uint32_t*>(codes + at) = encode8<MX>(v, ts, r6, !turned && short_ts, &sc);
      if (scale_mine) scales[at >> (MX ? 4 : 3)] = (uint8_t)sc;
    }
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
  const int64_t per_row = c.heads * a.pieces, half = rope.rot / 2;
  a.row_items = make_fastdiv(per_row);
  a.head_items = make_fastdiv(a.pieces);
  a.half = make_fastdiv(half > 0 ? half : 1);
  int64_t most = kAppendRows;  // rows whose angles fit
  if (half > 0 && most > kAppendAngles / half) most = kAppendAngles / half;
  int64_t side = per_row < kAppendThreads ? kAppendThreads / per_row : 1;
  side = side < most ? side : most;
  int64_t n = side * kAppendItems;
  n = n < most ? n : most;
  while (n > side && (b.rows + n - 1) / n < 512) n -= side;
  a.rows_at_once = (int32_t)side;
  a.rows_wg = (int32_t)n;
  // As few threads as make the same number of passes over a row.
  const int64_t passes = (per_row + kAppendThreads - 1) / kAppendThreads;
  const int64_t threads = (side * ((per_row + passes - 1) / passes) + 63) / 64 * 64;
  const dim3 grid((unsigned)((b.rows + n - 1) / n), 2);
  if (c.mx) {
    if (bf16) kv_append_kernel<true, true><<<grid, (unsigned)threads, 0, s>>>(a);
    else kv_append_kernel<true, false><<<grid, (unsigned)threads, 0, s>>>(a);
  } else {
    if (bf16) kv_append_kernel<false, true><<<grid, (unsigned)threads, 0, s>>>(a);
    else kv_append_kernel<false, false><<<grid, (unsigned)threads, 0, s>>>(a);
  }
}

}  // namespace nvfp4
