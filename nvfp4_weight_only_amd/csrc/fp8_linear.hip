// E4M3 x E4M3 linear with FP32 scales per 128 elements of K:
//   y[i, j] = BF16( sum_b xs[i, b] ws[j / 128, b] sum_{k in b} x[i, k] w[j, k] ).
//
// The inner sum over a block of 128 is one 16x16x128 matrix instruction per
// 16 x 16 outputs (C = 0); its result is scaled and added in FP32 by the vector
// ALU.  The weights are the A operand (rows n) and the activations the B
// operand (columns m), so the four results of a lane belong to one activation
// row: one factor xs[m, b] ws[n / 128, b] per lane.  Both operands place the
// same element of K at the same position, whatever the order within the block.
#include "device_common.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4_t mfma128(const uint4& a0, const uint4& a1, const uint4& b0, const uint4& b1) {
  const i32x8_t a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
  const i32x8_t b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

struct SkinnyArgs {
  const uint8_t* xq;  // [rows of x, k]
  const float* xs;    // [rows of x, kb]
  const uint8_t* wq;  // [n, k] ([experts, n, k])
  const float* ws;    // [nb, kb] ([experts, nb, kb])
  uint16_t* y;        // [m, n] ([pairs, n])
  int64_t m, n, k;    // m: rows of y
  int kb, nb;
  // Routed form: the sort's int32 arrays, and pairs per token.
  const int32_t* groups;
  int64_t experts, topk;
};

// The rows of y that a workgroup computes and where their activations are.
struct RowSpan {
  int64_t first, count;   // rows first .. first + count of the (sorted) pairs
  const int32_t* perm;    // pair of a sorted row (nullptr: the row itself)
  int64_t topk;
  __device__ __forceinline__ int64_t out_row(int64_t i) const { return perm ? perm[first + i] : first + i; }
  __device__ __forceinline__ int64_t x_row(int64_t i) const { return perm ? perm[first + i] / topk : first + i; }
};

constexpr int kSkWaves = 8;

// 16 rows of W against 16 MT rows of X per workgroup; wavefront w takes blocks
// w, w + 8, ... of K, and the eight partial sums meet in LDS, added in
// wavefront order.
template <int MT>
__device__ __forceinline__ void skinny_tile(const SkinnyArgs& p, const uint8_t* wq, const float* ws, int64_t n0,
                                            const RowSpan& rows, int64_t i0, float (&red)[kSkWaves][MT][256]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t wr = n0 + r < p.n ? n0 + r : p.n - 1;
  const uint8_t* wp = wq + wr * p.k + 16 * g;
  const float* wsp = ws + (n0 >> 7) * p.kb;
  const uint8_t* xp[MT];
  const float* xsp[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t i = i0 + 16 * t + r < rows.count ? i0 + 16 * t + r : rows.count - 1;
    const int64_t xr = rows.x_row(i);
    xp[t] = p.xq + xr * p.k + 16 * g;
    xsp[t] = p.xs + xr * p.kb;
  }
  f32x4_t acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int b = w; b < p.kb; b += kSkWaves) {
    const int64_t k0 = (int64_t)b * 128;
    // Pieces past the end of a row are zero in both operands.
    const bool in0 = k0 + 16 * g < p.k, in1 = k0 + 64 + 16 * g < p.k;
    const uint4 z = make_uint4(0, 0, 0, 0);
    const uint4 a0 = in0 ? *reinterpret_cast<const uint4*>(wp + k0) : z;
    const uint4 a1 = in1 ? *reinterpret_cast<const uint4*>(wp + k0 + 64) : z;
    const float sw = wsp[b];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint4 b0 = in0 ? *reinterpret_cast<const uint4*>(xp[t] + k0) : z;
      const uint4 b1 = in1 ? *reinterpret_cast<const uint4*>(xp[t] + k0 + 64) : z;
      const float s = xsp[t][b] * sw;
      const f32x4_t d = mfma128(a0, a1, b0, b1);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = __builtin_fmaf(d[e], s, acc[t][e]);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) *reinterpret_cast<f32x4_t*>(&red[w][t][4 * lane]) = acc[t];
  __syncthreads();
  if (w < MT) {
    f32x4_t sum = *reinterpret_cast<const f32x4_t*>(&red[0][w][4 * lane]);
#pragma unroll
    for (int i = 1; i < kSkWaves; ++i) {
      const f32x4_t o = *reinterpret_cast<const f32x4_t*>(&red[i][w][4 * lane]);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += o[e];
    }
    // Item e of lane (r, g): weight row 4 g + e, activation row r.
    const int64_t i = i0 + 16 * w + r;
    if (i < rows.count) {
      uint16_t* dst = p.y + rows.out_row(i) * p.n + n0 + 4 * g;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n0 + 4 * g + e < p.n) dst[e] = (uint16_t)f32_to_bf16_rne(sum[e]);
    }
  }
}

template <int MT>
__global__ void __launch_bounds__(64 * kSkWaves) fp8_skinny_kernel(SkinnyArgs p) {
  __shared__ float red[kSkWaves][MT][256];
  const int64_t i0 = (int64_t)blockIdx.y * (16 * MT);
  skinny_tile<MT>(p, p.wq, p.ws, (int64_t)blockIdx.x * 16, RowSpan{0, p.m, nullptr, 1}, i0, red);
}

// Workgroup (x, y): 16 rows of W of the expert that owns tile y of the sort
// (up to 128 pairs); past the last tile, rows of zeros for the pairs whose id
// is out of range.
template <int MT>
__global__ void __launch_bounds__(64 * kSkWaves) fp8_skinny_grouped_kernel(SkinnyArgs p) {
  __shared__ float red[kSkWaves][MT][256];
  const int32_t* pair_off = p.groups + p.experts;
  const int32_t* tile_off = p.groups + 2 * p.experts + 1;
  const int32_t* perm = p.groups + 3 * p.experts + 2;
  const int64_t n0 = (int64_t)blockIdx.x * 16, tile = blockIdx.y, tiles = tile_off[p.experts];
  if (tile >= tiles) {
    const int64_t valid = pair_off[p.experts], spare = gridDim.y - tiles;
    for (int64_t i = valid + tile - tiles; i < p.m; i += spare)
      if (threadIdx.x < 16 && n0 + threadIdx.x < p.n) p.y[perm[i] * p.n + n0 + threadIdx.x] = 0;
    return;
  }
  int64_t lo = 0, hi = p.experts - 1;  // the expert with tile_off[e] <= tile < tile_off[e + 1]
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (tile_off[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  const int64_t first = pair_off[lo] + (tile - tile_off[lo]) * 128, end = pair_off[lo + 1];
  const RowSpan rows{first, end - first < 128 ? end - first : 128, perm, p.topk};
  for (int64_t i0 = 0; i0 < rows.count; i0 += 16 * MT) {
    skinny_tile<MT>(p, p.wq + lo * p.n * p.k, p.ws + lo * p.nb * p.kb, n0, rows, i0, red);
    __syncthreads();
  }
}

}  // namespace

// 16 rows of W per workgroup along x (at most 2^32 threads), 64 rows of X along y.
bool fp8_linear_supported(int64_t m, int64_t n, int64_t k) {
  return n <= ((int64_t)1 << 26) && (m + 63) / 64 <= 65535 && k <= ((int64_t)1 << 37);
}

static bool use_gemm(int64_t m, int64_t n, int64_t k) { return m > 64 && fp8_gemm_supported(m, n, k); }

int64_t fp8_linear_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return use_gemm(m, n, k) ? fp8_gemm_workspace_bytes(m, n, k) : 0;
}

bool fp8_grouped_supported(int64_t t_count, int64_t topk, int64_t experts, int64_t n, int64_t k) {
  return fp8_linear_supported(1, n, k) && topk <= ((int64_t)1 << 30) / t_count &&
         experts <= ((int64_t)1 << 28) && prefill_grouped_tile_bound(t_count * topk, experts) <= 65535;
}

void launch_fp8_linear(const uint8_t* xq, const float* xs, int64_t m, int64_t n, int64_t k, const uint8_t* wq,
                       const float* ws, uint16_t* y, void* workspace, hipStream_t s) {
  const SkinnyArgs a{xq, xs, wq, ws, y, m, n, k, (int)((k + 127) / 128), (int)((n + 127) / 128), nullptr, 1, 1};
  const unsigned gx = (unsigned)((n + 15) / 16);
  if (use_gemm(m, n, k)) return launch_fp8_gemm(xq, xs, m, n, k, wq, ws, y, workspace, s);
  if (m <= 16) fp8_skinny_kernel<1><<<dim3(gx, 1), 64 * kSkWaves, 0, s>>>(a);
  else fp8_skinny_kernel<4><<<dim3(gx, (unsigned)((m + 63) / 64)), 64 * kSkWaves, 0, s>>>(a);
}

void launch_fp8_linear_grouped(const uint8_t* xq, const float* xs, int64_t t_count, int64_t topk, const int32_t* route,
                               int64_t experts, int64_t n, int64_t k, const uint8_t* wq, const float* ws, uint16_t* y,
                               void* workspace, hipStream_t s) {
  const int64_t pairs = t_count * topk;
  int32_t* groups = static_cast<int32_t*>(workspace);
  launch_group_sort(route, pairs, experts, groups, s);
  const SkinnyArgs a{xq, xs, wq, ws, y, pairs, n, k, (int)((k + 127) / 128), (int)((n + 127) / 128), groups, experts,
                     topk};
  const dim3 grid((unsigned)((n + 15) / 16), (unsigned)prefill_grouped_tile_bound(pairs, experts));
  fp8_skinny_grouped_kernel<2><<<grid, 64 * kSkWaves, 0, s>>>(a);
}

}  // namespace nvfp4
