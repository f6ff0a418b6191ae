// E4M3 x E4M3 linear with FP32 scales per 128 elements of K:
//   y[i, j] = BF16( sum_b xs[i, b] ws[j / 128, b] sum_{k in b} x[i, k] w[j, k] ).
//
// The inner sum over a block of 128 is one 16x16x128 matrix instruction per
// 16 x 16 outputs (C = 0); its result is scaled (fp8_mfma.hpp) and added in FP32 by
// the vector ALU.  The weights are the A operand (rows n) and the activations the B
// operand (columns m), so the four results of a lane belong to one activation
// row: one factor per lane.  Both operands place the
// same element of K at the same position, whatever the order within the block.

#include "device_common.hpp"
#include "fp8_mfma.hpp"
#include "fp8_tiles.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

struct SkinnyArgs {
  const uint8_t* xq;  // [rows of x, k]
  const float* xs;    // [rows of x, kb]
  const uint8_t* wq;  // [n, k] ([experts, n, k])
  const float* ws;    // [nb, kb] ([experts, nb, kb])
  uint16_t* y;        // [m, n] ([pairs, n])
  int64_t m, n, k;    // m: rows of y
  int kb, nb;
  int span;           // rows of W per workgroup, a multiple of 4
  // Routed form: expert ids of the m pairs, and pairs per token.
  const int32_t* route;
  int64_t experts, topk;
};

// The rows of y that a workgroup computes and where their activations are.
struct RowSpan {
  int64_t count;
  const int32_t* pairs;  // the rows of y (nullptr: 0, 1, ...)
  uint32_t topk;         // rows of y per row of X
  __device__ __forceinline__ int64_t out_row(int64_t i) const { return pairs ? pairs[i] : i; }
  __device__ __forceinline__ int64_t x_row(int64_t i) const { return pairs ? (uint32_t)pairs[i] / topk : i; }
};

// `span` rows of W (up to 16 NT) against 16 MT rows of X by a workgroup of `waves`
// wavefronts, each of which takes a contiguous share of the whole blocks of K, U
// blocks of both operands at a time with the next U on their way (in registers:
// nothing of W is used twice, and X by one wavefront only); the last wavefront
// adds the last, short block.  Their sums meet in LDS and are added in wavefront
// order.  SXL: the rows' scales are first copied to LDS.
constexpr int sums_at_a_time(int t) { return t <= 10 ? t : (t + 1) / 2; }

template <int MT, int NT, int U, bool SXL>
__device__ __forceinline__ void skinny_tile(const SkinnyArgs& p, const uint8_t* wq, const float* ws, int64_t n0,
                                            const RowSpan& rows, int64_t i0, int waves, f32x4_t* red, float* sxl) {
  constexpr int T = MT * NT;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n1 = n0 + p.span < p.n ? n0 + p.span : p.n;  // past the last row of W
  const uint8_t* wp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t wr = n0 + 16 * t + r < n1 ? n0 + 16 * t + r : n1 - 1;
    wp[t] = wq + wr * p.k + 16 * g;
  }
  // The rows of W lie in one block of 128 or two; four neighbouring ones, as a
  // lane has them of each 16, in one (spans are multiples of 4).
  const float* wsp = ws + (n0 >> 7) * p.kb;
  const float* wsp2 = ws + ((n1 - 1) >> 7) * p.kb;
  const int rest = 128 - (int)(n0 & 127);
  const uint8_t* xp[MT];
  const float* xsp[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t i = i0 + 16 * t + r < rows.count ? i0 + 16 * t + r : rows.count - 1;
    const int64_t xr = rows.x_row(i);
    xp[t] = p.xq + xr * p.k + 16 * g;
    xsp[t] = p.xs + xr * p.kb;
  }
  const int ld = p.kb | 1;  // an odd number of words from row to row
  const auto sx = [&](int t, int b) -> float { return SXL ? sxl[(16 * t + r) * ld + b] : xsp[t][b]; };
  // The scales of block b: ea and fa by this lane's row of W as an operand (r) and as
  // an output (4 g), eb and fb of the row of X; of zeros for a block that is not `in`.
  struct Factors {
    int ea[NT], eb[MT];
    float fa[NT], fb[MT];
  };
  const auto factors = [&](int b, bool in) {
    Factors v;
    const float sw = wsp[b], sw2 = wsp2[b];
    const int e = scale_exp(sw), e2 = scale_exp(sw2);
    const float f = scale_rest(sw, e), f2 = scale_rest(sw2, e2);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      v.ea[t] = 16 * t + r < rest ? e : e2;
      v.fa[t] = in ? (16 * t + 4 * g < rest ? f : f2) : 0.0f;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float s = in ? sx(t, b) : 0.0f;
      v.eb[t] = scale_exp(s);
      v.fb[t] = scale_rest(s, v.eb[t]);
    }
    return v;
  };
  const auto load = [](const uint8_t* q) { return *reinterpret_cast<const uint4*>(q); };
  f32x4_t acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int full = (int)(p.k >> 7);  // whole blocks
  const int b0 = (int)((int64_t)full * w / waves), b1 = (int)((int64_t)full * (w + 1) / waves);

  struct Blocks {
    uint4 w[U][NT][2], x[U][MT][2];
  };
  // Past the share's end: the last block again (with factor zero).
  const auto fetch = [&](int b, Blocks& v) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t o = 128 * (int64_t)(b + u < b1 ? b + u : b1 - 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) v.w[u][t][0] = load(wp[t] + o), v.w[u][t][1] = load(wp[t] + o + 64);
#pragma unroll
      for (int t = 0; t < MT; ++t) v.x[u][t][0] = load(xp[t] + o), v.x[u][t][1] = load(xp[t] + o + 64);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto step = [&](int b, const Blocks& v) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = u == 0 || b + u < b1;
      const Factors s = factors(in ? b + u : b1 - 1, in);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int i = t / MT, j = t % MT;
        const float ft = s.fb[j] * s.fa[i];
        const f32x4_t d = mfma128(mfma_frag(v.w[u][i][0], v.w[u][i][1]), mfma_frag(v.x[u][j][0], v.x[u][j][1]), s.ea[i],
                                  s.eb[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = __builtin_fmaf(d[e], ft, acc[t][e]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  Blocks va, vb;
  if (b0 < b1) fetch(b0, va);
  if constexpr (SXL) {
    for (int i = threadIdx.x; i < 16 * MT * p.kb; i += blockDim.x) {
      const int rr = i / p.kb, c = i - rr * p.kb;
      const int64_t xi = i0 + rr < rows.count ? i0 + rr : rows.count - 1;
      sxl[rr * ld + c] = p.xs[rows.x_row(xi) * p.kb + c];
    }
    __syncthreads();
  }
  if (b0 < b1) {
    int b = b0;
    for (; b + 2 * U < b1; b += 2 * U) {
      fetch(b + U, vb);
      step(b, va);
      fetch(b + 2 * U, va);
      step(b + U, vb);
    }
    if (b + U < b1) {
      fetch(b + U, vb);
      step(b, va);
      step(b + U, vb);
    } else {
      step(b, va);
    }
  }
  if (full < p.kb && w == waves - 1) {
    // Pieces past the end of a row: the row's last piece of W, zeros of X.
    const int64_t k0 = 128 * (int64_t)full, end = p.k - 16 - 16 * g;
    const bool in0 = k0 <= end, in1 = k0 + 64 <= end;
    const int64_t o0 = in0 ? k0 : end, o1 = in1 ? k0 + 64 : end;
    const Factors s = factors(full, true);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int i = t / MT, j = t % MT;
      const uint8_t *wt = wp[i], *xt = xp[j];
      const uint4 z = make_uint4(0, 0, 0, 0), x0 = load(xt + o0), x1 = load(xt + o1);
      const f32x4_t d = mfma128(mfma_frag(load(wt + o0), load(wt + o1)), mfma_frag(in0 ? x0 : z, in1 ? x1 : z), s.ea[i],
                                s.eb[j]);
      const float f = s.fb[j] * s.fa[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = __builtin_fmaf(d[e], f, acc[t][e]);
    }
  }
  // The sums of GT blocks at a time (what LDS holds of all wavefronts).
  constexpr int GT = sums_at_a_time(T);
#pragma unroll
  for (int t0 = 0; t0 < T; t0 += GT) {
    if (t0 > 0) __syncthreads();
#pragma unroll
    for (int t = 0; t < GT; ++t)
      if (t0 + t < T) red[(w * GT + t) * 64 + lane] = acc[t0 + t < T ? t0 + t : 0];
    __syncthreads();
    for (int tt = w; tt < GT && t0 + tt < T; tt += waves) {
      const int t = t0 + tt;
      f32x4_t sum = red[tt * 64 + lane];
      for (int i = 1; i < waves; ++i) {
        const f32x4_t o = red[(i * GT + tt) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += o[e];
      }
      // Item e of lane (r, g): weight row 4 g + e, activation row r.
      const int64_t i = i0 + 16 * (t % MT) + r, col = n0 + 16 * (t / MT) + 4 * g;
      if (i >= rows.count || col >= n1) continue;
      uint16_t* dst = p.y + rows.out_row(i) * p.n + col;
      if ((p.n & 3) == 0) {
        const bf16x2_t lo = {(__bf16)sum[0], (__bf16)sum[1]}, hi = {(__bf16)sum[2], (__bf16)sum[3]};
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < n1) dst[e] = (uint16_t)f32_to_bf16_rne(sum[e]);
      }
    }
  }
}

template <int MT, int NT, int U, int MAXW, bool SXL>
__global__ void __launch_bounds__(64 * MAXW) fp8_skinny_kernel(SkinnyArgs p) {
  __shared__ f32x4_t red[MAXW * sums_at_a_time(MT * NT) * 64];
  extern __shared__ float sxl[];
  const int64_t i0 = (int64_t)blockIdx.y * (16 * MT);
  skinny_tile<MT, NT, U, SXL>(p, p.wq, p.ws, (int64_t)blockIdx.x * p.span, RowSpan{p.m, nullptr, 1}, i0,
                         blockDim.x >> 6, red, sxl);
}

// Few pairs over an expert stack, without a sort: workgroup (x, p) multiplies
// span rows of W of pair p's expert with the activations of every pair that chose
// that expert, if p is the first of them (the others' workgroups end); a pair
// whose id is out of range gets zeros.  The order in which the pairs are found
// varies; every output depends on its own rows only.  HBM bounds it: 8 tokens, top
// 8 of 128, 2048 x 4096: 410 MB in 70 us, 5.9 TB/s (81 us with two blocks of K at a
// time and the registers for two workgroups per CU instead of four).
constexpr int kMaxPairs = 512;

template <int MT, int NT, int U, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) fp8_routed_kernel(SkinnyArgs p) {
  __shared__ f32x4_t red[WAVES * sums_at_a_time(MT * NT) * 64];
  __shared__ int32_t same[kMaxPairs];
  __shared__ int32_t count, earlier;
  const int pair = blockIdx.y, pairs = (int)p.m;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
  const int32_t id = p.route[pair];
  if (id < 0 || id >= p.experts) {
    for (int c = threadIdx.x; c < 16 * NT && n0 + c < p.n; c += blockDim.x) p.y[pair * p.n + n0 + c] = 0;
    return;
  }
  if (threadIdx.x == 0) count = 0, earlier = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    if (p.route[i] != id) continue;
    if (i < pair) earlier = 1;
    else same[atomicAdd(&count, 1)] = i;
  }
  __syncthreads();
  if (earlier) return;
  const RowSpan rows{count, same, (uint32_t)p.topk};
  for (int64_t i0 = 0; i0 < rows.count; i0 += 16 * MT) {
    if (i0 > 0) __syncthreads();  // red is free again
    skinny_tile<MT, NT, U, false>(p, p.wq + id * p.n * p.k, p.ws + (int64_t)id * p.nb * p.kb, n0, rows, i0, WAVES, red,
                                  nullptr);
  }
}

}  // namespace

namespace {

using fp8_tiles::kCus;
constexpr int kMaxSpan = 80;
constexpr size_t kScalesLds = 65536;

// Few rows of X: each CU streams its share of W through registers and reads all of X,
// and the sum of both bounds it.  A CU takes 43 ns per KB from HBM (6.1 TB/s over
// the chip; a CU by itself is no faster, so shares have to be even) and 31 ns per
// KB of X from L2, the lines in flight being what is scarce; a launch takes 1 us and
// a workgroup's start and sums 3.  17408 x 5120 with M = 1, 16, 32, 48: 19.6, 21.1,
// 24.4 and 28.2 us.
struct Skinny {
  int mt = 1;        // 16 mt rows of X per workgroup
  int64_t span = 0;  // rows of W per workgroup; 0: scales too long for LDS
  int64_t rounds = 1;
  double ns = 0;  // estimated
};

// The rows of W in even shares, multiples of 4, of one workgroup per CU, or of as
// many rounds of them as spans of at most 80 need; 64 rows of X at most per
// workgroup, or fewer where W is small and X is what a CU reads (64 x 430 x 12032:
// 30.0 us with 64, 12.8 with 16; 1024 x 2048, M = 64: 7.7 and 4.6).
Skinny skinny_plan(int64_t m, int64_t n, int64_t k) {
  Skinny best;
  best.ns = 1e300;
  const int64_t kb = (k + 127) / 128, fit = (int64_t)(kScalesLds / 64) / (kb | 1);
  const int64_t most = (m + 15) / 16 < 4 ? (m + 15) / 16 : 4;
  for (int64_t mt = most < fit ? most : fit; mt >= 1; --mt) {
    const int64_t gy = (m + 16 * mt - 1) / (16 * mt), cols = kCus / gy > 0 ? kCus / gy : 1;
    const int64_t rounds = (n + cols * kMaxSpan - 1) / (cols * kMaxSpan);
    const int64_t span = ((n + cols * rounds - 1) / (cols * rounds) + 3) / 4 * 4;
    const double wgs = (double)((n + span - 1) / span) * (double)gy, turns = wgs > kCus ? wgs / kCus : 1.0;
    const double ns =
        1000.0 + turns * (3000.0 + (43.0 * (double)span + 31.0 * 16 * (double)mt) * (double)k / 1024);
    if (ns < best.ns) best = Skinny{(int)mt, span, rounds, ns};
  }
  return best;
}

// At least 4 rows of W per workgroup along x, at least 16 of X along y.
bool skinny_supported(int64_t m, int64_t n, int64_t k) {
  return n <= ((int64_t)1 << 26) && m <= 16 * 65535 && k <= ((int64_t)1 << 37);
}

}  // namespace

// Measured, skinny against GEMM, us: M = 48 17408 x 5120 28.4 / 38.8, 5120 x 17408
// 43.5 / 26.6; M = 96 5120 x 5120 21.8 / 18.1, 1024 x 2048 8.1 / 10.5; M = 200
// 17408 x 128 13.3 / 6.4, 512 x 1024 5.4 / 6.5.  Up to 16 rows the estimate is not
// asked: M = 16 17408 x 5120 21.3 / 26.5, 5120 x 5120 10.7 / 12.9, 34816 x 5120 36.5 /
// 47.6, 2048 x 8192 10.1 / 12.5, 1024 x 16384 15.3 / 15.8; but 5120 x 17408 26.9 / 23.6
// (M = 8 22.9 / 23.0).
// `split`: whether there is a workspace to split K with.
static bool use_gemm(int64_t m, int64_t n, int64_t k, bool split) {
  if (!skinny_supported(m, n, k)) return true;
  return m > 16 && fp8_gemm_supported(m, n, k) && fp8_gemm_ns(m, n, k, split) < skinny_plan(m, n, k).ns;
}

bool fp8_linear_supported(int64_t m, int64_t n, int64_t k) {
  return skinny_supported(m, n, k) || fp8_gemm_supported(m, n, k);
}

int64_t fp8_linear_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return use_gemm(m, n, k, true) ? fp8_gemm_workspace_bytes(m, n, k) : 0;
}

// Few pairs without a sort, by estimate: 32 rows of W per workgroup, passed over
// once per 16 pairs of the expert, and the workgroups that end at once; against
// sort and GEMM, whose tiles of 256 rows of W slow each other down as they fill the
// chip (fp8_gemm_grouped_ns).  us, this / those: 64 pairs, 8 of 184 x 448, 3.6 /
// 12.3; 64, 8 of 4096 x 4096, 37 / 44; 128 of the same, 50 / 44; 512, 16 of 512 x
// 2048, 23.6 / 20.4; 512, 128 of 2048 x 4096, 201 / 198.
static bool use_routed(int64_t t_count, int64_t topk, int64_t experts, int64_t n, int64_t k) {
  const int64_t pairs = t_count * topk;
  if (pairs > kMaxPairs || n > ((int64_t)1 << 26) || k > ((int64_t)1 << 37)) return false;
  if (!fp8_gemm_grouped_supported(t_count, topk, experts, n, k)) return true;
  const double chosen = fp8_experts_chosen(pairs, experts), per = (double)pairs / chosen;
  const double tiles = (double)((n + 31) / 32), passes = per <= 8.0 ? 1.0 : per / 16.0 + 0.5;
  const double turns = chosen * tiles / kCus > 1.0 ? chosen * tiles / kCus : 1.0;
  const double loads = (43.0 * 32 + 31.0 * (per < 16.0 ? per : 16.0)) * (double)k / 1024;
  const double ns = 3500.0 + 700.0 * passes + turns * (500.0 + passes * loads) +
                    100.0 * ((double)pairs - chosen) * tiles / kCus;
  return ns < fp8_gemm_grouped_ns(pairs, experts, n, k);
}

bool fp8_grouped_supported(int64_t t_count, int64_t topk, int64_t experts, int64_t n, int64_t k) {
  if (topk > ((int64_t)1 << 30) / t_count || experts > ((int64_t)1 << 28)) return false;
  return use_routed(t_count, topk, experts, n, k) || fp8_gemm_grouped_supported(t_count, topk, experts, n, k);
}

// As few wavefronts as keep the number of passes over U blocks that MAXW allow.
template <int MT, int NT, int U, int MAXW, bool SXL = true>
static void launch_skinny_shape(const SkinnyArgs& a, hipStream_t s) {
  const int passes = (a.kb + MAXW * U - 1) / (MAXW * U), waves = (a.kb + passes * U - 1) / (passes * U);
  const dim3 grid((unsigned)((a.n + a.span - 1) / a.span), (unsigned)((a.m + 16 * MT - 1) / (16 * MT)));
  const size_t lds = SXL ? sizeof(float) * 16 * MT * (a.kb | 1) : 0;
  fp8_skinny_kernel<MT, NT, U, MAXW, SXL><<<grid, 64 * waves, lds, s>>>(a);
}

// Blocks of W in flight: about 8 to 10 KB per wavefront and buffer.  Eight
// wavefronts, or four where two workgroups are to share a CU (34816 x 5120, M = 1
// / 32: 34.8 / 44.1 us against 37.2 / 46.6) or eight would not leave the registers
// (MT = 4, NT = 5).
template <int MT>
static void launch_skinny(const SkinnyArgs& a, int64_t rounds, hipStream_t s) {
  if (a.span <= 16) return launch_skinny_shape<MT, 1, MT == 1 ? 4 : MT == 2 ? 3 : 2, 8>(a, s);
  if (a.span <= 32) return launch_skinny_shape<MT, 2, MT <= 2 ? 2 : 1, 8>(a, s);
  if (a.span <= 48) return launch_skinny_shape<MT, 3, 1, 8>(a, s);
  if constexpr (MT < 4)
    if (rounds == 1) return launch_skinny_shape<MT, 5, 1, 8>(a, s);
  launch_skinny_shape<MT, 5, 1, 4>(a, s);
}

void launch_fp8_linear(const uint8_t* xq, const float* xs, int64_t m, int64_t n, int64_t k, const uint8_t* wq,
                       const float* ws, uint16_t* y, void* workspace, hipStream_t s) {
  if (use_gemm(m, n, k, workspace != nullptr)) return launch_fp8_gemm(xq, xs, m, n, k, wq, ws, y, workspace, s);
  const Skinny p = skinny_plan(m, n, k);
  SkinnyArgs a{xq, xs, wq, ws, y, m, n, k, (int)((k + 127) / 128), (int)((n + 127) / 128), (int)p.span, nullptr, 1, 1};
  if (p.span == 0) {
    a.span = 32;
    return launch_skinny_shape<1, 2, 2, 4, false>(a, s);
  }
  switch (p.mt) {
    case 1: return launch_skinny<1>(a, p.rounds, s);
    case 2: return launch_skinny<2>(a, p.rounds, s);
    case 3: return launch_skinny<3>(a, p.rounds, s);
    default: return launch_skinny<4>(a, p.rounds, s);
  }
}

void launch_fp8_linear_grouped(const uint8_t* xq, const float* xs, int64_t t_count, int64_t topk, const int32_t* route,
                               int64_t experts, int64_t n, int64_t k, const uint8_t* wq, const float* ws, uint16_t* y,
                               void* workspace, hipStream_t s) {
  const int64_t pairs = t_count * topk;
  if (use_routed(t_count, topk, experts, n, k)) {
    const SkinnyArgs a{xq, xs, wq, ws, y, pairs, n, k, (int)((k + 127) / 128), (int)((n + 127) / 128), 32, route, experts,
                       topk};
    const dim3 grid((unsigned)((n + 31) / 32), (unsigned)pairs);
    fp8_routed_kernel<1, 2, 1, 4><<<grid, 256, 0, s>>>(a);
    return;
  }
  int32_t* groups = static_cast<int32_t*>(workspace);
  launch_group_sort(route, pairs, experts, groups, s);
  launch_fp8_gemm_grouped(xq, xs, topk, groups, pairs, experts, n, k, wq, ws, y, s);
}

}  // namespace nvfp4
