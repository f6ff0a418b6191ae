// E4M3 x E4M3 GEMM with FP32 scales per 128 elements of K, for many rows of X
// (the arithmetic is fp8_linear.hip's).
//
// A workgroup of eight wavefronts owns a TN x TM tile of outputs (TN rows of W,
// TM rows of X).  K advances in chunks of 128, one scale block each: both
// operands' chunk goes to LDS by direct loads (16 bytes per lane, whole
// 128-byte lines per row) into a ring of ST stages, so that up to ST - 1 chunks
// are in flight behind the one in use.  A 16 x 16 block of outputs takes one
// 16x16x128 matrix instruction per chunk (C = 0) and four fused multiply-adds per
// lane that scale the block's sum into the FP32 accumulators; those of one block
// are issued two blocks later, while the matrix instructions run on.
//
// What bounds it: 2048 x 17408 x 5120 takes 184 us, 2.0 PFLOP/s (an earlier build 190,
// 177 if every load found its line in L2; the matrix instructions and multiply-adds by
// themselves 115 us, the LDS reads, 192 KB per chunk of 64 KB, 90 us); 4096^3 65 us,
// 2.1 PFLOP/s.  With few rows of X the loads: 333 x 5000 x 17392 66 us, 58 if they
// found their lines in L2; 64 x 5120 x 17408 29 us, 3.1 TB/s of W.
//
// LDS image of a chunk: row r (128 bytes) at 128 r, its 16-byte piece p at
// piece p ^ (r & 7): a 128-bit read of one logical piece by 8 consecutive rows
// covers all banks.
#include <type_traits>

#include "device_common.hpp"
#include "fp8_mfma.hpp"
#include "fp8_tiles.hpp"
#include "launch.hpp"
#include "lds_dma.hpp"

namespace nvfp4 {
namespace {

using namespace fp8_tiles;

struct GemmArgs {
  const uint8_t* xq;
  const float* xs;
  const uint8_t* wq;
  const float* ws;
  uint16_t* y;
  int64_t m, n, k;  // m: rows of y
  int64_t ld;       // values from one row of y to the next
  int kb, nb;
  int n_tiles, m_tiles;
  // Split: slices of K, and their FP32 sums [slices, m, np] (slices = 1: none), np
  // being n rounded up to a multiple of 4.
  int slices;
  int64_t np;
  float* part;
  // Grouped form: the sort's int32 arrays, pairs per token.
  const int32_t* groups;
  int64_t experts, topk;
};

// At most N of this wavefront's loads still in flight, and its LDS reads done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N <= 63, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
}

__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
  const bf16x2_t r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

template <int TN, int TM>
struct Stage {
  uint4 w[TN * 8];
  uint4 x[TM * 8];
  float sx[TM];  // the chunk's scale of each row of X
  float sw[64];  // ... of the tile's blocks of 128 rows of W (the first 3 at most are used)
};

template <int TN, int TM, int WN, int WM, int ST, bool GROUPED>
__global__ void __launch_bounds__(512, 2) fp8_gemm_kernel(GemmArgs p) {
  static_assert(WN * WM == 8 && TN % (32 * WN) == 0 && TM % (16 * WM) == 0 && TN % 64 == 0 && TM % 64 == 0, "tile");
  constexpr int NT = TN / WN / 16, MT = TM / WM / 16, T = NT * MT;  // 16 x 16 blocks of a wavefront
  static_assert(T % 4 == 0 && NT % 2 == 0 && MT >= 2 && 128 % (TN / WN) == 0, "register rings; one scale of W");
  constexpr int LW = TN / 64, LX = TM / 64, L2 = ST == 2, NL = LW + LX + 1 + L2;  // loads per wavefront and chunk
  constexpr int QJ = NL <= T ? 1 : 2;  // loads behind each matrix instruction
  static_assert(NL <= QJ * T, "a chunk's loads are issued before the next barrier");
  __shared__ Stage<TN, TM> stage[ST];
  __shared__ uint32_t sink[L2 ? 64 : 1];
  static_assert(sizeof(stage) >= sizeof(uint16_t) * TN * TM, "the epilogue's tile fits the stages");
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = w % WN, wm = w / WN;

  int id = (int)blockIdx.x, slice = 0, nt, mt;
  if constexpr (GROUPED) {
    nt = (id >> 3) % p.n_tiles, mt = (id >> 3) / p.n_tiles;
  } else {
    const int tiles = p.n_tiles * p.m_tiles;
    slice = id / tiles;
    id -= slice * tiles;
    id = tile_of_id(id, tiles);
    nt = id / p.m_tiles, mt = id % p.m_tiles;
  }
  const int64_t n0 = (int64_t)nt * TN;
  const uint8_t* wq = p.wq;
  const float* ws = p.ws;
  int64_t m0 = (int64_t)mt * TM, rows = p.m - m0 < TM ? p.m - m0 : TM;
  const int32_t* perm = nullptr;
  if constexpr (GROUPED) {
    const int32_t* pair_off = p.groups + p.experts;
    const int32_t* tile_off = p.groups + 2 * p.experts + 1;
    perm = p.groups + 3 * p.experts + 2;
    // Each XCD takes an eighth of the tiles in use, all of their n tiles, so that
    // the rows of X too are fetched into its L2 once (2048 x 4096, 256 tokens, top 8
    // of 128: 213 us so, 277 by n tile).  The workgroups left over
    // write zero rows for the pairs whose id is out of range.
    const int64_t used = tile_off[p.experts], xcd = id & 7, t0 = first_of_xcd(used, xcd), tn = first_of_xcd(used, xcd + 1) - t0;
    if (mt >= tn) {
      const int64_t cols = p.n - n0 < TN ? p.n - n0 : TN, left = left_places(used, p.m_tiles);
      for (int64_t i = pair_off[p.experts] + left_rank(xcd, p.m_tiles, t0, tn, mt); i < p.m; i += left)
        for (int64_t c = tid; c < cols; c += 512) p.y[perm[i] * p.ld + n0 + c] = 0;
      return;
    }
    mt += (int)t0;
    // The last expert with tile_off[e] <= mt: 64 candidates at a time.
    int64_t lo = 0, len = p.experts;
    while (len > 1) {
      const int64_t step = (len + 63) >> 6, e = lo + step * lane;
      const uint64_t in = __ballot(step * lane < len && tile_off[step * lane < len ? e : lo] <= mt);
      const int64_t at = step * (63 - __builtin_clzll(in | 1));
      lo += at, len = len - at < step ? len - at : step;
    }
    m0 = pair_off[lo] + (int64_t)(mt - tile_off[lo]) * TM;
    rows = pair_off[lo + 1] - m0 < TM ? pair_off[lo + 1] - m0 : TM;
    wq += lo * p.n * p.k;
    ws += lo * p.nb * p.kb;
  }

  const int piece = lane_piece(lane);
  const auto x_row = [&](int r) -> int64_t {  // the row of X behind row r of the tile
    const int64_t rm = row_or_last(r, rows);
    return GROUPED ? (int64_t)((uint32_t)perm[m0 + rm] / (uint32_t)p.topk) : rm;
  };
  const uint8_t* wbase = uniform_ptr(wq + n0 * p.k);
  const uint8_t* xbase = uniform_ptr(GROUPED ? p.xq : p.xq + m0 * p.k);
  uint32_t offw[LW], offx[LX];
#pragma unroll
  for (int j = 0; j < LW; ++j) {
    offw[j] = piece_offset(row_or_last(load_row(w, j, lane), p.n - n0), p.k, piece);
  }
#pragma unroll
  for (int j = 0; j < LX; ++j) offx[j] = piece_offset(x_row(load_row(w, j, lane)), p.k, piece);
  // Scales: wavefront w < LX the rows 64 w .. + 63 of X, the others the blocks of W.
  const float* sbase;
  uint32_t soff;
  if (w < LX) {
    sbase = GROUPED ? p.xs : p.xs + m0 * p.kb;
    soff = scale_offset(x_row(64 * w + lane), p.kb);
  } else {
    const int64_t b0 = n0 / 128;
    sbase = ws + b0 * p.kb;
    soff = scale_offset(row_or_last(lane, p.nb - b0), p.kb);
  }
  sbase = uniform_ptr(sbase);

  // Lines brought into L2 ahead of their chunk's loads (one 4-byte read each, to
  // a part of LDS that nothing reads).
  static_assert(!L2 || (!GROUPED && TN + TM <= 512), "one line per lane");
  const uint8_t* pf = nullptr;
  if constexpr (L2) {
    const Line l = line_ahead(TN, TM, p.n_tiles, p.m_tiles, nt, mt, w, lane);
    pf = l.of_w ? wbase + row_or_last(l.row, p.n - n0) * p.k : xbase + x_row(l.row) * p.k;
  }
  // Chunks of this slice.
  const int c0 = first_chunk(p.kb, slice, p.slices), c1 = first_chunk(p.kb, slice + 1, p.slices);
  const int last = c1 - 1;
  // A last, short chunk: pieces past the end of K are read from the row's last
  // one, and X's are set to zero in LDS when they have landed (finish).  W's keep
  // the copy: times zero, or NaN where that row's sum is NaN by its own piece.
  const int ktail = tail_of(p.k);
  const bool past = past_end(ktail, piece);
  const uint32_t back = step_back(ktail, piece);

  // Load q (of NL) of chunk cc into stage s.
  const auto issue = [&](int q, int cc, int s) {
    Stage<TN, TM>& sg = stage[s];
    const int64_t k0 = (int64_t)cc * kChunk;
    const uint32_t bk = cc == p.kb - 1 ? back : 0u;
    if (q < LW) lds_dma16(wbase + k0, offw[q < LW ? q : 0] - bk, lds_addr(&sg.w[0]) + load_dst(w, q));
    else if (q < LW + LX)
      lds_dma16(xbase + k0, offx[q >= LW && q < LW + LX ? q - LW : 0] - bk,
            lds_addr(&sg.x[0]) + load_dst(w, q - LW));
    else if (q == LW + LX)
      lds_dma4(sbase + cc, soff, w < LX ? lds_addr(&sg.sx[64 * (w < LX ? w : 0)]) : lds_addr(&sg.sw[0]));
    else
      lds_dma4(pf + (int64_t)chunk_ahead(cc, last) * kChunk, lds_addr(&sink[0]));
  };
  // This wavefront's loads of chunk c, in stage s, have landed.
  const auto finish = [&](int c, int s) {
    if (ktail == 0 || c != p.kb - 1) return;
    if (past) {
#pragma unroll
      for (int j = 0; j < LX; ++j) stage[s].x[64 * (w + 8 * j) + lane] = make_uint4(0, 0, 0, 0);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  };

  f32x4_t acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // Byte offsets in a stage of this lane's first row of each operand.
  const uint32_t lane_off = read_offset(l16, g);
  const uint32_t rx = lane_off + (uint32_t)(sizeof(uint4) * TN * 8) + 128 * 16 * wm * MT;
  const uint32_t rw = lane_off + 128 * 16 * wn * NT;
  const char* const lds0 = reinterpret_cast<const char*>(&stage[0]);
  const auto read = [&](uint32_t off, int rows16) {
    return mfma_frag(*reinterpret_cast<const uint4*>(lds0 + off + 2048 * rows16),
                     *reinterpret_cast<const uint4*>(lds0 + (off ^ 16) + 2048 * rows16));
  };
  const auto meet = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };

  // The matrix instructions of a wavefront run on without a break from chunk to
  // chunk: fragments of W are read one row of blocks ahead (two registers sets),
  // and behind the last use of each fragment of X the next chunk's is read over
  // it.  The one barrier of a chunk stands before its last row of blocks, where
  // everything of this chunk's stage has been read and the next chunk has
  // landed: after it the next chunk's fragments are read, and the chunk that
  // takes this stage is loaded, one load behind each matrix instruction.
  constexpr int PART = QJ * MT < NL ? QJ * MT : NL;  // of a chunk's loads, those behind the last row of blocks
#pragma unroll
  for (int s = 0; s < ST; ++s)
    if (c0 + s <= last)
#pragma unroll
      for (int q = 0; q < (s < ST - 1 ? NL : PART); ++q) issue(q, c0 + s, s);
  if (c0 + ST - 1 <= last) wait_loads<(ST - 2) * NL + PART>();
  else wait_loads<0>();
  finish(c0, 0);
  meet();
  i32x8_t a[2], b[MT];
  float sx[MT], sw;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    b[j] = read(rx, j);
    sx[j] = stage[0].sx[16 * wm * MT + l16 + 16 * j];
  }
  a[0] = read(rw, 0);
  sw = stage[0].sw[((int)(n0 & 127) + 16 * wn * NT) >> 7];
  // No scalar load is under way in the loop, where each wait for one would be a wait
  // for all reads of LDS (2048 x 17408 x 5120: 194.5 us without, 192.5 with).
  __builtin_amdgcn_s_waitcnt(0xC07F);
  // Sums of the last blocks: block t is scaled behind the matrix instruction of
  // block t + 2, so that the multiply-adds never wait for it.
  f32x4_t d[4];
  float f[MT], f_old[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < MT; ++j) f[j] = 0.0f;
  int sidx = 0;
  uint64_t far = 0;  // lanes that met two scales for which is_far
  // REST, NEXT: the rest of chunk c - 1 + ST, and the first loads of chunk c + ST, are there to be issued.
  const auto step = [&](int c, auto rest, auto next) {
    constexpr bool REST = decltype(rest)::value, NEXT = decltype(next)::value;
    const int here = sidx;
    sidx = sidx + 1 == ST ? 0 : sidx + 1;
    const uint32_t so = (uint32_t)(here * sizeof(Stage<TN, TM>)), sn = (uint32_t)(sidx * sizeof(Stage<TN, TM>));
    f_old[0] = f[MT - 2], f_old[1] = f[MT - 1];
#pragma unroll
    for (int j = 0; j < MT; ++j) f[j] = sx[j] * sw;
    const float fw = sw;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (i < NT - 1) {
        a[(i + 1) & 1] = read(so + rw, i + 1);
      } else {
        wait_loads<REST ? (ST - 2) * NL + L2 : 0>();
        finish(c + 1, sidx);
        meet();
        a[0] = read(sn + rw, 0);
        sw = stage[sidx].sw[((int)(n0 & 127) + 16 * wn * NT) >> 7];
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        // In this order: the compiler would gather the matrix instructions and
        // sink the multiply-adds.
        const int t = i * MT + j, u = (t + T - 2) % T;
        d[t & 3] = mfma128(a[i & 1], b[j]);
        __builtin_amdgcn_sched_barrier(0);
        if (i == 1 && j == 0) {  // here nothing waits for it
          bool normal = true;
#pragma unroll
          for (int q = 0; q < MT; ++q) normal &= is_normal(f[q]);
          if (__builtin_amdgcn_ballot_w64(!normal) != 0) {
#pragma unroll
            for (int q = 0; q < MT; ++q) far |= __builtin_amdgcn_ballot_w64(is_far(sx[q], fw));
          }
        }
        if (i == NT - 1) {
          b[j] = read(sn + rx, j);
          sx[j] = stage[sidx].sx[16 * wm * MT + l16 + 16 * j];
#pragma unroll
          for (int q = QJ * j; NEXT && q < QJ * (j + 1) && q < NL; ++q) issue(q, c + ST, here);
        } else {
#pragma unroll
          for (int q = QJ * (t + MT); REST && q < QJ * (t + MT + 1) && q < NL; ++q)
            issue(q, c - 1 + ST, here == 0 ? ST - 1 : here - 1);
        }
        const float fu = t < 2 ? f_old[t] : f[u % MT];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[u][e] = __builtin_fmaf(d[u & 3][e], fu, acc[u][e]);
        asm volatile("" : "+v"(acc[u]));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // GROUPED: a wavefront whose rows of X are all past the tile's (its partner on the
  // SIMD has the matrix cores for itself) loads and waits with the others (2048
  // tokens, top 8 of 128: 301 us without, 289 with; 256 tokens: 210, 203).
  const auto idle = [&](int c, auto rest, auto next) {
    constexpr bool REST = decltype(rest)::value, NEXT = decltype(next)::value;
    const int here = sidx;
    sidx = sidx + 1 == ST ? 0 : sidx + 1;
#pragma unroll
    for (int q = PART; REST && q < NL; ++q) issue(q, c - 1 + ST, here == 0 ? ST - 1 : here - 1);
    wait_loads<REST ? (ST - 2) * NL + L2 : 0>();
    finish(c + 1, sidx);
    meet();
#pragma unroll
    for (int q = 0; NEXT && q < PART; ++q) issue(q, c + ST, here);
  };
  const auto run = [&](const auto& f) {
    int c = c0;
    for (; c + ST <= last; ++c) f(c, std::true_type(), std::true_type());
    if (c - 1 + ST <= last) f(c++, std::true_type(), std::false_type());
    for (; c <= last; ++c) f(c, std::false_type(), std::false_type());
  };
  if (GROUPED && 16 * wm * MT >= rows) run(idle);
  else run(step);
#pragma unroll
  for (int u = T - 2; u < T; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[u][e] = __builtin_fmaf(d[u & 3][e], f[u % MT], acc[u][e]);
  wait_loads<0>();
  __syncthreads();

  // Block t = i MT + j: lane (l16, g) holds row 16 j + l16 of X and rows 4 g +
  // 0..3 of the 16 of W, four neighbouring outputs of one row.  The FP32 sums of a
  // slice go to the workspace.  A BF16 tile goes through LDS (the stages are free),
  // so that the stores to Y are whole rows: [TM rows][TN columns], 16-byte pieces
  // swizzled as above.
  const int64_t cols = p.n - n0 < TN ? p.n - n0 : TN;
  uint16_t* yt = reinterpret_cast<uint16_t*>(&stage[0]);
  const auto put_sums = [&](int i, int j, const f32x4_t& v) {
    const int r = 16 * (wm * MT + j) + l16, col = 16 * (wn * NT + i) + 4 * g;
    float* part = p.part + (int64_t)slice * p.m * p.np;
    if (r < rows && col < cols) *reinterpret_cast<f32x4_t*>(part + (m0 + r) * p.np + n0 + col) = v;
  };
  const auto put_tile = [&](int i, int j, const f32x4_t& v) {
    const int r = 16 * (wm * MT + j) + l16, col = 16 * (wn * NT + i) + 4 * g;
    *reinterpret_cast<uint2*>(yt + r * TN + 8 * ((col >> 3) ^ (r & 7)) + (col & 4)) =
        make_uint2(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]));
  };
  if (far == 0) {
    if (p.slices > 1) {
#pragma unroll
      for (int t = 0; t < T; ++t) put_sums(t / MT, t % MT, acc[t]);
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) put_tile(t / MT, t % MT, acc[t]);
    }
  } else {
    // Two scales, neither 0, whose product is no normal FP32 number: this wavefront's
    // sums again, block by block from memory, with the scales taken apart.  (So in the
    // loop above, for every tile: 2048 x 17408 x 5120 198.5 us, 190.5 this way, and
    // 3.1 ms where every tile has such scales.)
    const uint8_t* xq = GROUPED ? p.xq : p.xq + m0 * p.k;
    const float* xs = GROUPED ? p.xs : p.xs + m0 * p.kb;
#pragma unroll 1
    for (int t = 0; t < T; ++t) {
      const int64_t wr = row_or_last(n0 + 16 * (wn * NT + t / MT) + l16, p.n);
      const int64_t xr = x_row(16 * (wm * MT + t % MT) + l16);
      const uint8_t *wp = wq + wr * p.k, *xp = xq + xr * p.k;
      const float *wsp = ws + (wr >> 7) * p.kb, *xsp = xs + xr * p.kb;
      f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        // Pieces past the end of a row: the row's last piece of W, zeros of X.
        bool in0, in1;
        const int64_t o0 = again_offset(c, p.k, g, 0, &in0), o1 = again_offset(c, p.k, g, 1, &in1);
        const auto load = [](const uint8_t* q) { return *reinterpret_cast<const uint4*>(q); };
        const uint4 z = make_uint4(0, 0, 0, 0), x0 = load(xp + o0), x1 = load(xp + o1);
        const float sw = wsp[c], sx = xsp[c];
        const int ew = scale_exp(sw), ex = scale_exp(sx);
        const f32x4_t d = mfma128(mfma_frag(load(wp + o0), load(wp + o1)), mfma_frag(in0 ? x0 : z, in1 ? x1 : z), ew, ex);
        const float f = scale_rest(sx, ex) * scale_rest(sw, ew);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(d[e], f, v[e]);
      }
      if (p.slices > 1) put_sums(t / MT, t % MT, v);
      else put_tile(t / MT, t % MT, v);
    }
  }
  if (p.slices > 1) return;
  __syncthreads();
  typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
  const bool vec = (p.n & 7) == 0 && (p.ld & 7) == 0;
#pragma unroll 4
  for (int pi = tid; pi < TM * (TN / 8); pi += 512) {
    const int r = pi / (TN / 8), c8 = 8 * (pi - r * (TN / 8));
    if (r >= rows || c8 >= cols) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(yt + r * TN + 8 * ((c8 >> 3) ^ (r & 7)));
    const int64_t row = GROUPED ? (int64_t)perm[m0 + r] : m0 + r;
    uint16_t* dst = p.y + row * p.ld + n0 + c8;
    if (vec) {
      *reinterpret_cast<u32x4_t*>(dst) = u32x4_t{v.x, v.y, v.z, v.w};
    } else {
      const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (c8 + t < cols) dst[t] = (uint16_t)(e[t >> 1] >> (16 * (t & 1)));
    }
  }
}

// Sums of the slices in slice order, 4 outputs per thread: bound by its reads (4
// slices of 333 x 5000: 5.6 us with the launch).
__global__ void __launch_bounds__(256) fp8_join_kernel(const float* __restrict__ part, int slices, uint32_t quads,
                                                       uint32_t n, uint16_t* __restrict__ y) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  f32x4_t s = reinterpret_cast<const f32x4_t*>(part)[i];
  for (int t = 1; t < slices; ++t) {
    const f32x4_t o = reinterpret_cast<const f32x4_t*>(part)[(size_t)t * quads + i];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += o[e];
  }
  if ((n & 3) == 0) {
    reinterpret_cast<uint2*>(y)[i] = make_uint2(bf16x2_of(s[0], s[1]), bf16x2_of(s[2], s[3]));
    return;
  }
  const uint32_t per_row = (n + 3) >> 2, row = i / per_row, col = 4 * (i - row * per_row);
  for (uint32_t e = 0; e < 4 && col + e < n; ++e) y[(size_t)row * n + col + e] = (uint16_t)f32_to_bf16_rne(s[e]);
}

}  // namespace

namespace {

template <int S>
void launch_tiles(GemmArgs a, hipStream_t s) {
  constexpr Shape t = kShapes[S];
  a.n_tiles = (int)((a.n + t.tn - 1) / t.tn);
  a.m_tiles = (int)((a.m + t.tm - 1) / t.tm);
  fp8_gemm_kernel<t.tn, t.tm, t.wn, t.wm, t.stages, false>
      <<<dim3((unsigned)((int64_t)a.n_tiles * a.m_tiles * a.slices)), 512, 0, s>>>(a);
}

void launch_shape(int shape, const GemmArgs& a, hipStream_t s) {
  switch (shape) {
    case 0: launch_tiles<0>(a, s); break;
    case 1: launch_tiles<1>(a, s); break;
    case 2: launch_tiles<2>(a, s); break;
    default: launch_tiles<3>(a, s); break;
  }
}

}  // namespace

bool fp8_gemm_supported(int64_t m, int64_t n, int64_t k) { return gemm_supported(m, n, k); }

double fp8_gemm_ns(int64_t m, int64_t n, int64_t k, bool split) { return gemm_plan(m, n, k, split).ns; }

int64_t fp8_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  const Plan p = gemm_plan(m, n, k, true);
  return p.slices > 1 ? 4 * m * sums_per_row(n) * p.slices : 0;
}

bool fp8_gemm_grouped_supported(int64_t t_count, int64_t topk, int64_t experts, int64_t n, int64_t k) {
  return grouped_supported(t_count, topk, experts, n, k);
}

// Experts that pairs with independent uniform ids are expected to choose.
double fp8_experts_chosen(int64_t pairs, int64_t experts) {
  return -(double)experts * expm1(-(double)pairs / (double)experts);
}

// Estimated time of sort and GEMM, for up to 128 pairs per expert.
double fp8_gemm_grouped_ns(int64_t pairs, int64_t experts, int64_t n, int64_t k) {
  const int64_t chunks = (k + kChunk - 1) / kChunk;
  const double wgs = (double)((n + 255) / 256) * fp8_experts_chosen(pairs, experts);
  const double rounds = ceil(wgs / kCus), filled = wgs < kCus ? wgs : kCus;
  return 10500.0 + rounds * (3000.0 + (600.0 + 3.6 * filled) * (double)chunks);
}

void launch_fp8_gemm_grouped(const uint8_t* xq, const float* xs, int64_t topk, const int32_t* groups, int64_t pairs,
                             int64_t experts, int64_t n, int64_t k, const uint8_t* wq, const float* ws, uint16_t* y,
                             hipStream_t s) {
  const int64_t m_tiles = grouped_m_tiles(pairs, experts);  // per XCD
  const int64_t n_tiles = (n + 255) / 256;
  const GemmArgs a{xq, xs, wq, ws, y, pairs, n, k, n, (int)((k + kChunk - 1) / kChunk), (int)((n + 127) / 128),
                   (int)n_tiles, (int)m_tiles, 1, 0, nullptr, groups, experts, topk};
  constexpr Shape t = kShapes[kGroupedShape];
  fp8_gemm_kernel<t.tn, t.tm, t.wn, t.wm, t.stages, true><<<dim3((unsigned)(8 * n_tiles * m_tiles)), 512, 0, s>>>(a);
}

void launch_fp8_gemm(const uint8_t* xq, const float* xs, int64_t m, int64_t n, int64_t k, const uint8_t* wq,
                     const float* ws, uint16_t* y, void* workspace, hipStream_t s) {
  const Plan p = gemm_plan(m, n, k, workspace != nullptr);
  GemmArgs a{xq, xs, wq, ws, y, m, n, k, n, (int)((k + kChunk - 1) / kChunk), (int)((n + 127) / 128), 0, 0, p.slices,
             sums_per_row(n), static_cast<float*>(workspace), nullptr, 1, 1};
  Launch l[2];
  const int launches = launches_of(p, n, l);
  for (int i = 0; i < launches; ++i) {  // n0: a multiple of 256
    a.wq = wq + l[i].n0 * k, a.ws = ws + l[i].n0 / 128 * a.kb, a.y = y + l[i].n0;
    a.n = l[i].n, a.nb = (int)((l[i].n + 127) / 128);
    launch_shape(l[i].shape, a, s);
  }
  if (p.slices > 1) {
    const int64_t quads = m * (a.np / 4);  // at most 2^24 and a few
    fp8_join_kernel<<<dim3((unsigned)((quads + 255) / 256)), 256, 0, s>>>(a.part, p.slices, (uint32_t)quads,
                                                                          (uint32_t)n, y);
  }
}

}  // namespace nvfp4
