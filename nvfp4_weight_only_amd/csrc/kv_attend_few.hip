// Attention over a paged FP4 cache for few rows a sequence (decoding, a few drafted
// tokens): bound by reading the cache.
//
// Every workgroup takes an equal, consecutive share of all units (a unit: 32 tw tokens
// of one tile of rows of one sequence, for hw heads), found from the lengths on the
// device, so that long and short sequences mix without idle CUs and the host needs no
// length.  A share that covers a unit list's end in the middle leaves partial results,
// which kv_attend_join_kernel joins.  A wavefront takes one key/value head and every
// tw-th tile of 32 tokens: the heads of a group share the lines of codes and scales.
//
// A tile: the scores as S^T = K Q^T, tokens by rows.  A lane holds a quarter of a token's
// key as it lies in memory (16 bytes of codes at 128 elements), which is a fragment of K
// if the query's elements are taken in the same order.  The output is O^T = V^T P^T: the
// scores' layout is that of P^T's fragments, if V's tokens are taken in that order;
// values go through LDS in 16 bits, where transposing reads (ds_read_b64_tr_b16) pick
// up 4 tokens of a column.  A lane then holds scores, statistics and outputs of one row
// (lane % 16), and the maximum is exchanged only where it has grown by kSlack.
#include <type_traits>

#include "kv_attend.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

constexpr int kFewThreads = 512, kFewWaves = kFewThreads / 64;
constexpr int kFewTokens = 32;

// LDS of a wavefront: 32 tokens' values, rows 32 bytes longer than the values so that 8
// rows start in different banks; at the end 16 rows of outputs, maximum and sum.
template <int NS>
struct FewLds {
  static constexpr int kD = 32 * NS;
  static constexpr int kRow = 2 * kD + 32;
  static constexpr int kOut = kD + 4;  // floats of an output row
  static constexpr int kStats = 16 * kOut * 4;
  static constexpr int kBytes = (kFewTokens * kRow > kStats + 128 ? kFewTokens * kRow : kStats + 128);
};

// A tile's codes and scales as loaded: token lane % 16 (+ 16) of the tile, quarter lane / 16 of its row.
template <int NS>
struct FewTile {
  uint32_t k[2][NS], v[2][NS];
  uint32_t ks[2], vs[2];
  uint32_t there[2];  // bit t: token t of the half tile is in the cache
};

// Sum over the workgroup of one value a thread, and the sum of the threads before.
__device__ __forceinline__ int64_t few_scan(int64_t v, int64_t* total) {
  __shared__ int64_t wsum[kFewWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t up = __shfl_up(inc, d, 64);
    if (lane >= d) inc += up;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kFewWaves; ++i) {
    before += i < wave ? wsum[i] : 0;
    all += wsum[i];
  }
  __syncthreads();
  *total = all;
  return before + inc - v;
}

template <bool MX, bool BF16, int NS, int RT>
__global__ void __launch_bounds__(kFewThreads) kv_attend_few_kernel(AttendArgs a) {
  using L = FewLds<NS>;
  using SB = ScaleBytes<MX, NS>;
  constexpr int kD = L::kD, kRows = 16 * RT, kTerms = AttendTypes<MX, BF16>::kTerms;
  __shared__ __attribute__((aligned(16))) char lds[kFewWaves * L::kBytes];
  __shared__ int64_t start[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quarter = lane >> 4;
  const int hg = blockIdx.x % a.hgroups, wg = blockIdx.x / a.hgroups;
  const int head = hg * a.hw + wave % a.hw, slice = wave / a.hw;
  const bool active = slice < a.tw && head < (int)a.c.heads;
  const int tokens_tile = kFewTokens * a.tw;

  // This workgroup's units.
  int64_t total = 0, pre = 0, u = 0;
  for (int64_t s0 = 0; s0 < a.b.seqs; s0 += kFewThreads) {
    const int64_t s = s0 + tid;
    u = 0;
    if (s < a.b.seqs) {
      const SeqWork w = seq_work(a, s, kRows, tokens_tile);
      u = w.rtiles * w.ttiles;
    }
    int64_t chunk;
    pre = total + few_scan(u, &chunk);
    total += chunk;
    if (blockIdx.x == 0 && s < a.b.seqs) a.prefix[s] = pre;
  }
  if (blockIdx.x == 0 && tid == 0) a.prefix[a.b.seqs] = total;
  const int64_t nwg = sharing(a, total);
  if (wg >= nwg) return;
  int64_t cur = wg * total / nwg;
  const int64_t end = (wg + 1) * total / nwg;
  if (a.b.seqs <= kFewThreads) {
    if (pre <= cur && cur < pre + u) {
      start[0] = tid;
      start[1] = cur - pre;
    }
  } else {
    int64_t sum = 0;
    for (int64_t s0 = 0; s0 < a.b.seqs && sum <= cur; s0 += kFewThreads) {
      const int64_t s = s0 + tid;
      u = 0;
      if (s < a.b.seqs) {
        const SeqWork w = seq_work(a, s, kRows, tokens_tile);
        u = w.rtiles * w.ttiles;
      }
      int64_t chunk;
      pre = sum + few_scan(u, &chunk);
      sum += chunk;
      if (pre <= cur && cur < pre + u) {
        start[0] = s;
        start[1] = cur - pre;
      }
    }
  }
  __syncthreads();
  int64_t seq = start[0], off = start[1];

  const float ts_k = MX ? 1.0f : *a.c.tscale[0], ts_v = MX ? 1.0f : *a.c.tscale[1];
  char* vbuf = lds + wave * L::kBytes;
  const int64_t head_at = head < (int)a.c.heads ? head : 0;

  while (cur < end) {
    const SeqWork w = seq_work(a, seq, kRows, tokens_tile);
    if (w.rtiles == 0) {
      ++seq;
      continue;
    }
    const int64_t rtile = off / w.ttiles, t0 = off - rtile * w.ttiles;
    const int64_t n = w.ttiles - t0 < end - cur ? w.ttiles - t0 : end - cur;
    const int32_t lo = (int32_t)w.lo, hi = (int32_t)w.hi, packed = (int32_t)(w.r.count * a.g);
    const int32_t* table = a.b.block_table + seq * a.b.max_blocks;

    // The rows of this tile: row col of sub-tile rt is packed row i g + j, query head head g + j of row i.
    u32x4v_t q[RT][kTerms][NS];
    f32x4_t o[RT][2 * NS];
    float factor[RT], m[RT], l[RT];
    int32_t pos[RT], first[RT];  // tokens first .. pos are seen
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int64_t pr = rtile * kRows + 16 * rt + col;
      const bool live = active && pr < packed;
      const int32_t i = fastdiv(live ? (int32_t)pr : 0, a.group), j = live ? (int32_t)pr - i * a.g : 0;
      const int64_t p = w.r.first + i + w.r.shift;
      pos[rt] = (int32_t)(p < -1 ? -1 : p);
      first[rt] = a.window > 0 && p - a.window + 1 > 0 ? (int32_t)(p - a.window + 1) : 0;
      const uint16_t* src = a.q + (w.r.first + i) * a.q_row + (head_at * a.g + j) * a.q_head + quarter * 8 * NS;
      float amax = 0.0f;
      u32x4v_t raw[NS];
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        raw[c] = live ? *reinterpret_cast<const u32x4v_t*>(src + 8 * c) : u32x4v_t{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(half_to_f32<BF16>(raw[c][e] & 0xFFFFu)), fabsf(half_to_f32<BF16>(raw[c][e] >> 16))));
      }
      amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
      amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
      const RowScale rs = row_scale<MX>(amax, a.scale, ts_k);
      factor[rt] = rs.factor;
#pragma unroll
      for (int c = 0; c < NS; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = half_to_f32<BF16>(raw[c][e] & 0xFFFFu) * rs.mul, y = half_to_f32<BF16>(raw[c][e] >> 16) * rs.mul;
          const uint32_t t = pack2<MX>(x, y);
          q[rt][0][c][e] = t;
          if constexpr (kTerms == 2) q[rt][kTerms - 1][c][e] = pack2_rest(x, y, t);
        }
#pragma unroll
      for (int d = 0; d < 2 * NS; ++d) o[rt][d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      m[rt] = -__builtin_inff();
      l[rt] = 0.0f;
    }
    // Tokens that every row of the tile sees.
    const int64_t i0 = rtile * kRows / a.g;
    const int64_t i1 = ((rtile + 1) * kRows - 1) / a.g < w.r.count ? ((rtile + 1) * kRows - 1) / a.g : w.r.count - 1;
    const int64_t all_pos = w.r.first + i0 + w.r.shift;
    const int64_t all_first = a.window > 0 ? w.r.first + i1 + w.r.shift - a.window + 1 : 0;

    const auto base_of = [&](int64_t tile) { return lo + (int32_t)((t0 + tile) * a.tw + slice) * kFewTokens; };
    // Cache rows of this lane's two tokens of a tile, -1 where there is none.
    const auto find = [&](int64_t tile, int64_t (&row)[2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        row[h] = -1;
        const int32_t t = base_of(tile) + 16 * h + col;
        if (active && tile < n && t < hi) {
          const int32_t page = fastdiv(t, a.page);
          const int64_t id = table[page];
          if (id >= 0 && id < a.c.num_blocks)
            row[h] = (id * a.c.block_size + (t - page * a.page.d)) * a.c.heads + head_at;
        }
      }
    };
    const auto load = [&](const int64_t (&row)[2], FewTile<NS>& t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        t.there[h] = (uint32_t)__ballot(row[h] >= 0) & 0xFFFFu;
        const int64_t r = row[h] >= 0 ? row[h] : 0;
        const uint32_t* kc = reinterpret_cast<const uint32_t*>(a.c.codes[0] + r * (kD / 2)) + quarter * NS;
        const uint32_t* vc = reinterpret_cast<const uint32_t*>(a.c.codes[1] + r * (kD / 2)) + quarter * NS;
        __builtin_memcpy(t.k[h], kc, 4 * NS);
        t.ks[h] = SB::load(a.c.scales[0] + r * SB::kRow + SB::base(quarter));
        __builtin_memcpy(t.v[h], vc, 4 * NS);
        t.vs[h] = SB::load(a.c.scales[1] + r * SB::kRow + SB::base(quarter));
        if (row[h] < 0) {  // values of tokens that are not there count as 0, whatever lies in the cache
#pragma unroll
          for (int c = 0; c < NS; ++c) t.v[h][c] = 0;
          t.vs[h] = 0;
        }
      }
    };
    const auto compute = [&](int64_t tile, const FewTile<NS>& t) {
      const int32_t tb = base_of(tile);
      const bool masked = t.there[0] != 0xFFFFu || t.there[1] != 0xFFFFu || tb + 31 > all_pos || tb < all_first;
      f32x4_t sc[RT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4v_t kf[NS];
        decode_quarter<MX, NS>(t.k[h], t.ks[h], quarter, kf);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int x = 0; x < kTerms; ++x)
#pragma unroll
            for (int c = 0; c < NS; ++c) acc = mfma16<MX>(kf[c], q[rt][x][c], acc);
          sc[rt][h] = acc;
        }
        u32x4v_t vf[NS];
        decode_quarter<MX, NS>(t.v[h], t.vs[h], quarter, vf);
#pragma unroll
        for (int c = 0; c < NS; ++c)
          *reinterpret_cast<u32x4v_t*>(vbuf + (16 * h + col) * L::kRow + (quarter * NS + c) * 16) = vf[c];
      }
      wave_lds_sync();
      // Some row sees a token that another does not: where its value is not finite, 0 times it is not 0.
      const bool apart = masked && __any(scale_nonfinite<MX>(t.vs[0], SB::kLoad) || scale_nonfinite<MX>(t.vs[1], SB::kLoad));
      u32x4v_t pf[RT][kTerms];
      float pw[RT][2][4];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = -__builtin_inff();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float s = sc[rt][h][e] * factor[rt];
            if (masked) {
              const int32_t tok = tb + 16 * h + 4 * quarter + e;
              const bool seen = (t.there[h] >> (4 * quarter + e)) & 1u && tok <= pos[rt] && tok >= first[rt];
              s = seen ? s : -__builtin_inff();
            }
            sc[rt][h][e] = s;
            top = fmaxf(top, s);
          }
        if (__any(top > m[rt] + kSlack)) {
          top = fmaxf(top, __shfl_xor(top, 16, 64));
          top = fmaxf(top, __shfl_xor(top, 32, 64));
          const float next = fmaxf(m[rt], top);
          const float shrink = next == m[rt] ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - next);
          m[rt] = next;
          l[rt] *= shrink;
#pragma unroll
          for (int d = 0; d < 2 * NS; ++d) o[rt][d] *= shrink;
        }
        const float mm = m[rt] == -__builtin_inff() ? 0.0f : m[rt] - kWeightBias;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pw[rt][h][e] = __builtin_amdgcn_exp2f(sc[rt][h][e] - mm);
            l[rt] += pw[rt][h][e];
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t p = pack2<MX>(pw[rt][h][2 * e], pw[rt][h][2 * e + 1]);
            pf[rt][0][2 * h + e] = p;
            if constexpr (kTerms == 2) pf[rt][kTerms - 1][2 * h + e] = pack2_rest(pw[rt][h][2 * e], pw[rt][h][2 * e + 1], p);
          }
        }
      }
      if (!apart) {
        // Tokens 4 quarter .. + 3 of both half tiles, columns 16 d ..: lane col of a quarter reads row col / 4.
        const char* at = vbuf + (4 * quarter + (col >> 2)) * L::kRow + (col & 3) * 8;
#pragma unroll
        for (int d = 0; d < 2 * NS; ++d) {
          typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
          const i16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(__attribute__((address_space(3))) char*)(at + 32 * d));
          const i16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(__attribute__((address_space(3))) char*)(at + 32 * d + 16 * L::kRow));
          const u32x4v_t vt = __builtin_bit_cast(u32x4v_t, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int x2 = 0; x2 < kTerms; ++x2) o[rt][d] = mfma16<MX>(vt, pf[rt][x2], o[rt][d]);
        }
      } else {
        // Token by token, each row adding only what it sees.
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll 1
          for (int tk = 0; tk < 16; ++tk) {
            const int32_t tok = tb + 16 * h + tk;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              const float mine = tk & 2 ? (tk & 1 ? pw[rt][h][3] : pw[rt][h][2]) : (tk & 1 ? pw[rt][h][1] : pw[rt][h][0]);
              const float p = __shfl(mine, (tk >> 2) * 16 + col, 64);
              const bool seen = (t.there[h] >> tk) & 1u && tok <= pos[rt] && tok >= first[rt];
#pragma unroll
              for (int d = 0; d < 2 * NS; ++d) {
                const uint16_t* row = reinterpret_cast<const uint16_t*>(vbuf + (16 * h + tk) * L::kRow) + 16 * d + 4 * quarter;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[rt][d][e] += seen ? p * half_to_f32<MX>(row[e]) : 0.0f;
              }
            }
          }
      }
      wave_lds_sync();
    };

    FewTile<NS> even, odd;
    int64_t row[2];
    find(0, row);
    load(row, even);
    find(1, row);
    for (int64_t tile = 0; tile < n; tile += 2) {
      load(row, odd);
      find(tile + 2, row);
      if (active) compute(tile, even);
      if (tile + 1 >= n) break;
      load(row, even);
      find(tile + 3, row);
      if (active) compute(tile + 1, odd);
    }

    // Join the slices; whole sequences' outputs are written, parts kept.
    const bool whole = t0 == 0 && n == w.ttiles;
    float* part = a.part + ((int64_t)blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * (a.hw * kRows * (kD + 2));
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] += __shfl_xor(l[rt], 16, 64);
      l[rt] += __shfl_xor(l[rt], 32, 64);
      __syncthreads();  // the values, or the rows before, are done with
      float* ob = reinterpret_cast<float*>(vbuf);
      float2* st = reinterpret_cast<float2*>(vbuf + L::kStats);
#pragma unroll
      for (int d = 0; d < 2 * NS; ++d)
        *reinterpret_cast<f32x4_t*>(ob + col * L::kOut + 16 * d + 4 * quarter) = o[rt][d];
      if (quarter == 0) st[col] = make_float2(m[rt], l[rt]);
      __syncthreads();
      for (int i = tid; i < a.hw * 16 * (kD / 4); i += kFewThreads) {
        const int d4 = i % (kD / 4), r = i / (kD / 4) % 16, hh = i / (kD / 4) / 16;
        const int64_t pr = rtile * kRows + 16 * rt + r;
        if (hg * a.hw + hh >= (int)a.c.heads || pr >= packed) continue;
        float top = -__builtin_inff();
        for (int k = 0; k < a.tw; ++k)
          top = fmaxf(top, reinterpret_cast<const float2*>(lds + (k * a.hw + hh) * L::kBytes + L::kStats)[r].x);
        const float mm = top == -__builtin_inff() ? 0.0f : top;
        float sum = 0.0f;
        f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < a.tw; ++k) {
          const char* buf = lds + (k * a.hw + hh) * L::kBytes;
          const float2 ml = reinterpret_cast<const float2*>(buf + L::kStats)[r];
          const float f = __builtin_amdgcn_exp2f(ml.x - mm);
          sum += ml.y * f;
          acc += *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(buf) + r * L::kOut + 4 * d4) * f;
        }
        if (whole) {
          const int32_t qi = fastdiv((int32_t)pr, a.group), qj = (int32_t)pr - qi * a.g;
          const float inv = sum == 0.0f ? 0.0f : ts_v / sum;
          store_out4<BF16>(a.out + ((w.r.first + qi) * a.q_heads + (hg * a.hw + hh) * a.g + qj) * kD + 4 * d4, acc * inv);
        } else {
          const int at = (hh * RT + rt) * 16 + r;
          *reinterpret_cast<f32x4_t*>(part + (int64_t)at * kD + 4 * d4) = acc;
          if (d4 == 0) reinterpret_cast<float2*>(part + (int64_t)a.hw * kRows * kD)[at] = make_float2(top, sum);
        }
      }
    }
    __syncthreads();
    cur += n;
    off += n;
    if (off == w.rtiles * w.ttiles) {
      ++seq;
      off = 0;
    }
  }
}

// Joins the parts of one row and query head, if its tokens were shared: their maxima,
// sums and outputs, in the workgroups' order.
constexpr int kJoinThreads = 256;
constexpr int kJoinParts = 2048;  // workgroups at most

template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) kv_attend_join_kernel(AttendArgs a, int rows_tile, int head_dim,
                                                                      const float* ts_p) {
  __shared__ float weight[kJoinParts];
  __shared__ f32x4_t acc[kJoinThreads];
  __shared__ float red[kJoinThreads / 64];
  __shared__ int64_t at[2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t r = blockIdx.x;
  const int qh = blockIdx.y;
  if (tid < 64) {
    int64_t s = r;
    if (a.b.row_start) {
      int64_t lo = 0, hi = a.b.seqs;
      while (hi - lo > 1) {
        const int64_t step = (hi - lo + 63) / 64, x = lo + lane * step;
        const bool le = x < hi && (int64_t)a.b.row_start[x] <= r;
        const int n = __popcll(__ballot(le));
        if (n == 0) break;
        lo += (int64_t)(n - 1) * step;
        hi = lo + step < hi ? lo + step : hi;
      }
      s = lo;
    }
    if (lane == 0) at[0] = s;
  }
  __syncthreads();
  const int64_t s = at[0];
  if (s >= a.b.seqs) return;
  const SeqWork w = seq_work(a, s, rows_tile, kFewTokens * a.tw);
  if (w.rtiles == 0 || r < w.r.first || r >= w.r.first + w.r.count) return;
  const int64_t total = a.prefix[a.b.seqs], nwg = sharing(a, total);
  const int head = qh / a.g, hg = head / a.hw, hh = head - hg * a.hw;
  const int64_t pr = (r - w.r.first) * a.g + (qh - head * a.g), rtile = pr / rows_tile;
  const int64_t u0 = a.prefix[s] + rtile * w.ttiles, u1 = u0 + w.ttiles;
  const int64_t w0 = ((u0 + 1) * nwg - 1) / total, w1 = (u1 * nwg - 1) / total;
  const int parts = (int)(w1 - w0 + 1);
  if (parts <= 1) return;
  const int64_t slot = (int64_t)a.hw * rows_tile * (head_dim + 2);
  const int64_t row = (int64_t)hh * rows_tile + (pr - rtile * rows_tile);
  const auto part_of = [&](int p) { return a.part + (((w0 + p) * a.hgroups + hg) * 2 + (p == 0 ? 1 : 0)) * slot; };
  const auto stats_of = [&](int p) { return reinterpret_cast<const float2*>(part_of(p) + (int64_t)a.hw * rows_tile * head_dim)[row]; };
  float top = -__builtin_inff();
  for (int p = tid; p < parts; p += kJoinThreads) {
    const float m = stats_of(p).x;
    weight[p] = m;
    top = fmaxf(top, m);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  if (lane == 0) red[tid >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float mm = top == -__builtin_inff() ? 0.0f : top;
  float sum = 0.0f;
  for (int p = tid; p < parts; p += kJoinThreads) {
    const float f = __builtin_amdgcn_exp2f(weight[p] - mm);
    weight[p] = f;
    sum += f * stats_of(p).y;
  }
  sum = wave_sum(sum);
  __syncthreads();
  if (lane == 0) red[tid >> 6] = sum;
  __syncthreads();
  sum = red[0] + red[1] + red[2] + red[3];
  const int quads = head_dim / 4, groups = kJoinThreads / quads, d4 = tid % quads, gi = tid / quads;
  f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (gi < groups)
    for (int p = gi; p < parts; p += groups)
      x += *reinterpret_cast<const f32x4_t*>(part_of(p) + row * head_dim + 4 * d4) * weight[p];
  acc[tid] = x;
  __syncthreads();
  if (gi == 0) {
    for (int i = 1; i < groups; ++i) x += acc[i * quads + d4];
    const float ts = ts_p ? *ts_p : 1.0f;
    store_out4<BF16>(a.out + (r * a.q_heads + qh) * head_dim + 4 * d4, x * (sum == 0.0f ? 0.0f : ts / sum));
  }
}

template <int RT>
void launch_few(AttendArgs a, bool bf16, hipStream_t s) {
  const dim3 grid((unsigned)(a.nwg * a.hgroups));
  const auto go = [&](auto mx, auto bf, auto ns) {
    kv_attend_few_kernel<decltype(mx)::value, decltype(bf)::value, decltype(ns)::value, RT>
        <<<grid, kFewThreads, 0, s>>>(a);
  };
  const auto dim = [&](auto mx, auto bf) {
    switch (a.c.head_dim / 32) {
      case 2: return go(mx, bf, std::integral_constant<int, 2>{});
      case 3: return go(mx, bf, std::integral_constant<int, 3>{});
      case 4: return go(mx, bf, std::integral_constant<int, 4>{});
      case 6: return go(mx, bf, std::integral_constant<int, 6>{});
      default: return go(mx, bf, std::integral_constant<int, 8>{});
    }
  };
  if (a.c.mx) {
    if (bf16) dim(std::true_type{}, std::true_type{});
    else dim(std::true_type{}, std::false_type{});
  } else {
    if (bf16) dim(std::false_type{}, std::true_type{});
    else dim(std::false_type{}, std::false_type{});
  }
  const dim3 join((unsigned)a.b.rows, (unsigned)a.q_heads);
  const float* ts = a.c.mx ? nullptr : a.c.tscale[1];
  if (bf16) kv_attend_join_kernel<true><<<join, kJoinThreads, 0, s>>>(a, 16 * RT, (int)a.c.head_dim, ts);
  else kv_attend_join_kernel<false><<<join, kJoinThreads, 0, s>>>(a, 16 * RT, (int)a.c.head_dim, ts);
}

// Heads of a workgroup, its token slices, workgroups and 16-row tiles.
struct FewPlan {
  int hw, tw, hgroups, nwg, rt;
  int64_t part_floats;
};
FewPlan few_plan(int64_t heads, int64_t head_dim, int64_t q_heads, int64_t rows, int64_t seqs) {
  FewPlan p;
  const int64_t groups = (heads + kFewWaves - 1) / kFewWaves;
  p.hw = (int)((heads + groups - 1) / groups);
  p.hgroups = (int)((heads + p.hw - 1) / p.hw);
  p.tw = kFewWaves / p.hw;
  const int per_cu = head_dim > 192 ? 1 : 2;
  p.nwg = 256 * per_cu / p.hgroups;
  if (p.nwg < 1) p.nwg = 1;
  p.rt = rows * (q_heads / heads) > 16 * seqs ? 2 : 1;
  p.part_floats = (int64_t)p.nwg * p.hgroups * 2 * p.hw * 16 * p.rt * (head_dim + 2);
  return p;
}

}  // namespace

int64_t kv_attend_workspace_bytes(int64_t heads, int64_t head_dim, int64_t q_heads, int64_t rows, int64_t seqs) {
  const FewPlan p = few_plan(heads, head_dim, q_heads, rows, seqs);
  return p.part_floats * 4 + (seqs + 2) / 2 * 16;
}

void launch_kv_attend(const KvCache& c, const KvBatch& b, bool bf16, const uint16_t* q, int64_t q_heads, int64_t q_row,
                      int64_t q_head, float scale, int64_t window, uint16_t* out, void* workspace, hipStream_t s) {
  const FewPlan p = few_plan(c.heads, c.head_dim, q_heads, b.rows, b.seqs);
  AttendArgs a;
  a.c = c;
  a.b = b;
  a.page = make_fastdiv(c.block_size);
  a.group = make_fastdiv(q_heads / c.heads);
  a.cap = b.max_blocks * c.block_size;
  a.q = q;
  a.q_row = q_row;
  a.q_head = q_head;
  a.out = out;
  a.q_heads = (int32_t)q_heads;
  a.g = (int32_t)(q_heads / c.heads);
  a.scale = scale;
  a.window = (int32_t)window;
  a.hw = p.hw;
  a.tw = p.tw;
  a.hgroups = p.hgroups;
  a.nwg = p.nwg;
  a.part = static_cast<float*>(workspace);
  a.prefix = reinterpret_cast<int64_t*>(a.part + p.part_floats);
  if (p.rt == 1) launch_few<1>(a, bf16, s);
  else launch_few<2>(a, bf16, s);
}

}  // namespace nvfp4
