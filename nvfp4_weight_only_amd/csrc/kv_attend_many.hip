// Attention over a paged FP4 cache for many rows a sequence (prompts, chunks of prompts):
// bound by the matrix cores and the softmax's vector instructions.
//
// A workgroup takes tiles of 32 rows a wavefront (row i of a sequence with its g query
// heads of one key/value head: rows i g .. i g + g - 1 of the packed rows) and walks over
// 64 tokens at a time.  Each thread loads a quarter of a token's key or value, two tiles
// ahead its page's id and one tile ahead its codes, and decodes it into LDS once for all
// rows, in 16 bits and double buffered, so that one barrier a tile is enough.  Scores are
// S^T = K Q^T (32 tokens by 32 rows), outputs O^T = V^T P^T: a lane then holds scores,
// statistics and outputs of one row (lane % 32), and the scores' layout is that of P^T's
// fragments if a step of 16 tokens takes them in the order 0-3, 8-11 (lanes 0-31), 4-7,
// 12-15 (lanes 32-63); V^T's fragments in that order come from transposing reads.
//
// The work is split evenly as for few rows, but over units (64 tokens of one tile of
// rows) that some row sees: kv_attend_plan_kernel lists the tiles of rows with the number
// of units before each.  Workgroups are numbered so that an XCD's are consecutive: they
// read the same key/value head's tokens from its L2.
//
// Measured: 2048 rows behind 6144 tokens (40 query heads on 8 of 128, 3.0e11 operations;
// NVFP4 and BF16, one term a weight) 360 us, 0.8 PFLOP/s (a large library product reaches
// 1.4), plan 5 and join 17: matrix cores busy 42 % of the clocks, vector instructions 48 %, LDS
// reads 128 bytes a clock in the phases that multiply.  All three kernels in a captured graph:
// 343 us, MXFP4 415, FP16 427; MXFP4 and FP16 with two terms of query and weights 568, where
// heads of 128 spill 41 registers a lane (of 64 none, of 96 18, of 256 19; one term of the
// query and two of the weights at most 7).
#include <type_traits>

#include "kv_attend.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kManyTokens = 64;

template <int NS>
struct Many {
  static constexpr int kD = 32 * NS;
  static constexpr int kWaves = NS <= 4 ? 8 : 4;  // two a SIMD with 256 registers, or one with 512
  static constexpr int kThreads = 64 * kWaves, kRows = 32 * kWaves;
  static constexpr int kItems = 512 / kThreads;  // quarters of keys and values that a thread decodes
  // Rows in LDS: 32 tokens' 16-byte pieces of a key, and 4 tokens' 64-byte pieces of a value, in different banks.  Piece p
  // (16 bytes) of token t's value lies at p ^ (t / 4 % 4), for the writes: a wavefront writes 16 tokens' pieces at once.
  static constexpr int kKeyRow = 2 * kD + 16, kValueRow = 2 * kD + 64;
  static constexpr int kValues = kManyTokens * kKeyRow, kBuffer = kValues + kManyTokens * kValueRow;
};

// A tile of rows and the tokens that some row of it sees.
struct Tile {
  int32_t first, packed, pos;  // as SeqWork's
  int32_t lo, hi, units;
};
template <int ROWS>
__device__ __forceinline__ Tile tile_of(const AttendArgs& a, const SeqWork& w, int32_t rtile) {
  const int32_t live = w.packed - rtile * ROWS < ROWS ? w.packed - rtile * ROWS : ROWS;
  const int32_t p0 = w.pos + fastdiv(rtile * ROWS, a.group), p1 = w.pos + fastdiv(rtile * ROWS + live - 1, a.group) + 1;
  Tile t;
  t.first = w.first;
  t.packed = w.packed;
  t.pos = w.pos;
  t.hi = p1 < w.hi ? (p1 < 0 ? 0 : p1) : w.hi;
  t.lo = first_tile(p0, a.window, kManyTokens, t.hi);
  t.units = t.hi > t.lo ? (t.hi - t.lo + kManyTokens - 1) / kManyTokens : 1;
  return t;
}

// The list: tiles of rows in the sequences' order.  plan[0] tiles, plan[1] units; then
// per tile the units before it, sequence and tile in the sequence; then the first tile of
// each sequence.
struct ManyTile {
  int64_t before;
  int32_t seq, rtile;
};
struct ManyPlan {
  int64_t* head;
  ManyTile* tiles;    // most + 1
  int32_t* first_of;  // seqs + 1
  int32_t most;
};

constexpr int kPlanThreads = 1024;

// Sum over the workgroup of one value a thread, and the sum of the threads before.
__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t* total) {
  __shared__ int64_t wsum[kPlanThreads / 64];
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
  for (int i = 0; i < kPlanThreads / 64; ++i) {
    before += i < wave ? wsum[i] : 0;
    all += wsum[i];
  }
  __syncthreads();
  *total = all;
  return before + inc - v;
}

template <int ROWS>
__global__ void __launch_bounds__(kPlanThreads) kv_attend_plan_kernel(AttendArgs a, ManyPlan p) {
  const int tid = threadIdx.x;
  const int32_t seqs = (int32_t)a.b.seqs;
  int64_t tiles = 0, sum;
  for (int32_t s0 = 0; s0 < seqs; s0 += kPlanThreads) {
    const int32_t s = s0 + tid;
    const int64_t n = s < seqs ? seq_work<ROWS>(a, s).rtiles : 0;
    const int64_t at = tiles + plan_scan(n, &sum);
    // A row_start that falls can ask for more tiles than the list holds: those are left out.
    if (s < seqs) p.first_of[s] = (int32_t)(at < p.most ? at : p.most);
    tiles += sum;
  }
  tiles = tiles < p.most ? tiles : p.most;
  if (tid == 0) p.first_of[seqs] = (int32_t)tiles;
  __threadfence_block();
  __syncthreads();
  int64_t units = 0;
  for (int32_t i0 = 0; i0 < (int32_t)tiles; i0 += kPlanThreads) {
    const int32_t i = i0 + tid;
    int32_t lo = 0, hi = seqs;  // the last sequence whose first tile is at or before i
    int64_t n = 0;
    if (i < (int32_t)tiles) {
      while (hi - lo > 1) {
        const int32_t mid = lo + (hi - lo) / 2;
        if (p.first_of[mid] <= i) lo = mid;
        else hi = mid;
      }
      n = tile_of<ROWS>(a, seq_work<ROWS>(a, lo), i - p.first_of[lo]).units;
    }
    const int64_t before = units + plan_scan(n, &sum);
    if (i < (int32_t)tiles) p.tiles[i] = ManyTile{before, lo, i - p.first_of[lo]};
    units += sum;
  }
  if (tid == 0) {
    p.tiles[tiles] = ManyTile{units, seqs, 0};
    p.head[0] = tiles;
    p.head[1] = units;
  }
}

// x, but not for the compiler: what is computed from it is not kept in registers across the loop over tokens.
__device__ __forceinline__ int here_only(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The end of a phase: the workgroup's barrier, met from different places in the code.
__device__ __forceinline__ void phase_end() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
  __builtin_amdgcn_sched_barrier(0);
}

template <bool MX>
__device__ __forceinline__ f32x16_t mfma32(const u32x4v_t& a, const u32x4v_t& b, const f32x16_t& c) {
  if constexpr (MX)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

// Outputs of a part, as a wavefront holds them: piece (32 dims d, 4 rows of 4 m) of every lane together; then
// maximum and sum of each row.
template <int NS>
constexpr int64_t many_part_floats() {
  return (int64_t)Many<NS>::kRows * (Many<NS>::kD + 2);
}

template <bool MX, bool BF16, int NS>
__global__ void __launch_bounds__(Many<NS>::kThreads) kv_attend_many_kernel(AttendArgs a, ManyPlan p) {
  constexpr int kTerms = AttendTerms<MX, BF16, true>::kQuery, kWeightTerms = AttendTerms<MX, BF16, true>::kWeight;
  using M = Many<NS>;
  using SB = ScaleBytes<MX, NS>;
  constexpr int kD = M::kD, kRows = M::kRows, kItems = M::kItems, kSteps = 2 * NS;
  constexpr int kAlign = NS % 4 == 0 ? 16 : (NS % 2 == 0 ? 8 : 4);
  __shared__ __attribute__((aligned(16))) char lds[2 * M::kBuffer];
  __shared__ uint32_t there_of[2][4];      // 16 tokens each: which are in the cache
  __shared__ uint32_t nan_of[2][4];        // 16 tokens each: whether a value's block is NaN
  __shared__ uint32_t bad_of[2][256];      // the scale words of those
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int ltok = (tid & 255) >> 2, lquarter = tid & 3;

  const int64_t units = p.head[1], total = units * a.c.heads;
  const int nwg = sharing(a, total);
  const int per_xcd = (a.nwg + 7) / 8;
  const int wg = ((int)blockIdx.x & 7) * per_xcd + ((int)blockIdx.x >> 3);
  if (wg >= nwg) return;
  int64_t cur = div_i64(wg * total, nwg);
  const int64_t end = div_i64((wg + 1) * total, nwg);
  int32_t head = (int32_t)div_i64(cur, units);
  int32_t item = 0;
  {
    // The last tile of rows at or before the first unit, 64 at a time.
    const int64_t at = cur - head * units;
    int32_t hi = (int32_t)p.head[0];
    while (hi - item > 1) {
      const int32_t step = (hi - item + 63) / 64, i = item + lane * step;
      const int n = __popcll(__ballot(i < hi && p.tiles[i].before <= at));
      item += (n > 0 ? n - 1 : 0) * step;
      hi = item + step < hi ? item + step : hi;
    }
    item = __builtin_amdgcn_readfirstlane(item);
  }
  const float ts_k = MX ? 1.0f : *a.c.tscale[0], ts_v = MX ? 1.0f : *a.c.tscale[1];
  const uint32_t heads = (uint32_t)a.c.heads, page_rows = (uint32_t)(a.c.block_size * a.c.heads);
  const uint32_t pages = a.c.num_blocks < INT32_MAX ? (uint32_t)a.c.num_blocks : (uint32_t)INT32_MAX;

  while (cur < end) {
    const ManyTile mt = p.tiles[item];
    const int32_t seq = __builtin_amdgcn_readfirstlane(mt.seq), rtile = __builtin_amdgcn_readfirstlane(mt.rtile);
    const Tile w = tile_of<kRows>(a, seq_work<kRows>(a, seq), rtile);
    const int32_t u0 = (int32_t)(cur - head * units - mt.before);
    const int32_t n = (int32_t)(w.units - u0 < end - cur ? w.units - u0 : end - cur);
    const int32_t* table = a.b.block_table + (int64_t)seq * a.b.max_blocks;
    const int32_t tb0 = w.lo + u0 * kManyTokens, last = w.hi > 0 ? w.hi - 1 : 0;

    // This thread's quarter of a token: page id, cache row, codes.
    int32_t id, slot;
    bool inside, in_row, in;
    uint32_t row;
    uint32_t code[kItems][NS], sc[kItems];
    const auto find = [&](int32_t u) {
      int32_t t = tb0 + u * kManyTokens + ltok;
      inside = t < w.hi;
      t = inside ? t : last;
      const int32_t page = fastdiv(t, a.page);
      id = table[page];
      slot = t - page * a.page.d;
    };
    const auto load = [&]() {
      const bool paged = (uint32_t)id < pages;
      in_row = paged && inside;
      row = (paged ? (uint32_t)id : 0u) * page_rows + (uint32_t)slot * heads + (uint32_t)head;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int which = kItems == 2 ? i : wave >> 2;  // uniform: the pointers stay in scalar registers
        __builtin_memcpy(code[i],
                         __builtin_assume_aligned((which ? a.c.codes[1] : a.c.codes[0]) + (uint64_t)(row * 4 + lquarter) * (4 * NS), kAlign),
                         4 * NS);
        if constexpr (SB::kEven) sc[i] = SB::load((which ? a.c.scales[1] : a.c.scales[0]) + (uint64_t)(row * 4 + lquarter) * SB::kLoad);
        else sc[i] = SB::load((which ? a.c.scales[1] : a.c.scales[0]) + (uint64_t)row * SB::kRow + SB::base(lquarter));
      }
    };

    // Rows: row col of this wavefront is packed row rtile kRows + 32 wave + col.
    const int lane_q = here_only(lane);
    const int32_t pr0 = rtile * kRows + 32 * wave, pr = pr0 + (lane_q & 31);
    const bool live = pr < w.packed;
    const int32_t qi = live ? fastdiv(pr, a.group) : 0, qj = live ? pr - qi * a.g : 0;
    const int32_t pos = w.pos + qi;
    u32x4v_t q[kTerms][kSteps];
    const uint16_t* src = a.q + (int64_t)(w.first + qi) * a.q_row + (int64_t)(head * a.g + qj) * a.q_head + 8 * (lane_q >> 5);
    u32x4v_t raw[kSteps];
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
      raw[c] = live ? *reinterpret_cast<const u32x4v_t*>(src + 16 * c) : u32x4v_t{0u, 0u, 0u, 0u};
    find(0);
    typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t mags = {0, 0};  // magnitude bits order like the values; NaN and infinities on top
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        mags = __builtin_elementwise_max(mags, __builtin_bit_cast(u16x2_t, raw[c][e] & 0x7FFF7FFFu));
    uint32_t largest = mags[0] > mags[1] ? mags[0] : mags[1];
    largest = max(largest, (uint32_t)__shfl_xor((int)largest, 32, 64));
    const RowScale rs = row_scale(half_to_f32<BF16>(largest), a.scale, ts_k);
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = half_to_f32<BF16>(raw[c][e] & 0xFFFFu) * rs.mul, y = half_to_f32<BF16>(raw[c][e] >> 16) * rs.mul;
        q[0][c][e] = pack2<MX>(x, y);
        if constexpr (kTerms == 2) q[kTerms - 1][c][e] = pack2_rest<MX>(x, y, q[0][c][e]);
      }
    f32x16_t o[NS];
#pragma unroll
    for (int d = 0; d < NS; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;
    bool far = false;

    // Tokens that every row, of the workgroup's tile and of the wavefront's, sees, and the last that one of the
    // wavefront's sees.
    const auto pos_of = [&](int32_t packed_row) { return w.pos + fastdiv(packed_row, a.group); };
    const int32_t live_end = w.packed < (rtile + 1) * kRows ? w.packed : (rtile + 1) * kRows;
    const int32_t wave_end = live_end < pr0 + 32 ? live_end : pr0 + 32;
    const bool wave_live = pr0 < wave_end;
    const int32_t tile_pos = pos_of(rtile * kRows), tile_first = first_seen(pos_of(live_end - 1), a.window);
    const int32_t wave_pos = wave_live ? pos_of(pr0) : 0, wave_last = wave_live ? pos_of(wave_end - 1) : -1;
    const int32_t wave_first = wave_live ? first_seen(wave_last, a.window) : 0;
    const int32_t wave_low = wave_live ? first_seen(wave_pos, a.window) : 0;

    // Unit u's quarters into its buffer.
    const auto decode = [&](int32_t u) {
      const int b = u & 1;
      char* buf = lds + b * M::kBuffer;
      const int32_t tb = tb0 + u * kManyTokens;
      const bool apart = tb + kManyTokens - 1 > tile_pos || tb < tile_first;  // a row sees what another does not
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const bool value = kItems == 2 ? i == 1 : wave >= 4;
        if (!value) {
          uint64_t bits = __ballot(in) & 0x1111111111111111ull;  // one lane in four
          if (lane == 0) {
            bits = (bits | bits >> 3) & 0x0303030303030303ull;
            bits = (bits | bits >> 6) & 0x000F000F000F000Full;
            bits = (bits | bits >> 12) & 0x000000FF000000FFull;
            there_of[b][wave & 3] = ((uint32_t)bits | (uint32_t)(bits >> 24)) & 0xFFFFu;
          }
        } else {
          // Values of tokens that are not there count as 0; a NaN block that not every row sees is taken out and added
          // by the rows that see it (0 times NaN is not 0).
          bool nan = false;
          if (!in) {
#pragma unroll
            for (int c = 0; c < NS; ++c) code[i][c] = 0;
            sc[i] = 0;
          }
          if (apart) {
            const uint32_t bad = sc[i];
#pragma unroll
            for (int c = 0; c < NS; ++c) {
              const bool x = scale_nonfinite<MX>((bad >> (8 * SB::index(lquarter, c))) & 0xFFu);
              nan = nan || x;
              code[i][c] = x ? 0u : code[i][c];
            }
            nan = __any(nan);
            if (nan) {
              bad_of[b][tid & 255] = bad;
              sc[i] = drop_nan<MX>(bad);
            }
          }
          if (lane == 0) nan_of[b][wave & 3] = nan;
        }
        u32x4v_t f[NS];
        decode_quarter<MX, NS>(code[i], sc[i], lquarter, f);
        char* at = value ? buf + M::kValues + ltok * M::kValueRow : buf + ltok * M::kKeyRow;
        const int turn = value ? (ltok >> 2) & 3 : 0;
#pragma unroll
        for (int c = 0; c < NS; ++c) *reinterpret_cast<u32x4v_t*>(at + ((lquarter * NS + c) ^ turn) * 16) = f[c];
      }
    };

    // Whether some row of this wavefront sees a token of unit u.
    const auto needs = [&](int32_t u) {
      const int32_t tb = tb0 + u * kManyTokens;
      return tb <= wave_last && tb + kManyTokens > wave_low;
    };
    uint32_t th[2];     // of the unit whose scores are in s: its tokens that are in the cache
    uint32_t nan_any;  // whether NaN blocks were taken out of its values
    const auto seen = [&](int32_t tb, int t) {
      return ((th[t >> 5] >> (t & 31)) & 1u) && sees(pos, a.window, tb + t);
    };
    f32x16_t s[2];  // register e of s[t] is token 32 t + 8 (e / 4) + 4 half + e % 4
    u32x4v_t pf[kWeightTerms][4];
    const auto weights = [&](int32_t u) {
      const int b = u & 1;
      const int32_t tb = tb0 + u * kManyTokens;
      th[0] = there_of[b][0] | there_of[b][1] << 16;
      th[1] = there_of[b][2] | there_of[b][3] << 16;
      nan_any = __builtin_amdgcn_readfirstlane(nan_of[b][0] | nan_of[b][1] | nan_of[b][2] | nan_of[b][3]);
      const bool masked = (th[0] & th[1]) != 0xFFFFFFFFu || tb + kManyTokens - 1 > wave_pos || tb < wave_first;
      float top = -__builtin_inff();
      if (masked) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t bits = (th[t] & seen_bits(pos, a.window, tb + 32 * t)) >> (4 * half);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            s[t][e] = bits & (1u << (8 * (e / 4) + e % 4)) ? s[t][e] : -__builtin_inff();
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[t][e]);
      top *= rs.factor;  // positive, or NaN
      if (__any(top > m + (far ? 0.0f : kSlack))) {
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m, top);
        const float shrink = next == m ? 1.0f : __builtin_amdgcn_exp2f(m - next);
        m = next;
        l *= shrink;
#pragma unroll
        for (int d = 0; d < NS; ++d) o[d] *= shrink;
        far = far || __any(is_far(next));
      }
      float mm = m == -__builtin_inff() ? 0.0f : m - weight_bias<MX>();
      if (__builtin_expect(far, 0)) {
        // The differences take the scores' place, divided by the factor that the loop below multiplies with.
        const float inv = 1.0f / rs.factor;
        mm = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[t][e] = (below(s[t][e] * rs.factor, m) + weight_bias<MX>()) * inv;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][e], rs.factor, -mm));
          float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][e + 1], rs.factor, -mm));
          l += p0 + p1;
          const uint32_t x = pack2<MX>(p0, p1);
          pf[0][2 * t + e / 8][e / 2 % 4] = x;
          if constexpr (kWeightTerms == 2) pf[kWeightTerms - 1][2 * t + e / 8][e / 2 % 4] = pack2_rest<MX>(p0, p1, x);
        }
    };
    // Scores of unit u, or outputs of unit v, or both: products whose fragments are read kAhead steps before their use
    // (the order is pinned, since the compiler would wait for nearly every read; with 128 elements and two terms 6 spill
    // more: 2048 rows behind 6144, MXFP4 and FP16, 650 us instead of 614).  A value's fragment: lane 16 j + i of a
    // transposing read gets column i of tokens 4 half .. + 3 (and 8 on) of a step, columns 32 d + 16 (j % 2) on, and
    // points at row i / 4, columns 4 (i % 4) of them.
    const auto matrix = [&](auto with_scores, auto with_outputs, int32_t u, int32_t v) {
      constexpr int kFirst = decltype(with_scores)::value ? 0 : 4 * NS;
      constexpr int kEnd = decltype(with_outputs)::value ? 8 * NS : 4 * NS, kAhead = NS == 4 && kWeightTerms == 2 ? 4 : 6;
      typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
      typedef __attribute__((address_space(3))) char lds_char;
      const char* kbuf = lds + (u & 1) * M::kBuffer + col * M::kKeyRow + 16 * half;
      const char* vrow = lds + (v & 1) * M::kBuffer + M::kValues + (4 * half + ((lane & 15) >> 2)) * M::kValueRow +
                         (lane & 1) * 8;
      const int piece = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
      const char* vbuf = vrow + (piece ^ half) * 16;                               // tokens 4 half .. of 16
      const char* vbuf8 = vrow + 8 * M::kValueRow + (piece ^ (half + 2)) * 16;  // 8 + 4 half ..
      u32x4v_t f[kAhead];
      const auto fetch = [&](int i) {
        if (i < 4 * NS) {
          f[i % kAhead] = *reinterpret_cast<const u32x4v_t*>(kbuf + 32 * (i & 1) * M::kKeyRow + 32 * (i >> 1));
        } else {
          const int at = 16 * ((i - 4 * NS) / NS) * M::kValueRow + 64 * ((i - 4 * NS) % NS);
          const i16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(lds_char*)(vbuf + at));
          const i16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(lds_char*)(vbuf8 + at));
          f[i % kAhead] = __builtin_bit_cast(u32x4v_t, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
        }
      };
      if constexpr (kFirst == 0)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
      for (int i = kFirst; i < kFirst + kAhead; ++i) fetch(i);
#pragma unroll
      for (int i = kFirst; i < kEnd; ++i) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < (i < 4 * NS ? kTerms : kWeightTerms); ++x) {
          if (i < 4 * NS) s[i & 1] = mfma32<MX>(f[i % kAhead], q[x][i >> 1], s[i & 1]);
          else o[(i - 4 * NS) % NS] = mfma32<MX>(f[i % kAhead], pf[x][(i - 4 * NS) / NS], o[(i - 4 * NS) % NS]);
        }
        if (i + kAhead < kEnd) fetch(i + kAhead);
      }
    };
    // The NaN blocks of unit u that were taken out.
    const auto nans = [&](int32_t u) {
      const int b = u & 1;
      if (nan_any) {
#pragma unroll 1
        for (int t = 0; t < kManyTokens; ++t) {
          if (!nan_of[b][t >> 4]) continue;
          const uint32_t* words = &bad_of[b][4 * t];
          const bool sees = seen(tb0 + u * kManyTokens, t);
#pragma unroll
          for (int d = 0; d < NS; ++d)
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // 16 dims: registers 8 k ..
              const int piece = 4 * d + 2 * k;
              const uint32_t byte = (words[piece / NS] >> (8 * SB::index(piece / NS, piece % NS))) & 0xFFu;
              if (scale_nonfinite<MX>(byte))
#pragma unroll
                for (int e = 0; e < 8; ++e) o[d][8 * k + e] += sees ? __builtin_nanf("") : 0.0f;
            }
        }
      }
    };

    const auto advance = [&](int32_t u) {  // decodes unit u, loads u + 1
      in = in_row;
      decode(u);
      if (u + 1 < n) load();
      if (u + 2 < n) find(u + 2);
    };
    load();
    if (n > 1) find(1);
    advance(0);
    __syncthreads();
    if constexpr (kItems == 1) {
      // Two wavefronts a SIMD in opposite phases: while one keeps the matrix cores busy (scores of unit t, outputs of
      // t - 1), the other takes the weights of its unit and decodes (wavefronts 0-3 keys, 4-7 values).  Keys of unit u
      // are decoded after both have done the scores of u - 2, values after both have done the outputs of u - 2.
      // One loop for both, the second half a barrier behind.
      const bool ahead = wave < 4;
      constexpr std::true_type yes{};
      constexpr std::false_type no{};
      if (!ahead) phase_end();
      matrix(yes, no, 0, 0);
      phase_end();
      for (int32_t t = 0; t + 1 < n; ++t) {
        weights(t);
        advance(t + 1);
        phase_end();
        __builtin_amdgcn_s_setprio(1);
        matrix(yes, yes, t + 1, t);
        nans(t);
        __builtin_amdgcn_s_setprio(0);
        phase_end();
      }
      weights(n - 1);
      phase_end();
      matrix(no, yes, 0, n - 1);
      nans(n - 1);
      phase_end();
      if (ahead) phase_end();
    } else {
      for (int32_t t = 0; t < n; ++t) {
        if (t + 1 < n) advance(t + 1);
        if (needs(t)) {
          matrix(std::true_type{}, std::false_type{}, t, t);
          weights(t);
          matrix(std::false_type{}, std::true_type{}, t, t);
          nans(t);
        }
        __syncthreads();
      }
    }

    l += __shfl_xor(l, 32, 64);
    const bool whole = u0 == 0 && n == w.units;
    const int lane_now = here_only(lane), col_now = lane_now & 31, half_now = lane_now >> 5;
    if (whole) {
      const int32_t row_now = pr0 + col_now;
      if (row_now < w.packed) {
        const int32_t i = fastdiv(row_now, a.group), j = row_now - i * a.g;
        uint16_t* out = a.out + ((int64_t)(w.first + i) * a.q_heads + head * a.g + j) * kD + 4 * half_now;
#pragma unroll
        for (int d = 0; d < NS; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const f32x4_t v = {o[d][4 * k], o[d][4 * k + 1], o[d][4 * k + 2], o[d][4 * k + 3]};
            store_out4<BF16>(out + 32 * d + 8 * k, finish(v, l, ts_v));
          }
      }
    } else if (wave_live) {
      float* part = a.part + ((int64_t)wg * 2 + (u0 > 0 ? 0 : 1)) * many_part_floats<NS>();
#pragma unroll
      for (int d = 0; d < NS; ++d)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          reinterpret_cast<f32x4_t*>(part)[((wave * NS + d) * 4 + k) * 64 + lane_now] =
              f32x4_t{o[d][4 * k], o[d][4 * k + 1], o[d][4 * k + 2], o[d][4 * k + 3]};
      if (half_now == 0) reinterpret_cast<float2*>(part + kRows * kD)[32 * wave + col_now] = make_float2(m, l);
    }
    cur += n;
    if (u0 + n == w.units && ++item == (int32_t)p.head[0]) {
      item = 0;
      ++head;
    }
  }
}

// Joins the parts of a tile of rows: a workgroup takes a wavefront's 32 rows of it and a key/value head, a thread the
// pieces that a lane of that wavefront held, a quarter of them.
template <bool BF16, int NS>
__global__ void __launch_bounds__(256) kv_attend_many_join_kernel(AttendArgs a, ManyPlan p, const float* ts_p) {
  using M = Many<NS>;
  __shared__ float total_of[32], best[32];
  const int32_t item = blockIdx.x / M::kWaves, wave = blockIdx.x % M::kWaves, head = blockIdx.y;
  if (item >= (int32_t)p.head[0]) return;
  const int64_t units = p.head[1], total = units * a.c.heads;
  const int nwg = sharing(a, total);
  const ManyTile mt = p.tiles[item];
  const int64_t f0 = head * units + mt.before, f1 = head * units + p.tiles[item + 1].before;
  const int32_t w0 = (int32_t)div_i64((f0 + 1) * nwg - 1, total), w1 = (int32_t)div_i64(f1 * nwg - 1, total);
  if (w0 == w1) return;
  const SeqWork w = seq_work<M::kRows>(a, mt.seq);
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, quarter = tid >> 6;
  const int32_t pr = mt.rtile * M::kRows + 32 * wave + r;
  if (mt.rtile * M::kRows + 32 * wave >= w.packed) return;
  const float ts = ts_p ? *ts_p : 1.0f;
  const auto part_of = [&](int32_t x) { return a.part + ((int64_t)x * 2 + (x == w0 ? 1 : 0)) * many_part_floats<NS>(); };
  const auto stats_of = [&](int32_t x, int row) {
    return reinterpret_cast<const float2*>(part_of(x) + M::kRows * M::kD)[32 * wave + row];
  };
  // Maximum and sum of every row: eight threads a row, each every eighth part.
  const int row = tid >> 3, lead = tid & 7;
  float top = -__builtin_inff();
  for (int32_t x = w0 + lead; x <= w1; x += 8) top = fmaxf(top, stats_of(x, row).x);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  const float mm_row = top == -__builtin_inff() ? 0.0f : top;
  float sum = 0.0f;
  for (int32_t x = w0 + lead; x <= w1; x += 8) {
    const float2 ml = stats_of(x, row);
    sum += __builtin_amdgcn_exp2f(ml.x - mm_row) * ml.y;
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor(sum, d, 64);
  if (lead == 0) {
    best[row] = mm_row;
    total_of[row] = sum;
  }
  __syncthreads();
  const float mm = best[r];
  f32x4_t acc[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (int32_t x = w0; x <= w1; ++x) {
    const float f = __builtin_amdgcn_exp2f(stats_of(x, r).x - mm);
#pragma unroll
    for (int i = 0; i < NS; ++i)
      acc[i] += reinterpret_cast<const f32x4_t*>(part_of(x))[(wave * 4 * NS + quarter * NS + i) * 64 + lane] * f;
  }
  if (pr >= w.packed) return;
  const int32_t qi = fastdiv(pr, a.group), qj = pr - qi * a.g;
  uint16_t* out = a.out + ((int64_t)(w.first + qi) * a.q_heads + head * a.g + qj) * M::kD + 4 * (lane >> 5);
#pragma unroll
  for (int i = 0; i < NS; ++i) store_out4<BF16>(out + 8 * (quarter * NS + i), finish(acc[i], total_of[r], ts));
}

int64_t many_tiles(int64_t rows, int64_t g, int64_t seqs, int64_t tile) {
  const int64_t n = rows * g / tile + seqs + 1;
  return n < INT32_MAX ? n : INT32_MAX;
}

template <int NS>
void launch_many(AttendArgs a, bool bf16, void* workspace, hipStream_t s) {
  using M = Many<NS>;
  ManyPlan p;
  p.most = (int32_t)many_tiles(a.b.rows, a.g, a.b.seqs, M::kRows);
  a.part = static_cast<float*>(workspace);
  p.head = reinterpret_cast<int64_t*>(a.part + (int64_t)a.nwg * 2 * many_part_floats<NS>());
  p.tiles = reinterpret_cast<ManyTile*>(p.head + 2);
  p.first_of = reinterpret_cast<int32_t*>(p.tiles + p.most + 1);
  kv_attend_plan_kernel<M::kRows><<<1, kPlanThreads, 0, s>>>(a, p);
  const dim3 grid((unsigned)((a.nwg + 7) / 8 * 8)), join((unsigned)(p.most * M::kWaves), (unsigned)a.c.heads);
  const float* ts = a.c.mx ? nullptr : a.c.tscale[1];
  const auto go = [&](auto mx, auto bf) {
    kv_attend_many_kernel<decltype(mx)::value, decltype(bf)::value, NS><<<grid, M::kThreads, 0, s>>>(a, p);
    kv_attend_many_join_kernel<decltype(bf)::value, NS><<<join, 256, 0, s>>>(a, p, ts);
  };
  if (a.c.mx) {
    if (bf16) go(std::true_type{}, std::true_type{});
    else go(std::true_type{}, std::false_type{});
  } else {
    if (bf16) go(std::false_type{}, std::true_type{});
    else go(std::false_type{}, std::false_type{});
  }
}

template <int NS>
int64_t many_bytes(int64_t g, int64_t rows, int64_t seqs) {
  using M = Many<NS>;
  const int64_t most = many_tiles(rows, g, seqs, M::kRows);
  return (4 * kManyWorkgroups * 2 * many_part_floats<NS>() + 16 + (most + 1) * (int64_t)sizeof(ManyTile) +
          (seqs + 1) * 4 + 15) / 16 * 16;
}

}  // namespace

int64_t kv_attend_many_workspace_bytes(int64_t head_dim, int64_t g, int64_t rows, int64_t seqs) {
  switch (head_dim / 32) {
    case 2: return many_bytes<2>(g, rows, seqs);
    case 3: return many_bytes<3>(g, rows, seqs);
    case 4: return many_bytes<4>(g, rows, seqs);
    case 6: return many_bytes<6>(g, rows, seqs);
    default: return many_bytes<8>(g, rows, seqs);
  }
}

void launch_kv_attend_many(const AttendArgs& args, bool bf16, void* workspace, hipStream_t s) {
  AttendArgs a = args;
  a.nwg = kManyWorkgroups;
  a.unit = make_fastdiv(kManyTokens);
  a.least = 1;
  switch (a.c.head_dim / 32) {
    case 2: return launch_many<2>(a, bf16, workspace, s);
    case 3: return launch_many<3>(a, bf16, workspace, s);
    case 4: return launch_many<4>(a, bf16, workspace, s);
    case 6: return launch_many<6>(a, bf16, workspace, s);
    default: return launch_many<8>(a, bf16, workspace, s);
  }
}

}  // namespace nvfp4
