// Attention over a paged FP4 cache for few rows a sequence (decoding, a few drafted
// tokens): bound by reading the cache.
//
// Every workgroup takes an equal, consecutive share of all units (a unit: 32 tokens of
// one tile of rows of one sequence, for hw heads), found from the lengths on the device,
// so that long and short sequences mix without idle CUs and the host needs no length.
// A share that ends inside a sequence leaves partial results, which
// kv_attend_join_kernel joins.  A wavefront takes one key/value head and every tw-th unit
// of the share: the heads of a group share the lines of codes and scales.
//
// A tile: the scores as S^T = K Q^T, tokens by rows.  A lane holds a quarter of a token's
// key as it lies in memory (16 bytes of codes at 128 elements), which is a fragment of K
// if the query's elements are taken in the same order.  The output is O^T = V^T P^T: the
// scores' layout is that of P^T's fragments, if V's tokens are taken in that order;
// values go through LDS in 16 bits, where transposing reads (ds_read_b64_tr_b16) pick
// up 4 tokens of a column.  A lane then holds scores, statistics and outputs of one row
// (lane % 16), and the maximum is exchanged only where it has grown by kSlack.
//
// Measured (40 query heads on 8 of 128; medians in a trace): 16 single rows of up to 8192
// tokens (85 MB of NVFP4) 29.9 us and the join 5.5, 2.8 TB/s over the kernel (a plain read
// reaches 7.1): beside the loop over units stand finding the share, the first loads and
// joining the slices.  One row of 131072 tokens (143 MB of MXFP4, FP16 outputs: twice the
// score products) 35.7 and 7.0 us; one of 1000 tokens 10.5 and 4.7.
#include <type_traits>

#include "kv_attend.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace {

constexpr int kFewTokens = 32;

// One workgroup a CU, of 12 wavefronts where 168 registers do (16 would spill, and what a wavefront does once, some 800
// instructions, counts for each), else 8.  With the join, 12 and 8: 16 streams of up to 8192 tokens 35.9 and 36.6 us, one
// of 131072 43.9 and 46.0, one of 1000 14.9 and 13.4.  ns: head dimension / 32, rt: 16-row tiles.
constexpr int few_waves(int ns, int rt) { return ns == 8 ? 6 : (ns * rt <= 4 ? 12 : 8); }
// Heads of a workgroup, at most.  4: lines are shared (16 streams of up to 8192 tokens with the join 35.9 us, with 2
// 38.4); with 32 rows 2, for smaller parts (8 x 4 rows of 32 heads on 4, window 4096: 36.9 us, with 4 39.4).
constexpr int few_heads(int ns, int rt) { return ns == 8 || rt == 2 ? 2 : 4; }

// Sizes by head dimension, rows and terms.
template <int NS, int RT, int TERMS>
struct Few {
  static constexpr int kD = 32 * NS, kRows = 16 * RT;
  static constexpr int kWaves = few_waves(NS, RT), kHeads = few_heads(NS, RT);
  static constexpr bool kQInLds = NS * RT * TERMS > 4;       // queries: more than 16 registers
  // LDS: 32 tokens' values a wavefront, rows 32 bytes longer than the values, so that 8 rows start in different banks, and of
  // tokens 8-15 every two 16-byte pieces change places, so that a write's 16 rows use all of them;
  // the queries; at the end instead a wavefront's 16 rows of outputs with their maximum and sum.
  static constexpr int kRow = 2 * kD + 32;
  static constexpr int kValues = kFewTokens * kRow;
  static constexpr int kQ = kQInLds ? RT * TERMS * NS * 1024 : 0;
  static constexpr int kOut = kD + 4;  // floats of an output row
  static constexpr int kStats = 16 * kOut * 4;
  static constexpr int kEnd = kStats + 128;
  static constexpr int kLoop = kWaves * kValues + kHeads * kQ;
  static constexpr int kLds = kLoop > kWaves * kEnd ? kLoop : kWaves * kEnd;
};

// Sum over the workgroup of one value a thread, and the sum of the threads before.
template <int WAVES>
__device__ __forceinline__ int64_t few_scan(int64_t v, int64_t* total) {
  __shared__ int64_t wsum[WAVES];
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
  for (int i = 0; i < WAVES; ++i) {
    before += i < wave ? wsum[i] : 0;
    all += wsum[i];
  }
  __syncthreads();
  *total = all;
  return before + inc - v;
}

template <bool MX, bool BF16, int NS, int RT>
__global__ void __launch_bounds__((64 * Few<NS, RT, AttendTerms<MX, BF16, false>::kQuery>::kWaves))
    kv_attend_few_kernel(AttendArgs a) {
  constexpr int kTerms = AttendTerms<MX, BF16, false>::kQuery, kWeightTerms = AttendTerms<MX, BF16, false>::kWeight;
  using F = Few<NS, RT, kTerms>;
  using SB = ScaleBytes<MX, NS>;
  constexpr int kWaves = F::kWaves, kThreads = 64 * kWaves, kD = F::kD, kRows = F::kRows;
  constexpr int kAlign = NS % 4 == 0 ? 16 : (NS % 2 == 0 ? 8 : 4);  // of a quarter's codes
  __shared__ __attribute__((aligned(16))) char lds[F::kLds];
  __shared__ int64_t plan[4];  // first sequence, unit in it, first unit, end
  __shared__ SeqWork first_work;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quarter = lane >> 4;    // row and quarter of its elements, in the products
  const int ltok = lane >> 2, lquarter = lane & 3;  // token and quarter of its row, in the loads
  const int turn = (4 * col + quarter) * 4;         // the lane that loaded what this one multiplies
  const int wg = (int)blockIdx.x / a.hgroups, hg = (int)blockIdx.x - wg * a.hgroups;
  const int slice = wave / a.hw, hh = wave - slice * a.hw, head = hg * a.hw + hh;
  const bool active = slice < a.tw && head < (int)a.c.heads;

  const float ts_k = MX ? 1.0f : *a.c.tscale[0], ts_v = MX ? 1.0f : *a.c.tscale[1];

  // This workgroup's units: found by the first wavefront where 64 sequences are all there are (the others would only
  // take issue slots from it), else by all.
  if ((int32_t)a.b.seqs <= 64) {
    if (wave == 0) {
      int64_t u = 0;
      SeqWork w;
      if (lane < (int32_t)a.b.seqs) {
        w = seq_work<kRows>(a, lane);
        u = (int64_t)w.rtiles * w.ttiles;
      }
      int64_t inc = u;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int64_t up = __shfl_up(inc, d, 64);
        if (lane >= d) inc += up;
      }
      const int64_t pre = inc - u, total = __shfl(inc, 63, 64);
      if (blockIdx.x == 0 && lane < (int32_t)a.b.seqs) a.prefix[lane] = pre;
      if (blockIdx.x == 0 && lane == 0) a.prefix[a.b.seqs] = total;
      const int nwg = sharing(a, total);
      if (lane == 0) plan[2] = plan[3] = 0;
      if (wg < nwg) {
        const int64_t cur = div_i64(wg * total, nwg), end = div_i64((wg + 1) * total, nwg);
        if (pre <= cur && cur < pre + u) {
          first_work = w;
          plan[0] = lane;
          plan[1] = cur - pre;
          plan[2] = cur;
          plan[3] = end;
        }
      }
    }
  } else {
    int64_t total = 0;
    for (int32_t s0 = 0; s0 < (int32_t)a.b.seqs; s0 += kThreads) {
      const int32_t s = s0 + tid;
      int64_t u = 0;
      if (s < (int32_t)a.b.seqs) {
        const SeqWork w = seq_work<kRows>(a, s);
        u = (int64_t)w.rtiles * w.ttiles;
      }
      int64_t chunk;
      const int64_t pre = total + few_scan<kWaves>(u, &chunk);
      total += chunk;
      if (blockIdx.x == 0 && s < (int32_t)a.b.seqs) a.prefix[s] = pre;
    }
    if (blockIdx.x == 0 && tid == 0) a.prefix[a.b.seqs] = total;
    const int nwg = sharing(a, total);
    if (wg >= nwg) return;
    const int64_t cur = div_i64(wg * total, nwg), end = div_i64((wg + 1) * total, nwg);
    int64_t sum = 0;
    for (int32_t s0 = 0; s0 < (int32_t)a.b.seqs && sum <= cur; s0 += kThreads) {
      const int32_t s = s0 + tid;
      int64_t u = 0;
      SeqWork w;
      if (s < (int32_t)a.b.seqs) {
        w = seq_work<kRows>(a, s);
        u = (int64_t)w.rtiles * w.ttiles;
      }
      int64_t chunk;
      const int64_t pre = sum + few_scan<kWaves>(u, &chunk);
      sum += chunk;
      if (pre <= cur && cur < pre + u) {
        first_work = w;
        plan[0] = s;
        plan[1] = cur - pre;
        plan[2] = cur;
        plan[3] = end;
      }
    }
  }
  __syncthreads();
  int32_t seq = __builtin_amdgcn_readfirstlane((int32_t)plan[0]);
  int64_t off = plan[1], cur = plan[2];
  const int64_t end = plan[3];

  char* vbuf = lds + wave * F::kValues;
  char* qbuf = lds + kWaves * F::kValues + hh * F::kQ + lane * 16;
  const uint32_t head_at = head < (int)a.c.heads ? head : 0, heads = (uint32_t)a.c.heads;
  const uint32_t page_rows = (uint32_t)(a.c.block_size * a.c.heads);
  const uint32_t pages = a.c.num_blocks < INT32_MAX ? (uint32_t)a.c.num_blocks : (uint32_t)INT32_MAX;

  SeqWork w;
  {
    const int32_t* f = reinterpret_cast<const int32_t*>(&first_work);
    int32_t* t = reinterpret_cast<int32_t*>(&w);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(SeqWork) / 4); ++i) t[i] = __builtin_amdgcn_readfirstlane(f[i]);
  }
  while (cur < end) {
    const int32_t rtile = off < w.ttiles ? 0 : (int32_t)div_i64(off, w.ttiles), t0 = (int32_t)(off - (int64_t)rtile * w.ttiles);
    const int32_t n = (int32_t)(w.ttiles - t0 < end - cur ? w.ttiles - t0 : end - cur);
    const int32_t* table = a.b.block_table + (int64_t)seq * a.b.max_blocks;

    // The rows of this tile: row col of sub-tile rt is packed row i g + j, query head head g + j of row i.
    u32x4v_t raw[RT][NS];
    int32_t pos[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int32_t pr = rtile * kRows + 16 * rt + col;
      const bool live = active && pr < w.packed;
      const int32_t i = live ? fastdiv(pr, a.group) : 0, j = live ? pr - i * a.g : 0;
      pos[rt] = w.pos + i;
      const uint16_t* src = a.q + (int64_t)(w.first + i) * a.q_row + (int64_t)(head_at * a.g + j) * a.q_head + quarter * 8 * NS;
#pragma unroll
      for (int c = 0; c < NS; ++c)
        raw[rt][c] = live ? *reinterpret_cast<const u32x4v_t*>(src + 8 * c) : u32x4v_t{0u, 0u, 0u, 0u};
    }

    // A tile of 32 tokens: this wavefront's token col of its half h is token tb + 16 h + col.  First the page ids are
    // loaded, a tile ahead of the codes, which come a tile ahead of their use.  Tokens behind the last one read its row
    // (one row for all of them would be a hot line).
    const int32_t tb0 = w.lo + (t0 + slice) * kFewTokens, step = a.tw * kFewTokens;
    const int32_t mine = slice < n && active ? (n - slice + a.tw - 1) / a.tw : 0;  // this slice's tiles: every tw-th
    const int32_t last = w.hi > 0 ? w.hi - 1 : 0;
    uint32_t kc[2][NS], vc[2][NS], ks[2], vs[2];
    uint32_t here = 0;  // bit 16 h + t: token t of half h is in the cache
    int32_t id[2], slot[2];
    bool inside[2];
    uint32_t row[2];
    const auto find = [&](int32_t tile) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int32_t t = tb0 + tile * step + 16 * h + ltok;
        inside[h] = t < w.hi;
        t = inside[h] ? t : last;
        const int32_t page = fastdiv(t, a.page);
        id[h] = table[page];
        slot[h] = t - page * a.page.d;
      }
    };
    const auto place = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool paged = (uint32_t)id[h] < pages;
        row[h] = (paged ? (uint32_t)id[h] : 0u) * page_rows + (uint32_t)slot[h] * heads + head_at;
        // One lane in four: bits 0, 4, .. of the ballot, closed up.
        uint64_t x = __ballot(paged && inside[h]) & 0x1111111111111111ull;
        x = (x | x >> 3) & 0x0303030303030303ull;
        x = (x | x >> 6) & 0x000F000F000F000Full;
        x = (x | x >> 12) & 0x000000FF000000FFull;
        const uint32_t bits = ((uint32_t)x | (uint32_t)(x >> 24)) & 0xFFFFu;
        here = h == 0 ? bits : here | bits << 16;
      }
    };
    const auto load = [&](int which, int h, uint32_t (&c)[NS], uint32_t& sc) {
      __builtin_memcpy(c, __builtin_assume_aligned(a.c.codes[which] + (uint64_t)(row[h] * 4 + lquarter) * (4 * NS), kAlign),
                       4 * NS);
      if constexpr (SB::kEven) sc = SB::load(a.c.scales[which] + (uint64_t)(row[h] * 4 + lquarter) * SB::kLoad);
      else sc = SB::load(a.c.scales[which] + (uint64_t)row[h] * SB::kRow + SB::base(lquarter));
    };
    if (mine > 0) {
      find(0);
      place();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        load(0, h, kc[h], ks[h]);
        load(1, h, vc[h], vs[h]);
      }
      if (mine > 1) find(1);
    }

    u32x4v_t q[RT][kTerms][F::kQInLds ? 1 : NS];
    f32x4_t o[RT][2 * NS];
    float factor[RT], m[RT], l[RT];
    bool far = false;
    if (F::kQInLds) __syncthreads();  // the buffers' last use, by other wavefronts
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
      u16x2_t mags = {0, 0};  // magnitude bits order like the values; NaN and infinities on top
#pragma unroll
      for (int c = 0; c < NS; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mags = __builtin_elementwise_max(mags, __builtin_bit_cast(u16x2_t, raw[rt][c][e] & 0x7FFF7FFFu));
      uint32_t largest = mags[0] > mags[1] ? mags[0] : mags[1];
      largest = max(largest, (uint32_t)__shfl_xor((int)largest, 16, 64));
      largest = max(largest, (uint32_t)__shfl_xor((int)largest, 32, 64));
      const RowScale rs = row_scale(half_to_f32<BF16>(largest), a.scale, ts_k);
      factor[rt] = rs.factor;
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        u32x4v_t t[kTerms];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = half_to_f32<BF16>(raw[rt][c][e] & 0xFFFFu) * rs.mul, y = half_to_f32<BF16>(raw[rt][c][e] >> 16) * rs.mul;
          t[0][e] = pack2<MX>(x, y);
          if constexpr (kTerms == 2) t[kTerms - 1][e] = pack2_rest<MX>(x, y, t[0][e]);
        }
#pragma unroll
        for (int x = 0; x < kTerms; ++x) {
          if constexpr (!F::kQInLds) q[rt][x][c] = t[x];
          else if (slice == 0) *reinterpret_cast<u32x4v_t*>(qbuf + ((rt * kTerms + x) * NS + c) * 1024) = t[x];
        }
      }
#pragma unroll
      for (int d = 0; d < 2 * NS; ++d) o[rt][d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      m[rt] = -__builtin_inff();
      l[rt] = 0.0f;
    }
    if (F::kQInLds) __syncthreads();
    // Tokens all_first .. all_pos are seen by every row of the tile.
    const int32_t in_tile = w.packed - rtile * kRows < kRows ? w.packed - rtile * kRows : kRows;
    const int32_t all_pos = w.pos + fastdiv(rtile * kRows, a.group);
    const int32_t last_pos = w.pos + fastdiv(rtile * kRows + in_tile - 1, a.group);
    const int32_t all_first = first_seen(last_pos, a.window);

    // Loads that four neighbouring lanes make of one row reach the cache as one access, in the products' order they would
    // be four (16 streams of up to 8192 tokens: 28.8 instead of 31.8 us); a key's pieces change lanes afterwards.
    uint32_t kt[NS], kst;
    const auto take_k = [&](int h) {
#pragma unroll
      for (int c = 0; c < NS; ++c) kt[c] = (uint32_t)__builtin_amdgcn_ds_bpermute(turn, (int)kc[h][c]);
      kst = (uint32_t)__builtin_amdgcn_ds_bpermute(turn, (int)ks[h]);
    };
    // One tile; its registers take the next one's codes as soon as they are decoded.  Fragments are read from LDS kAhead
    // steps before their products (the order is pinned: the compiler would wait for nearly every read).
    constexpr int kAhead = 4;
    const auto compute = [&](int32_t tile) {
      const int32_t tb = tb0 + tile * step;
      const uint32_t there = here;
      const bool masked = there != 0xFFFFFFFFu || tb + 31 > all_pos || tb < all_first;
      const auto seen = [&](int rt, int t) {
        return ((there >> t) & 1u) && sees(pos[rt], a.window, tb + t);
      };
      const bool more = tile + 1 < mine;
      if (more) place();
      // Values into LDS first: they wait for nothing, and their latency passes under the scores.
      uint32_t bad[2] = {0, 0}, taken = 0;  // scale words of halves from which NaN blocks were taken out
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (masked) {
          // Values of tokens that are not there count as 0, whatever lies in the cache.
          const bool gone = !((there >> (16 * h + ltok)) & 1u);
#pragma unroll
          for (int c = 0; c < NS; ++c) vc[h][c] = gone ? 0u : vc[h][c];
          vs[h] = gone ? 0u : vs[h];
          // A NaN block is taken out (0 times NaN is not 0) and added below to the rows that see it.
          bad[h] = vs[h];
          bool any_bad = false;
#pragma unroll
          for (int c = 0; c < NS; ++c) {
            const bool nan = scale_nonfinite<MX>((bad[h] >> (8 * SB::index(lquarter, c))) & 0xFFu);
            any_bad = any_bad || nan;
            vc[h][c] = nan ? 0u : vc[h][c];
          }
          if (__any(any_bad)) {
            vs[h] = drop_nan<MX>(vs[h]);
            taken |= 1u << h;
          }
        }
        u32x4v_t vf[NS];
        decode_quarter<MX, NS>(vc[h], vs[h], lquarter, vf);
        if (more) load(1, h, vc[h], vs[h]);
        if (h == 1 && tile + 2 < mine) find(tile + 2);
#pragma unroll
        for (int c = 0; c < NS; ++c)
          *reinterpret_cast<u32x4v_t*>(vbuf + (16 * h + ltok) * F::kRow + ((lquarter * NS + c) ^ (ltok >> 3)) * 16) = vf[c];
      }
      f32x4_t sc[RT][2];
      if constexpr (F::kQInLds) {
        u32x4v_t kf[2][NS];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          take_k(h);
          decode_quarter<MX, NS>(kt, kst, quarter, kf[h]);
          if (more) load(0, h, kc[h], ks[h]);
        }
        constexpr int kSteps = RT * kTerms * NS;
        u32x4v_t qf[kAhead];
        const auto fetch_q = [&](int i) { qf[i % kAhead] = *reinterpret_cast<const u32x4v_t*>(qbuf + i * 1024); };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch_q(i);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sc[rt][0] = sc[rt][1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          const int rt = i / (kTerms * NS);
          sc[rt][0] = mfma16<MX>(kf[0][i % NS], qf[i % kAhead], sc[rt][0]);
          sc[rt][1] = mfma16<MX>(kf[1][i % NS], qf[i % kAhead], sc[rt][1]);
          if (i + kAhead < kSteps) fetch_q(i + kAhead);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4v_t kf[NS];
          take_k(h);
          decode_quarter<MX, NS>(kt, kst, quarter, kf);
          if (more) load(0, h, kc[h], ks[h]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            sc[rt][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int x = 0; x < kTerms; ++x)
#pragma unroll
              for (int c = 0; c < NS; ++c) sc[rt][h] = mfma16<MX>(kf[c], q[rt][x][c], sc[rt][h]);
          }
        }
      }
      u32x4v_t pf[RT][kWeightTerms];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = -__builtin_inff();
        uint32_t bits = 0;
        if (masked) bits = (there & seen_bits(pos[rt], a.window, tb)) >> (4 * quarter);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[rt][h][e] *= factor[rt];
            if (masked) sc[rt][h][e] = bits & (1u << (16 * h + e)) ? sc[rt][h][e] : -__builtin_inff();
            top = fmaxf(top, sc[rt][h][e]);
          }
        if (__any(top > m[rt] + (far ? 0.0f : kSlack))) {
          top = fmaxf(top, __shfl_xor(top, 16, 64));
          top = fmaxf(top, __shfl_xor(top, 32, 64));
          const float next = fmaxf(m[rt], top);
          const float shrink = next == m[rt] ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - next);
          m[rt] = next;
          l[rt] *= shrink;
#pragma unroll
          for (int d = 0; d < 2 * NS; ++d) o[rt][d] *= shrink;
          far = far || __any(is_far(next));
        }
        float mm = m[rt] == -__builtin_inff() ? 0.0f : m[rt] - weight_bias<MX>();
        if (__builtin_expect(far, 0)) {
          mm = -weight_bias<MX>();
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[rt][h][e] = below(sc[rt][h][e], m[rt]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = __builtin_amdgcn_exp2f(sc[rt][h][e] - mm);
            l[rt] += p[e];
          }
          pf[rt][0][2 * h] = pack2<MX>(p[0], p[1]);
          pf[rt][0][2 * h + 1] = pack2<MX>(p[2], p[3]);
          pf[rt][1][2 * h] = pack2_rest<MX>(p[0], p[1], pf[rt][0][2 * h]);
          pf[rt][1][2 * h + 1] = pack2_rest<MX>(p[2], p[3], pf[rt][0][2 * h + 1]);
        }
      }
      wave_lds_sync();
      // Tokens 4 quarter .. + 3 of both halves, columns 16 d ..: lane col of a quarter reads row col / 4.
      const char* at = vbuf + (4 * quarter + (col >> 2)) * F::kRow + ((((col >> 1) & 1) ^ (quarter >> 1)) * 16 + (col & 1) * 8);
      typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
      typedef __attribute__((address_space(3))) char lds_char;
      u32x4v_t vt[kAhead];
      const auto fetch_v = [&](int d) {
        const i16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(lds_char*)(at + 32 * d));
        const i16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(lds_char*)(at + 32 * d + 16 * F::kRow));
        vt[d % kAhead] = __builtin_bit_cast(u32x4v_t, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
      };
#pragma unroll
      for (int d = 0; d < kAhead; ++d) fetch_v(d);
#pragma unroll
      for (int d = 0; d < 2 * NS; ++d) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int z = 0; z < kWeightTerms; ++z) o[rt][d] = mfma16<MX>(vt[d % kAhead], pf[rt][z], o[rt][d]);
        if (d + kAhead < 2 * NS) fetch_v(d + kAhead);
      }
      if (taken) {
#pragma unroll 1
        for (int t = 0; t < kFewTokens; ++t) {
          if (!(taken & (t < 16 ? 1u : 2u))) continue;
          uint32_t q4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) q4[i] = (uint32_t)__builtin_amdgcn_readlane((int)(t < 16 ? bad[0] : bad[1]), 4 * (t & 15) + i);
#pragma unroll
          for (int d = 0; d < 2 * NS; ++d) {
            const uint32_t byte = (q4[2 * d / NS] >> (8 * SB::index(2 * d / NS, 2 * d % NS))) & 0xFFu;
            if (scale_nonfinite<MX>(byte))
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) o[rt][d] += seen(rt, t) ? __builtin_nanf("") : 0.0f;
          }
        }
      }
      wave_lds_sync();
    };
    {
      // A SIMD's wavefronts take turns in priority: left to themselves the oldest runs ahead, and the last runs alone in
      // the end.
      int turn_of = (wave >> 2) % 3;
      for (int32_t tile = 0; tile < mine; ++tile) {
        if (turn_of == 0) __builtin_amdgcn_s_setprio(0);
        else if (turn_of == 1) __builtin_amdgcn_s_setprio(1);
        else __builtin_amdgcn_s_setprio(2);
        turn_of = turn_of == 2 ? 0 : turn_of + 1;
        compute(tile);
      }
      __builtin_amdgcn_s_setprio(0);
    }

    // Join the slices; whole sequences' outputs are written, parts kept.
    const bool whole = t0 == 0 && n == w.ttiles;
    float* part = a.part + ((int64_t)blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * (a.hw * kRows * (kD + 2));
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] += __shfl_xor(l[rt], 16, 64);
      l[rt] += __shfl_xor(l[rt], 32, 64);
      __syncthreads();  // the values, the queries or the rows before are done with
      float* ob = reinterpret_cast<float*>(lds + wave * F::kEnd);
#pragma unroll
      for (int d = 0; d < 2 * NS; ++d)
        *reinterpret_cast<f32x4_t*>(ob + col * F::kOut + 16 * d + 4 * quarter) = o[rt][d];
      if (quarter == 0) reinterpret_cast<float2*>(ob + F::kStats / 4)[col] = make_float2(m[rt], l[rt]);
      __syncthreads();
      const int live = in_tile - 16 * rt < 16 ? in_tile - 16 * rt : 16;  // rows of this sub-tile
      const uint32_t per = live > 0 ? 65536u / (uint32_t)live + 1u : 0u;  // hr / live = hr per / 2^16 for hr < 128
      for (int i = tid; i < a.hw * live * (kD / 4); i += kThreads) {
        const int d4 = i % (kD / 4), hr = i / (kD / 4), h = (int)((uint32_t)hr * per >> 16), r = hr - h * live;
        const int32_t pr = rtile * kRows + 16 * rt + r;
        if (hg * a.hw + h >= (int)a.c.heads) continue;
        float top = -__builtin_inff();
        for (int k = 0; k < a.tw; ++k)
          top = fmaxf(top, reinterpret_cast<const float2*>(lds + (k * a.hw + h) * F::kEnd + F::kStats)[r].x);
        const float mm = top == -__builtin_inff() ? 0.0f : top;
        float sum = 0.0f;
        f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < a.tw; ++k) {
          const char* buf = lds + (k * a.hw + h) * F::kEnd;
          const float2 ml = reinterpret_cast<const float2*>(buf + F::kStats)[r];
          const float f = __builtin_amdgcn_exp2f(ml.x - mm);
          sum += ml.y * f;
          acc += *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(buf) + r * F::kOut + 4 * d4) * f;
        }
        if (whole) {
          const int32_t qi = fastdiv(pr, a.group), qj = pr - qi * a.g;
          store_out4<BF16>(a.out + ((int64_t)(w.first + qi) * a.q_heads + (hg * a.hw + h) * a.g + qj) * kD + 4 * d4,
                           finish(acc, sum, ts_v));
        } else {
          const int at = (h * RT + rt) * 16 + r;
          *reinterpret_cast<f32x4_t*>(part + (int64_t)at * kD + 4 * d4) = acc;
          if (d4 == 0) reinterpret_cast<float2*>(part + (int64_t)a.hw * kRows * kD)[at] = make_float2(top, sum);
        }
      }
    }
    __syncthreads();
    cur += n;
    off += n;
    if (off == (int64_t)w.rtiles * w.ttiles && cur < end) {
      off = 0;
      do w = seq_work<kRows>(a, ++seq);
      while (w.rtiles == 0);
    }
  }
}

// Joins the parts of one row and query head, if its tokens were shared: their maxima,
// sums and outputs.  A thread loads every part of its 4 elements that it adds at once;
// the order of the sums is fixed by the number of parts, the head dimension and THREADS,
// which launch_few takes by the rows, heads and width of the table: no atomics, so the same
// call gives the same bits.
constexpr int kJoinParts = 256;  // workgroups at most

template <bool BF16, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_attend_join_kernel(AttendArgs a, int head_dim, const float* ts_p) {
  __shared__ float weight[kJoinParts];
  __shared__ f32x4_t acc[THREADS];
  __shared__ float red[2][THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t r = blockIdx.x;
  const int qh = blockIdx.y;
  int64_t s = r;
  if (a.b.row_start) s = find_sequence(a.b, r, lane);
  if (s >= a.b.seqs) return;
  const int64_t total = a.prefix[a.b.seqs], first = a.prefix[s];
  const SeqWork w = seq_work<ROWS>(a, (int32_t)s);
  const int head = qh / a.g, hg = head / a.hw, hh = head - hg * a.hw;
  const int64_t pr = (r - w.first) * a.g + (qh - head * a.g);
  if (pr < 0 || pr >= w.packed) return;
  const int32_t nwg = sharing(a, total), rtile = (int32_t)pr / ROWS;
  const int64_t u0 = first + (int64_t)rtile * w.ttiles, u1 = u0 + w.ttiles;
  const int32_t w0 = (int32_t)div_i64((u0 + 1) * nwg - 1, total), w1 = (int32_t)div_i64(u1 * nwg - 1, total);
  const int parts = w1 - w0 + 1;
  if (parts <= 1) return;
  const int64_t slot = (int64_t)a.hw * ROWS * (head_dim + 2);
  const int64_t row = hh * ROWS + (pr - rtile * ROWS);
  const auto part_of = [&](int p) { return a.part + (((int64_t)(w0 + p) * a.hgroups + hg) * 2 + (p == 0 ? 1 : 0)) * slot; };
  float2 st = make_float2(-__builtin_inff(), 0.0f);
  if (tid < parts) st = reinterpret_cast<const float2*>(part_of(tid) + (int64_t)a.hw * ROWS * head_dim)[row];
  // The outputs' first loads do not wait for the statistics.
  constexpr int kAhead = 8;
  const int quads = head_dim / 4, groups = THREADS / quads, d4 = tid % quads, gi = tid / quads;
  const auto value_of = [&](int p) { return *reinterpret_cast<const f32x4_t*>(part_of(p) + row * head_dim + 4 * d4); };
  f32x4_t got[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int p = gi + i * groups;
    got[i] = gi < groups && p < parts ? value_of(p) : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  float top = st.x;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  if (lane == 0) red[0][tid >> 6] = top;
  __syncthreads();
  top = red[0][0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) top = fmaxf(top, red[0][i]);
  const float mm = top == -__builtin_inff() ? 0.0f : top;
  const float f = __builtin_amdgcn_exp2f(st.x - mm);
  if (tid < parts) weight[tid] = f;
  const float sum_mine = wave_sum(f * st.y);
  if (lane == 0) red[1][tid >> 6] = sum_mine;
  __syncthreads();
  f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (gi < groups) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int p = gi + i * groups;
      if (p < parts) x += got[i] * weight[p];
    }
    for (int p = gi + kAhead * groups; p < parts; p += groups) x += value_of(p) * weight[p];
  }
  acc[tid] = x;
  __syncthreads();
  if (gi == 0) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) sum += red[1][i];
    for (int i = 1; i < groups; ++i) x += acc[i * quads + d4];
    const float ts = ts_p ? *ts_p : 1.0f;
    store_out4<BF16>(a.out + (r * a.q_heads + qh) * head_dim + 4 * d4, finish(x, sum, ts));
  }
}

template <int RT>
void launch_few(AttendArgs a, bool bf16, hipStream_t s) {
  const dim3 grid((unsigned)(a.nwg * a.hgroups));
  const auto go = [&](auto mx, auto bf, auto ns) {
    constexpr bool kMx = decltype(mx)::value, kBf = decltype(bf)::value;
    constexpr int kNs = decltype(ns)::value;
    constexpr int kThreads = 64 * Few<kNs, RT, AttendTerms<kMx, kBf, false>::kQuery>::kWaves;
    if constexpr (RT == 1 || kNs <= 4) kv_attend_few_kernel<kMx, kBf, kNs, RT><<<grid, kThreads, 0, s>>>(a);
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
  const float* ts = a.c.mx ? nullptr : a.c.tscale[1];
  // 1024 threads take 256 parts of 128 elements at once; with a workgroup a CU and more, or sequences too short for many
  // parts, 256 threads start sooner (both kernels, 256 and 1024 threads: 16 rows of 40 heads 35.9 and 44.0 us, 1 row of
  // 1000 tokens 14.9 and 16.5, 1 row of 256 parts 45.2 and 43.9).
  const int dim32 = (int)a.c.head_dim;
  const auto join = [&](auto threads, auto bf) {
    constexpr int kThreads = decltype(threads)::value;
    kv_attend_join_kernel<decltype(bf)::value, 16 * RT, kThreads>
        <<<dim3((unsigned)a.b.rows, (unsigned)a.q_heads), kThreads, 0, s>>>(a, dim32, ts);
  };
  if (a.b.rows * a.q_heads < 256 && a.cap > 64 * kFewTokens) {
    if (bf16) join(std::integral_constant<int, 1024>{}, std::true_type{});
    else join(std::integral_constant<int, 1024>{}, std::false_type{});
  } else {
    if (bf16) join(std::integral_constant<int, 256>{}, std::true_type{});
    else join(std::integral_constant<int, 256>{}, std::false_type{});
  }
}

// Heads of a workgroup, its token slices, workgroups and 16-row tiles.
struct FewPlan {
  int hw, tw, hgroups, nwg, rt;
  int64_t part_floats;
};
FewPlan few_plan(int64_t heads, int64_t head_dim, int64_t q_heads, int64_t rows, int64_t seqs) {
  FewPlan p;
  p.rt = rows * (q_heads / heads) > 16 * seqs && head_dim <= 128 ? 2 : 1;
  const int ns = (int)(head_dim / 32);
  const int waves = few_waves(ns, p.rt), most = few_heads(ns, p.rt);
  const int64_t groups = (heads + most - 1) / most;
  p.hw = (int)((heads + groups - 1) / groups);
  p.hgroups = (int)((heads + p.hw - 1) / p.hw);
  p.tw = waves / p.hw;
  p.nwg = (256 + p.hgroups - 1) / p.hgroups;
  p.part_floats = (int64_t)p.nwg * p.hgroups * 2 * p.hw * 16 * p.rt * (head_dim + 2);
  return p;
}

}  // namespace

// Many rows or few, by the packed rows (rows times query heads of a key/value head) of a sequence on average: with 32 (8
// sequences of up to 16384 tokens, 4 rows each, 32 heads on 4) 37 us by the kernel for few and 44 by the one for many;
// with 235 (264 rows of 9 sequences, one a chunk, the others single tokens, 16 heads of 256 on 2) 69 by few, 53 by many;
// with 4092 (7161 rows of 7 prompts, 16 heads of 64 on 4) 403 by few, 94 by many.  Where they cross between 32 and 235 was
// not looked for.
static bool many_rows(int64_t g, int64_t rows, int64_t seqs) { return rows * g > 32 * seqs; }

int64_t kv_attend_workspace_bytes(int64_t heads, int64_t head_dim, int64_t q_heads, int64_t rows, int64_t seqs) {
  if (many_rows(q_heads / heads, rows, seqs)) return kv_attend_many_workspace_bytes(head_dim, q_heads / heads, rows, seqs);
  const FewPlan p = few_plan(heads, head_dim, q_heads, rows, seqs);
  return p.part_floats * 4 + (seqs + 2) / 2 * 16;
}

void launch_kv_attend(const KvCache& c, const KvBatch& b, bool bf16, const uint16_t* q, int64_t q_heads, int64_t q_row,
                      int64_t q_head, float scale, int64_t window, uint16_t* out, void* workspace, hipStream_t s) {
  AttendArgs a = {};
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
  if (many_rows(a.g, b.rows, b.seqs)) return launch_kv_attend_many(a, bf16, workspace, s);
  const FewPlan p = few_plan(c.heads, c.head_dim, q_heads, b.rows, b.seqs);
  a.unit = make_fastdiv(kFewTokens);
  a.least = p.tw;
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
