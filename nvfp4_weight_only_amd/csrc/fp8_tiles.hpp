// Index arithmetic and launch plans of the E4M3 GEMM (fp8_gemm.hip), apart from the
// kernel so that a program on the host runs the same code over every tile, wavefront,
// lane and chunk of a launch (tests/sanitize/fp8_tiles_driver.cpp).
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __HIPCC__
#define NVFP4_HD __host__ __device__ inline __attribute__((always_inline))
#else
#define NVFP4_HD inline
#endif

namespace nvfp4 {
namespace fp8_tiles {

constexpr int kChunk = 128;  // of K
// Tiles with two stages only: how many chunks ahead of the loads to LDS lines are
// brought into L2 (256 x 256 over 2048 x 16384 x 5120: 174 us without, 170 with;
// with three stages the lines come early enough, and the lines in flight are what
// is scarce: 64 x 5120 x 17408 30 us without, 38 with).
constexpr int kAhead = 2;

// ---------------------------------------------------------------------------
// Tiles.
// ---------------------------------------------------------------------------
// Workgroups go to the 8 XCDs round-robin by id.  An XCD's share of a slice, its
// ids in order, are consecutive tiles, m tiles first: a tile's rows of W are
// fetched into that XCD's L2 once (333 x 5000 x 17392, 60 tiles a slice: 74.6
// us with the tiles in the order of the ids, 69.8 so).
NVFP4_HD int tile_of_id(int id, int tiles) {
  const int xcd = id & 7, more = tiles & 7;
  return xcd * (tiles >> 3) + (xcd < more ? xcd : more) + (id >> 3);
}

// First chunk of a slice of K (slice = slices: past the last chunk).
NVFP4_HD int first_chunk(int kb, int slice, int slices) { return (int)((int64_t)kb * slice / slices); }

// Grouped: the first of the tiles in use that XCD `xcd` takes (xcd = 8: all of them).
NVFP4_HD int64_t first_of_xcd(int64_t used, int64_t xcd) { return used * xcd >> 3; }
// Each XCD has m_tiles places, tiles t0 .. t0 + tn - 1 in the first tn of them.  The
// places left over, left_places of them, write zero rows: place mt of an XCD every
// left_places-th row from row left_rank on.
NVFP4_HD int64_t left_places(int64_t used, int m_tiles) { return 8 * (int64_t)m_tiles - used; }
NVFP4_HD int64_t left_rank(int64_t xcd, int m_tiles, int64_t t0, int64_t tn, int mt) {
  return xcd * m_tiles - t0 + mt - tn;
}

// ---------------------------------------------------------------------------
// Loads.  Instruction j of wavefront w fills rows 8 (w + 8 j) .. + 7 of an operand's
// chunk in LDS, lane l row + l / 8, physical 16-byte piece l % 8: logical piece
// (l % 8) ^ (row % 8).
// ---------------------------------------------------------------------------
NVFP4_HD int lane_row(int lane) { return lane >> 3; }
NVFP4_HD int lane_piece(int lane) { return (lane & 7) ^ lane_row(lane); }
NVFP4_HD int load_row(int w, int j, int lane) { return 8 * (w + 8 * j) + lane_row(lane); }
// Where it writes, in bytes from the operand's start in the stage (lane 0).
NVFP4_HD uint32_t load_dst(int w, int j) { return (uint32_t)(1024 * w + 8192 * j); }
// Rows past the last one repeat it (their results are not stored).
NVFP4_HD int64_t row_or_last(int64_t r, int64_t rows) { return r < rows ? r : rows - 1; }
// Byte offset of the lane's piece of row r from the operand's base, in chunk 0.
NVFP4_HD uint32_t piece_offset(int64_t r, int64_t k, int piece) { return (uint32_t)(r * k + 16 * piece); }
// A last, short chunk: whether the lane's piece is past the end of K, and then how far
// behind the row's last one.
NVFP4_HD int tail_of(int64_t k) { return (int)(k & (kChunk - 1)); }
NVFP4_HD bool past_end(int ktail, int piece) { return ktail != 0 && 16 * piece >= ktail; }
NVFP4_HD uint32_t step_back(int ktail, int piece) {
  return past_end(ktail, piece) ? (uint32_t)(16 * piece - (ktail - 16)) : 0u;
}
// Byte offset of the scales of row (of X) or block of 128 rows (of W) r.
NVFP4_HD uint32_t scale_offset(int64_t r, int kb) { return (uint32_t)(4 * r * kb); }

// Lines brought into L2 ahead of their chunk's loads: the tiles that run on this XCD at
// the same time and share rows of W (m tiles, up to 8) or of X share this work.
struct Line {
  bool of_w;
  int row;  // of the tile
};
NVFP4_HD int share_of_w(int m_tiles) { return m_tiles < 8 ? m_tiles : 8; }
NVFP4_HD int share_of_x(int m_tiles, int n_tiles) {
  return 32 / share_of_w(m_tiles) < n_tiles ? 32 / share_of_w(m_tiles) : n_tiles;
}
NVFP4_HD Line line_ahead(int tn, int tm, int n_tiles, int m_tiles, int nt, int mt, int w, int lane) {
  const int share_w = share_of_w(m_tiles), share_x = share_of_x(m_tiles, n_tiles);
  const int lines_w = (tn + share_w - 1) / share_w, lines_x = (tm + share_x - 1) / share_x;
  const int i = 8 * lane + w;
  if (i < lines_w || i >= lines_w + lines_x) return Line{true, (i < lines_w ? i : 0) * share_w + mt % share_w};
  const int r = (i - lines_w) * share_x + nt % share_x;
  return Line{false, r < tm ? r : tm - 1};
}
NVFP4_HD int chunk_ahead(int c, int last) { return c + kAhead < last ? c + kAhead : last; }

// ---------------------------------------------------------------------------
// Reads of LDS: byte offset of the lane's first piece (2 g) of row l16 of a 16-row
// block; the second piece is at offset ^ 16, block t 2048 t further.
// ---------------------------------------------------------------------------
NVFP4_HD uint32_t read_offset(int l16, int g) { return (uint32_t)(128 * l16 + 16 * ((2 * g) ^ (l16 & 7))); }

// Sums done again from memory: offsets of lane group g's two pieces of chunk c in a row
// (from the row's start), pieces past its end at its last one; *in: those inside.
NVFP4_HD int64_t again_offset(int c, int64_t k, int g, int half, bool* in) {
  const int64_t o = (int64_t)kChunk * c + 16 * g + 64 * half;
  *in = o <= k - 16;
  return *in ? o : k - 16;
}

// ---------------------------------------------------------------------------
// Plans (host).
// ---------------------------------------------------------------------------
// Tile shapes: ns per chunk of 128 and per tile (first loads and epilogue), as
// measured with a CU's slots filled.  256 x 256 reaches 1.9 PFLOP/s over the chip,
// the smaller ones less (more LDS reads and loads per product), but they have finer
// steps for sizes that leave CUs idle.
struct Shape {
  int tn, tm;          // rows of W and of X
  int wn, wm, stages;  // wavefronts along them; chunks in LDS
  int per_cu;          // workgroups
  double chunk, tile;  // ns
};
constexpr Shape kShapes[4] = {{256, 256, 2, 4, 2, 1, 1900, 9000},
                              {256, 128, 4, 2, 3, 1, 1000, 7000},
                              {128, 64, 4, 2, 3, 2, 1050, 3700},
                              {256, 64, 8, 1, 3, 1, 1100, 5000}};
constexpr int kGroupedShape = 1;
constexpr int kCus = 256;

inline int64_t tiles_of(const Shape& s, int64_t m, int64_t n) {
  return ((n + s.tn - 1) / s.tn) * ((m + s.tm - 1) / s.tm);
}

// Estimated ns of the tiles over the chip, each K slice `chunks` long.  A chunk
// takes its compute time or that of its loads: 21 ns per KB that L2 holds, 43 per
// KB from HBM, where W comes from for one of the m tiles.
inline double shape_ns(const Shape& s, int64_t m, int64_t wgs, int64_t chunks) {
  const double m_tiles = (double)((m + s.tm - 1) / s.tm), slots = (double)kCus * s.per_cu;
  const double loads = 0.125 * (s.tn * (21.0 + 22.0 / m_tiles) + 21.0 * s.tm);
  // Half-filled CUs: a workgroup alone on its CU computes in a little under half the pair's time.
  const bool alone = s.per_cu == 2 && wgs <= kCus;
  const double compute = alone ? 400.0 : s.chunk, load = s.per_cu == 2 && !alone ? 2.0 * loads : loads;
  const double rounds = (double)((wgs + (int64_t)slots - 1) / (int64_t)slots);
  return rounds * (s.tile + (compute > load ? compute : load) * (double)chunks);
}

struct Plan {
  double ns = 1e300;
  int shape = 0, slices = 1;
  int64_t n1 = 0;  // columns of the 256 x 256 tiles that come first (0: one launch)
};

// The cheapest of: one shape; one shape with K split (the slices' sums take a
// write, a read and a second launch); whole rounds of 256 x 256 tiles and a
// second launch with small tiles for the columns left over, which would
// otherwise occupy a round by themselves.
inline Plan gemm_plan(int64_t m, int64_t n, int64_t k, bool split) {
  const int64_t chunks = (k + kChunk - 1) / kChunk;
  Plan best;
  for (int i = 0; i < 4; ++i) {
    const int64_t tiles = tiles_of(kShapes[i], m, n);
    for (int s = 1; s <= 8; ++s) {
      if (s > 1 && (!split || chunks < 4 * s || tiles * s > 2 * kCus ||
                    m * n > ((int64_t)1 << 26) / s))
        break;
      const double ns = shape_ns(kShapes[i], m, tiles * s, (chunks + s - 1) / s) +
                        (s > 1 ? 4000.0 + 4.0 * (double)(m * n) * s / 4000.0 : 0.0);
      if (ns < best.ns) best = Plan{ns, i, s, 0};
    }
  }
  const int64_t m_tiles = (m + 255) / 256, n_tiles = (n + 255) / 256;
  const int64_t rounds = n_tiles * m_tiles / kCus, cols = rounds * kCus / m_tiles;  // n tiles of whole rounds
  if (rounds > 0 && cols > 0 && cols < n_tiles) {
    const double ns = shape_ns(kShapes[0], m, cols * m_tiles, chunks) + 3000.0 +
                      shape_ns(kShapes[2], m, tiles_of(kShapes[2], m, n - 256 * cols), chunks);
    if (ns < best.ns) best = Plan{ns, 0, 1, 256 * cols};
  }
  return best;
}

// The launches of a plan: tile shape, and the columns n0 .. n0 + n - 1 of y.
struct Launch {
  int shape;
  int64_t n0, n;
};
inline int launches_of(const Plan& p, int64_t n, Launch (&out)[2]) {
  if (p.n1 == 0) {
    out[0] = Launch{p.shape, 0, n};
    return 1;
  }
  out[0] = Launch{0, 0, p.n1};
  out[1] = Launch{2, p.n1, n - p.n1};
  return 2;
}

// FP32 sums of one row in the workspace: n rounded up to a multiple of 4.
inline int64_t sums_per_row(int64_t n) { return (n + 3) / 4 * 4; }

// 32-bit offsets inside a tile, and at most 2^32 threads.
inline bool gemm_supported(int64_t m, int64_t n, int64_t k) {
  return k <= ((int64_t)1 << 23) && (m + 63) / 64 <= ((int64_t)1 << 22) / ((n + 127) / 128);
}

inline bool grouped_supported(int64_t t_count, int64_t topk, int64_t experts, int64_t n, int64_t k) {
  const int64_t pairs = t_count * topk, kb = (k + kChunk - 1) / kChunk;
  return k <= ((int64_t)1 << 23) && t_count <= ((int64_t)UINT32_MAX) / k && t_count <= (int64_t)UINT32_MAX / 4 / kb &&
         (pairs + 127) / 128 + experts + 8 <= ((int64_t)1 << 22) / ((n + 255) / 256);
}

// Grouped (256 x 128 tiles): m tiles per XCD.  Fewer than one tile past pairs / 128 for
// each expert that has pairs; at least one workgroup is left for rows of zeros if
// there are any.
inline int64_t grouped_m_tiles(int64_t pairs, int64_t experts) {
  return ((pairs + 127) / 128 + (experts < pairs ? experts : pairs) + 7) / 8;
}

}  // namespace fp8_tiles
}  // namespace nvfp4
