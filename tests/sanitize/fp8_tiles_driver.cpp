// Runs the E4M3 GEMM's index arithmetic (csrc/fp8_tiles.hpp, the code that the kernel
// and its launches use) on the host, for the launches that real plans make: every
// load of every wavefront, lane and instruction at the first, middle and last tiles
// and chunks lies inside its buffer and its offset fits the 32 bits that the
// instruction takes, every destination lies in its stage, the fragment reads cover
// the stage once, and every tile and zero row is some workgroup's, once.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <set>
#include <vector>

#include "fp8_tiles.hpp"

using namespace nvfp4::fp8_tiles;

namespace {

long g_checks = 0;
const char* g_where = "";

void need(bool ok, const char* what) {
  ++g_checks;
  if (!ok) {
    printf("%s: %s\n", g_where, what);
    exit(1);
  }
}

// bytes [at, at + size) of a buffer of `total`.
void inside(int64_t at, int64_t size, int64_t total, const char* what) { need(at >= 0 && at + size <= total, what); }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

std::set<int64_t> some(int64_t lo, int64_t hi) {  // of lo .. hi - 1
  std::set<int64_t> s;
  for (int64_t v : {lo, lo + 1, (lo + hi) / 2, hi - 2, hi - 1})
    if (v >= lo && v < hi) s.insert(v);
  return s;
}

// A tile: rows n0 .. of W of a matrix that ends at row n, and rows x[0 .. rows - 1] of X.
struct Tile {
  Shape s;
  int64_t n0, n, k;
  std::vector<int64_t> x;
  int64_t x_rows;          // rows of X
  int64_t x_base, s_base;  // base row of the loads of X and of its scales
  int nt, mt, n_tiles, m_tiles;
  bool ahead;
};

void check_loads(const Tile& t, int c0, int c1) {
  const int kb = (int)cdiv(t.k, kChunk), ktail = tail_of(t.k), last = c1 - 1;
  const int64_t nb = cdiv(t.n, 128), rows = (int64_t)t.x.size();
  const int lw = t.s.tn / 64, lx = t.s.tm / 64;
  const auto x_row = [&](int64_t r) { return t.x[(size_t)row_or_last(r, rows)] - t.x_base; };
  for (int w = 0; w < 8; ++w)
    for (int lane = 0; lane < 64; ++lane) {
      const int piece = lane_piece(lane);
      need(piece >= 0 && piece < 8, "piece");
      for (int64_t cc : some(c0, c1)) {
        const uint32_t back = cc == kb - 1 ? step_back(ktail, piece) : 0u;
        const auto load = [&](int64_t base_row, int64_t r, int64_t end_row, const char* what) {
          const uint32_t off = piece_offset(r, t.k, piece);
          need(r >= 0 && (int64_t)off == r * t.k + 16 * piece && off >= back, what);  // nothing lost to 32 bits
          // Inside the row, so inside the buffer.
          inside((int64_t)(off - back) + kChunk * cc - r * t.k, 16, t.k, what);
          need(base_row + r < end_row, what);
        };
        for (int j = 0; j < lw; ++j) {
          load(t.n0, row_or_last(load_row(w, j, lane), t.n - t.n0), t.n, "load of W");
          inside(load_dst(w, j) + 16 * lane, 16, 128 * t.s.tn, "W in the stage");
        }
        for (int j = 0; j < lx; ++j) {
          load(t.x_base, x_row(load_row(w, j, lane)), t.x_rows, "load of X");
          inside(load_dst(w, j) + 16 * lane, 16, 128 * t.s.tm, "X in the stage");
        }
        if (w < lx) {
          const int64_t r = x_row(64 * w + lane);
          need((int64_t)scale_offset(r, kb) == 4 * r * kb && r >= 0 && t.x_base + r < t.x_rows, "scale of X");
          inside(4 * (64 * w + lane), 4, 4 * t.s.tm, "scales of X in the stage");
        } else {
          const int64_t b0 = t.n0 / 128, b = row_or_last(lane, nb - b0);
          need((int64_t)scale_offset(b, kb) == 4 * b * kb && b >= 0 && b0 + b < nb, "scale of W");
        }
        if (t.ahead) {
          const Line l = line_ahead(t.s.tn, t.s.tm, t.n_tiles, t.m_tiles, t.nt, t.mt, w, lane);
          need(l.row >= 0 && chunk_ahead((int)cc, last) <= last && chunk_ahead((int)cc, last) >= c0, "chunk ahead");
          if (l.of_w) need(t.n0 + row_or_last(l.row, t.n - t.n0) < t.n, "line of W");
          else need(l.row < t.s.tm && t.x_base + x_row(l.row) < t.x_rows, "line of X");
        }
        // The sums done again: lane group and half.
        for (int half = 0; half < 2; ++half) {
          bool in;
          const int64_t o = again_offset((int)cc, t.k, lane >> 4, half, &in);
          inside(o, 16, t.k, "again");
          need(in == (kChunk * cc + 16 * (lane >> 4) + 64 * half + 16 <= t.k), "again: piece inside");
        }
      }
    }
}

// Every piece of every row of the stage is loaded once and read once by each wavefront
// that its rows belong to, and what is read is the row's own.
void check_stage(const Shape& s) {
  const int rows_of[2] = {s.tn, s.tm}, waves_of[2] = {s.wn, s.wm};
  for (int op = 0; op < 2; ++op) {
    const int rows = rows_of[op], waves = waves_of[op], blocks = rows / waves / 16;
    std::vector<int> logical((size_t)rows * 8, -1), seen((size_t)rows * 8, 0);
    for (int w = 0; w < 8; ++w)
      for (int j = 0; j < rows / 64; ++j)
        for (int lane = 0; lane < 64; ++lane) {
          const uint32_t at = (load_dst(w, j) + 16 * (uint32_t)lane) / 16;
          need((int)(at / 8) == load_row(w, j, lane) && logical[at] == -1, "loaded once, to its row");
          logical[at] = lane_piece(lane);
        }
    for (int wi = 0; wi < waves; ++wi)
      for (int b = 0; b < blocks; ++b)
        for (int lane = 0; lane < 64; ++lane)
          for (int half = 0; half < 2; ++half) {
            const int l16 = lane & 15, g = lane >> 4;
            const uint32_t off = (read_offset(l16, g) ^ (16u * half)) + 128 * 16 * wi * blocks + 2048 * b;
            inside(off, 16, 128 * rows, "read of LDS");
            need((int)(off / 128) == 16 * (wi * blocks + b) + l16, "row of the read");
            need(logical[off / 16] == 2 * g + half, "piece of the read");
            ++seen[off / 16];
          }
    for (int v : seen) need(v == 1, "read once");
  }
  need((int64_t)s.stages * (128 * s.tn + 128 * s.tm + 4 * s.tm + 256) + 256 <= 160 * 1024, "LDS");
  need((int64_t)s.stages * (128 * s.tn + 128 * s.tm) >= 2 * (int64_t)s.tn * s.tm, "the tile fits the stages");
}

// The lines brought ahead, whatever the numbers of tiles: rows of the tile, and those of
// the tiles that share them cover all.
void check_lines(const Shape& s) {
  g_where = "lines ahead";
  for (int m_tiles = 1; m_tiles <= 10; ++m_tiles)
    for (int n_tiles = 1; n_tiles <= 40; ++n_tiles) {
      const int share_w = share_of_w(m_tiles), share_x = share_of_x(m_tiles, n_tiles);
      std::vector<char> w_hit((size_t)s.tn, 0), x_hit((size_t)s.tm, 0);
      for (int mt = 0; mt < share_w; ++mt)
        for (int nt = 0; nt < share_x; ++nt)
          for (int w = 0; w < 8; ++w)
            for (int lane = 0; lane < 64; ++lane) {
              const Line l = line_ahead(s.tn, s.tm, n_tiles, m_tiles, nt, mt, w, lane);
              need(l.row >= 0 && (l.of_w || l.row < s.tm), "row of the line");
              if (l.of_w && l.row < s.tn) w_hit[(size_t)l.row] = 1;
              if (!l.of_w) x_hit[(size_t)l.row] = 1;
            }
      for (char v : w_hit) need(v, "all rows of W");
      for (char v : x_hit) need(v, "all rows of X");
    }
}

void check_dense(int64_t m, int64_t n, int64_t k, bool split) {
  static char where[128];
  snprintf(where, sizeof where, "%ld x %ld x %ld, split %d", (long)m, (long)n, (long)k, (int)split);
  g_where = where;
  need(gemm_supported(m, n, k), "supported");
  const Plan p = gemm_plan(m, n, k, split);
  const int kb = (int)cdiv(k, kChunk);
  need(split || p.slices == 1, "no slices without a workspace");
  need(m * sums_per_row(n) / 4 <= UINT32_MAX && sums_per_row(n) >= n, "join's index");
  Launch l[2];
  const int count = launches_of(p, n, l);
  int64_t covered = 0;
  for (int i = 0; i < count; ++i) {
    const Shape s = kShapes[l[i].shape];
    need(l[i].n0 == covered && l[i].n > 0 && l[i].n0 % 128 == 0 && (count == 1 || p.slices == 1), "columns");
    covered += l[i].n;
    const int n_tiles = (int)cdiv(l[i].n, s.tn), m_tiles = (int)cdiv(m, s.tm);
    const int64_t tiles = (int64_t)n_tiles * m_tiles;
    need(tiles * p.slices * 512 <= (int64_t)UINT32_MAX && tiles <= INT32_MAX, "grid");
    std::vector<char> hit((size_t)tiles, 0);
    for (int id = 0; id < (int)tiles; ++id) {
      const int t = tile_of_id(id, (int)tiles);
      need(t >= 0 && t < tiles && !hit[(size_t)t], "tile once");
      hit[(size_t)t] = 1;
    }
    for (int slice = 0, end = 0; slice < p.slices; ++slice) {
      const int c0 = first_chunk(kb, slice, p.slices), c1 = first_chunk(kb, slice + 1, p.slices);
      need(c0 == end && c1 > c0 && (p.slices == 1 || c1 - c0 > 1), "chunks of the slice");
      end = c1;
      if (slice + 1 == p.slices) need(c1 == kb, "all chunks");
      for (int64_t nt : some(0, n_tiles))
        for (int64_t mt : some(0, m_tiles)) {
          Tile t{s, nt * s.tn, l[i].n, k, {}, m, mt * s.tm, mt * s.tm, (int)nt, (int)mt, n_tiles, m_tiles, s.stages == 2};
          for (int64_t r = mt * s.tm; r < std::min<int64_t>(m, (mt + 1) * s.tm); ++r) t.x.push_back(r);
          check_loads(t, c0, c1);
        }
    }
  }
  need(covered == n, "all columns");
}

void check_grouped(int64_t tokens, int64_t topk, int64_t experts, int64_t n, int64_t k, int invalid_of_16, unsigned seed) {
  static char where[128];
  snprintf(where, sizeof where, "%ld tokens, %ld of %ld, %ld x %ld", (long)tokens, (long)topk, (long)experts, (long)n, (long)k);
  g_where = where;
  need(grouped_supported(tokens, topk, experts, n, k), "supported");
  const Shape s = kShapes[kGroupedShape];
  const int64_t pairs = tokens * topk;
  srand(seed);
  std::vector<std::vector<int64_t>> of((size_t)experts + 1);
  for (int64_t i = 0; i < pairs; ++i)
    of[(size_t)(rand() % 16 < invalid_of_16 ? experts : rand() % experts)].push_back(i);
  std::vector<int64_t> perm, pair_off{0}, tile_off{0};
  for (int64_t e = 0; e <= experts; ++e) {
    perm.insert(perm.end(), of[(size_t)e].begin(), of[(size_t)e].end());
    if (e < experts) {
      pair_off.push_back((int64_t)perm.size());
      tile_off.push_back(tile_off.back() + cdiv((int64_t)of[(size_t)e].size(), s.tm));
    }
  }
  const int n_tiles = (int)cdiv(n, s.tn), m_tiles = (int)grouped_m_tiles(pairs, experts);
  const int64_t used = tile_off[(size_t)experts];
  need((int64_t)8 * n_tiles * m_tiles * 512 <= (int64_t)UINT32_MAX, "grid");
  std::vector<int> tile_hit((size_t)used * n_tiles, 0), row_hit((size_t)pairs * n_tiles, 0);
  const std::set<int64_t> looked = some(0, used);
  for (int id = 0; id < 8 * n_tiles * m_tiles; ++id) {
    const int nt = (id >> 3) % n_tiles, mt = (id >> 3) / n_tiles, xcd = id & 7;
    const int64_t t0 = first_of_xcd(used, xcd), tn = first_of_xcd(used, xcd + 1) - t0;
    if (mt >= tn) {
      const int64_t left = left_places(used, m_tiles);
      need(left > 0, "places left");
      for (int64_t i = pair_off[(size_t)experts] + left_rank(xcd, m_tiles, t0, tn, mt); i < pairs; i += left) {
        need(i >= pair_off[(size_t)experts], "row of zeros");
        ++row_hit[(size_t)(perm[(size_t)i] * n_tiles + nt)];
      }
      continue;
    }
    const int64_t at = t0 + mt;
    need(at < used, "tile in use");
    ++tile_hit[(size_t)(at * n_tiles + nt)];
    if (!looked.count(at) || (nt != 0 && nt != n_tiles - 1)) continue;
    int64_t e = 0;
    while (e + 1 < experts && tile_off[(size_t)e + 1] <= at) ++e;
    Tile t{s, (int64_t)nt * s.tn, n, k, {}, tokens, 0, 0, nt, mt, n_tiles, m_tiles, false};
    const int64_t first = pair_off[(size_t)e] + (at - tile_off[(size_t)e]) * s.tm;
    for (int64_t i = first; i < std::min(pair_off[(size_t)e + 1], first + s.tm); ++i) t.x.push_back(perm[(size_t)i] / topk);
    need(!t.x.empty(), "rows of the tile");
    check_loads(t, 0, (int)cdiv(k, kChunk));
  }
  for (int v : tile_hit) need(v == 1, "tile once");
  for (int64_t i = 0; i < pairs; ++i)
    for (int nt = 0; nt < n_tiles; ++nt)
      need(row_hit[(size_t)(perm[(size_t)i] * n_tiles + nt)] == (i >= pair_off[(size_t)experts]), "zero row once");
}

}  // namespace

int main() {
  for (const Shape& s : kShapes) check_stage(s);
  check_lines(kShapes[0]);
  const int64_t sizes[][3] = {{17, 1, 16},        {65, 1, 16},         {100, 513, 384},     {333, 5000, 17392},
                              {2048, 17408, 5120}, {129, 3000, 3088},   {257, 300, 4112},    {700, 259, 16},
                              {64, 17408, 5120},   {64, 5120, 17408},   {4100, 4500, 400},   {128, 34816, 5120},
                              {512, 17408, 5120},  {4096, 4096, 4096},  {31, 5003, 8208},    {1100000, 64, 128},
                              {3, 2000003, 48},    {200, 1000, 1 << 23}, {300, 700, (1 << 23) - 16}};
  for (const auto& z : sizes)
    for (bool split : {false, true}) check_dense(z[0], z[1], z[2], split);
  check_grouped(2048, 8, 128, 2048, 4096, 0, 1);
  check_grouped(300, 4, 6, 300, 1040, 2, 2);
  check_grouped(4200, 8, 4, 16, 128, 1, 3);
  check_grouped(600, 1, 1000, 257, 48, 16, 4);
  check_grouped(513, 1, 3, 700, 400, 5, 5);
  check_grouped(1, 520, 1, 64, 1 << 23, 1, 6);
  check_grouped(511, 4, 3, 64, (1 << 23) - 16, 1, 7);
  printf("%ld checks\n", g_checks);
  return 0;
}
