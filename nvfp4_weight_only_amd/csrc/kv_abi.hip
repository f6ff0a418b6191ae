// C entry points of the operators around a paged FP4 cache: argument validation and dispatch.
// Declarations and the meaning of every argument are in include/nvfp4.h.
#include <math.h>
#include <stdint.h>

#include "abi_common.hpp"
#include "kv_common.hpp"
#include "launch.hpp"
#include "nvfp4.h"

namespace {

using namespace nvfp4_abi;

constexpr int64_t kMaxHeadDim = 2048;            // angles of a row that fit LDS
constexpr int64_t kMaxRow = (int64_t)1 << 24;    // elements of a row of heads
// Rows, sequences and rows times heads of a call: the launches' threads stay below 2^32.
constexpr int64_t kMaxRows = (int64_t)1 << 23;
constexpr int64_t kMaxSeqs = (int64_t)1 << 19;
constexpr int64_t kMaxRowHeads = (int64_t)1 << 28;
constexpr int64_t kMaxTokens = INT32_MAX - 4096;  // tokens of a sequence: a tile's end stays an int32

constexpr int64_t kMaxCacheRows = (int64_t)1 << 30;  // tokens times heads that attention addresses

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
  const void* p;
  int64_t bytes;
};

// Whether any of outs overlaps one of ins or another of outs.
bool clash(const Range* outs, int nouts, const Range* ins, int nins) {
  for (int i = 0; i < nouts; ++i) {
    for (int j = 0; j < nins; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
    for (int j = i + 1; j < nouts; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
  }
  return false;
}

bool known_type(int type) { return type == NVFP4_OUT_F16 || type == NVFP4_OUT_BF16; }

// Bytes from the first to behind the last element of a [rows, heads, head_dim] tensor
// of 16-bit values; strides of axes of length 1 are set to 0.
nvfp4_status extent(int64_t rows, int64_t heads, int64_t head_dim, int64_t* row_stride, int64_t* head_stride,
                    int64_t* bytes) {
  if (rows <= 1) *row_stride = 0;
  if (heads <= 1) *head_stride = 0;
  if (*row_stride < 0 || *head_stride < 0) return NVFP4_ERR_SHAPE;
  int64_t a, b;
  if (!mul_ok(rows > 0 ? rows - 1 : 0, *row_stride, &a) || !mul_ok(heads - 1, *head_stride, &b)) return NVFP4_ERR_SHAPE;
  if (a > INT64_MAX / 8 || b > INT64_MAX / 8) return NVFP4_ERR_SHAPE;
  *bytes = rows > 0 ? 2 * (a + b + head_dim) : 0;
  return NVFP4_OK;
}

// Whether no two elements of such a tensor share a place, with either axis outside.
bool apart(int64_t rows, int64_t heads, int64_t head_dim, int64_t row_stride, int64_t head_stride) {
  const bool r = rows > 1, h = heads > 1;
  if (r && h)
    return (head_stride >= head_dim && row_stride >= (heads - 1) * head_stride + head_dim) ||
           (row_stride >= head_dim && head_stride >= (rows - 1) * row_stride + head_dim);
  return (!r || row_stride >= head_dim) && (!h || head_stride >= head_dim);
}

nvfp4_status check_rope(const nvfp4_rope_spec* rope, int64_t head_dim, nvfp4::RopeArgs* out) {
  if (!rope->freqs) return NVFP4_ERR_NULL;
  if (rope->rot_dim <= 0 || rope->rot_dim % 16 != 0 || rope->rot_dim > head_dim) return NVFP4_ERR_SHAPE;
  if (!isfinite(rope->amplitude)) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned_to(rope->freqs, 8)) return NVFP4_ERR_ALIGN;
  *out = {rope->freqs, rope->rot_dim, rope->amplitude, rope->interleaved != 0};
  return NVFP4_OK;
}

struct CacheSizes {
  int64_t codes, scales;  // bytes of one tensor
};

nvfp4_status check_cache(const nvfp4_kv_cache* c, nvfp4::KvCache* out, CacheSizes* sz) {
  if (!c) return NVFP4_ERR_NULL;
  if (c->format != NVFP4_KV_NVFP4 && c->format != NVFP4_KV_MXFP4) return NVFP4_ERR_UNSUPPORTED;
  const bool mx = c->format == NVFP4_KV_MXFP4;
  const int64_t g = mx ? 32 : 16;
  if (c->num_blocks <= 0 || c->block_size <= 0 || c->heads <= 0 || c->head_dim <= 0 || c->head_dim % g != 0)
    return NVFP4_ERR_SHAPE;
  int64_t tokens, rows, elems;
  if (!mul_ok(c->num_blocks, c->block_size, &tokens) || !mul_ok(tokens, c->heads, &rows) ||
      !mul_ok(rows, c->head_dim, &elems))
    return NVFP4_ERR_SHAPE;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || (!mx && (!c->k_tscale || !c->v_tscale)))
    return NVFP4_ERR_NULL;
  if (c->head_dim > kMaxHeadDim || c->heads > kMaxRow / c->head_dim || c->block_size > kMaxTokens)
    return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales) ||
      (!mx && (!aligned_to(c->k_tscale, 4) || !aligned_to(c->v_tscale, 4))))
    return NVFP4_ERR_ALIGN;
  sz->codes = elems / 2;
  sz->scales = elems / g;
  *out = {mx, c->num_blocks, c->block_size, c->heads, c->head_dim, {c->k_codes, c->v_codes},
          {c->k_scales, c->v_scales}, {c->k_tscale, c->v_tscale}};
  return NVFP4_OK;
}

nvfp4_status check_batch(const nvfp4::KvCache& c, int64_t rows, const int32_t* block_table, int64_t max_blocks,
                         const int32_t* seq_lens, const int32_t* row_start, int64_t seqs, nvfp4::KvBatch* out) {
  int64_t cap, entries;
  if (rows < 0 || seqs < 0 || max_blocks <= 0 || !mul_ok(max_blocks, c.block_size, &cap) ||
      !mul_ok(seqs, max_blocks, &entries) || entries > INT64_MAX / 8 || (!row_start && rows != seqs))
    return NVFP4_ERR_SHAPE;
  if (rows > kMaxRows || seqs > kMaxSeqs || cap > kMaxTokens) return NVFP4_ERR_UNSUPPORTED;
  *out = {block_table, max_blocks, seq_lens, row_start, seqs, rows};
  if (rows == 0 || seqs == 0) return NVFP4_OK;
  if (!block_table || !seq_lens) return NVFP4_ERR_NULL;
  if (!aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(row_start, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_rope_frequencies(int scaling, int64_t rot_dim, double base, double factor, double original,
                                    double low, double high, double* freqs, void* stream) {
  if (scaling < NVFP4_ROPE_NONE || scaling > NVFP4_ROPE_WAVELENGTH) return NVFP4_ERR_UNSUPPORTED;
  if (rot_dim <= 0 || rot_dim % 16 != 0 || rot_dim > kMaxHeadDim) return NVFP4_ERR_SHAPE;
  if (!(base > 1.0 && isfinite(base))) return NVFP4_ERR_UNSUPPORTED;
  if (scaling != NVFP4_ROPE_NONE && !(factor >= 1.0 && isfinite(factor))) return NVFP4_ERR_UNSUPPORTED;
  if (scaling >= NVFP4_ROPE_RAMP &&
      !(original > 0.0 && isfinite(original) && low > 0.0 && high > low && isfinite(high)))
    return NVFP4_ERR_UNSUPPORTED;
  if (!freqs) return NVFP4_ERR_NULL;
  if (!aligned_to(freqs, 8)) return NVFP4_ERR_ALIGN;
  nvfp4_status st;
  if ((st = check_device()) != NVFP4_OK) return st;
  nvfp4::launch_rope_frequencies(scaling, rot_dim, base, factor, original, low, high, freqs,
                                 static_cast<hipStream_t>(stream));
  return launch_status();
}

nvfp4_status nvfp4_rope(int type, const uint16_t* x, int64_t rows, int64_t heads, int64_t head_dim,
                        int64_t x_row_stride, int64_t x_head_stride, const int32_t* positions,
                        const nvfp4_rope_spec* rope, int inverse, uint16_t* out, int64_t out_row_stride,
                        int64_t out_head_stride, void* stream) {
  if (!known_type(type)) return NVFP4_ERR_UNSUPPORTED;
  if (rows < 0 || heads <= 0 || head_dim <= 0 || head_dim % 8 != 0) return NVFP4_ERR_SHAPE;
  if (!rope) return NVFP4_ERR_NULL;
  nvfp4::RopeArgs turn;
  nvfp4_status st = check_rope(rope, head_dim, &turn);
  if (st != NVFP4_OK) return st;
  if (head_dim > kMaxHeadDim || heads > kMaxRow / head_dim) return NVFP4_ERR_UNSUPPORTED;
  int64_t xb, ob;
  if ((st = extent(rows, heads, head_dim, &x_row_stride, &x_head_stride, &xb)) != NVFP4_OK ||
      (st = extent(rows, heads, head_dim, &out_row_stride, &out_head_stride, &ob)) != NVFP4_OK)
    return st;
  if (!apart(rows, heads, head_dim, out_row_stride, out_head_stride)) return NVFP4_ERR_SHAPE;
  if (rows > kMaxRows) return NVFP4_ERR_UNSUPPORTED;
  if (rows == 0) return NVFP4_OK;
  if (!x || !positions || !out) return NVFP4_ERR_NULL;
  if (!aligned16(x) || !aligned16(out) || !aligned_to(positions, 4) ||
      ((x_row_stride | x_head_stride | out_row_stride | out_head_stride) & 7) != 0)
    return NVFP4_ERR_ALIGN;
  const bool in_place = x == out && x_row_stride == out_row_stride && x_head_stride == out_head_stride;
  const Range o = {out, ob};
  const Range ins[3] = {{x, in_place ? 0 : xb}, {positions, 4 * rows}, {turn.freqs, 4 * turn.rot}};
  if (clash(&o, 1, ins, 3)) return NVFP4_ERR_ALIAS;
  if ((st = check_device()) != NVFP4_OK) return st;
  nvfp4::launch_rope(type == NVFP4_OUT_BF16, x, rows, heads, head_dim, x_row_stride, x_head_stride, positions, turn,
                     inverse != 0, out, out_row_stride, out_head_stride, static_cast<hipStream_t>(stream));
  return launch_status();
}

nvfp4_status nvfp4_kv_append(const nvfp4_kv_cache* cache, int type, const uint16_t* k, const uint16_t* v, int64_t rows,
                             int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride, int64_t v_head_stride,
                             const int32_t* block_table, int64_t max_blocks, const int32_t* seq_lens,
                             const int32_t* row_start, int64_t seqs, const nvfp4_rope_spec* rope,
                             const int32_t* positions, void* stream) {
  nvfp4::KvCache c;
  CacheSizes sz;
  nvfp4_status st = check_cache(cache, &c, &sz);
  if (st != NVFP4_OK) return st;
  if (!known_type(type)) return NVFP4_ERR_UNSUPPORTED;
  nvfp4::KvBatch b;
  if ((st = check_batch(c, rows, block_table, max_blocks, seq_lens, row_start, seqs, &b)) != NVFP4_OK) return st;
  nvfp4::RopeArgs turn = {nullptr, 0, 1.0f, 0};
  if (rope && (st = check_rope(rope, c.head_dim, &turn)) != NVFP4_OK) return st;
  int64_t kb, vb;
  if ((st = extent(rows, c.heads, c.head_dim, &k_row_stride, &k_head_stride, &kb)) != NVFP4_OK ||
      (st = extent(rows, c.heads, c.head_dim, &v_row_stride, &v_head_stride, &vb)) != NVFP4_OK)
    return st;
  if (rows == 0 || seqs == 0) return NVFP4_OK;
  if (!k || !v) return NVFP4_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned_to(positions, 4) ||
      ((k_row_stride | k_head_stride | v_row_stride | v_head_stride) & 7) != 0)
    return NVFP4_ERR_ALIGN;
  const Range outs[4] = {{c.codes[0], sz.codes}, {c.scales[0], sz.scales}, {c.codes[1], sz.codes}, {c.scales[1], sz.scales}};
  const Range ins[9] = {{k, kb}, {v, vb}, {block_table, 4 * seqs * max_blocks}, {seq_lens, 4 * seqs},
                        {row_start, row_start ? 4 * (seqs + 1) : 0}, {positions, positions && rope ? 4 * rows : 0},
                        {turn.freqs, 4 * turn.rot}, {c.tscale[0], c.mx ? 0 : 4}, {c.tscale[1], c.mx ? 0 : 4}};
  if (clash(outs, 4, ins, 9)) return NVFP4_ERR_ALIAS;
  if ((st = check_device()) != NVFP4_OK) return st;
  nvfp4::launch_kv_append(c, b, type == NVFP4_OUT_BF16, k, v, k_row_stride, k_head_stride, v_row_stride, v_head_stride,
                          turn, rope ? positions : nullptr, static_cast<hipStream_t>(stream));
  return launch_status();
}

static bool attention_head_dim(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

int64_t nvfp4_kv_attention_workspace_bytes(int64_t heads, int64_t head_dim, int64_t q_heads, int64_t rows,
                                           int64_t seqs) {
  if (heads <= 0 || q_heads <= 0 || q_heads % heads != 0 || rows < 0 || seqs < 0 || !attention_head_dim(head_dim) ||
      heads > kMaxRow / head_dim || q_heads > UINT16_MAX || rows > kMaxRows || rows > kMaxRowHeads / q_heads ||
      seqs > kMaxSeqs)
    return -1;
  return rows == 0 || seqs == 0 ? 0 : nvfp4::kv_attend_workspace_bytes(heads, head_dim, q_heads, rows, seqs);
}

nvfp4_status nvfp4_kv_attention(const nvfp4_kv_cache* cache, int type, const uint16_t* q, int64_t rows,
                                int64_t q_heads, int64_t q_row_stride, int64_t q_head_stride,
                                const int32_t* block_table, int64_t max_blocks, const int32_t* seq_lens,
                                const int32_t* row_start, int64_t seqs, float scale, int64_t window, uint16_t* out,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  nvfp4::KvCache c;
  CacheSizes sz;
  nvfp4_status st = check_cache(cache, &c, &sz);
  if (st != NVFP4_OK) return st;
  if (!known_type(type) || !isfinite(scale)) return NVFP4_ERR_UNSUPPORTED;
  nvfp4::KvBatch b;
  if ((st = check_batch(c, rows, block_table, max_blocks, seq_lens, row_start, seqs, &b)) != NVFP4_OK) return st;
  if (q_heads <= 0 || q_heads % c.heads != 0 || window < 0 || workspace_bytes < 0) return NVFP4_ERR_SHAPE;
  if (!attention_head_dim(c.head_dim) || q_heads > UINT16_MAX || rows > kMaxRowHeads / q_heads ||
      c.num_blocks * c.block_size * c.heads > kMaxCacheRows)
    return NVFP4_ERR_UNSUPPORTED;
  int64_t qb;
  if ((st = extent(rows, q_heads, c.head_dim, &q_row_stride, &q_head_stride, &qb)) != NVFP4_OK) return st;
  if (rows == 0 || seqs == 0) return NVFP4_OK;
  if (!q || !out || !workspace) return NVFP4_ERR_NULL;
  const int64_t need = nvfp4::kv_attend_workspace_bytes(c.heads, c.head_dim, q_heads, rows, seqs);
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || ((q_row_stride | q_head_stride) & 7) != 0)
    return NVFP4_ERR_ALIGN;
  const Range outs[2] = {{out, 2 * rows * q_heads * c.head_dim}, {workspace, need}};
  const Range ins[10] = {{q, qb}, {c.codes[0], sz.codes}, {c.scales[0], sz.scales}, {c.codes[1], sz.codes},
                         {c.scales[1], sz.scales}, {block_table, 4 * seqs * max_blocks}, {seq_lens, 4 * seqs},
                         {row_start, row_start ? 4 * (seqs + 1) : 0}, {c.tscale[0], c.mx ? 0 : 4},
                         {c.tscale[1], c.mx ? 0 : 4}};
  if (clash(outs, 2, ins, 10)) return NVFP4_ERR_ALIAS;
  if ((st = check_device()) != NVFP4_OK) return st;
  nvfp4::launch_kv_attend(c, b, type == NVFP4_OUT_BF16, q, q_heads, q_row_stride, q_head_stride, scale,
                          window < INT32_MAX ? window : INT32_MAX, out, workspace, static_cast<hipStream_t>(stream));
  return launch_status();
}

}  // extern "C"
