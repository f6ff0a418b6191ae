// C entry points of the E4M3 operators: argument validation and dispatch.
// Declarations and the meaning of every argument are in include/nvfp4.h.
#include <float.h>
#include <stdint.h>

#include "abi_common.hpp"
#include "launch.hpp"
#include "nvfp4.h"

namespace {

using namespace nvfp4_abi;

// Sizes in bytes of count tensors [rows, k] of codes, their scales with
// block_rows x 128 blocks, and the BF16 tensors of the same shape.
struct Fp8Sizes {
  int64_t codes, scales, bf16;
};

nvfp4_status fp8_sizes(int64_t count, int64_t rows, int64_t k, int64_t block_rows, Fp8Sizes* s) {
  if (count < 0 || rows < 0 || k <= 0 || (k & 15) != 0) return NVFP4_ERR_SHAPE;
  int64_t all;
  if (!mul_ok(count, rows, &all) || !mul_ok(all, k, &s->codes) || !mul_ok(s->codes, 4, &s->bf16))
    return NVFP4_ERR_SHAPE;
  s->bf16 = 2 * s->codes;
  // At most one block per element, so 4 bytes of scale each do not overflow past the check above.
  const int64_t row_blocks = rows / block_rows + (rows % block_rows != 0);
  s->scales = s->codes == 0 ? 0 : 4 * count * row_blocks * (k / 128 + (k % 128 != 0));
  return NVFP4_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether any of outs overlaps one of ins or another of outs.
struct Buffer {
  const void* p;
  int64_t bytes;
};
bool clash(const Buffer* outs, int nouts, const Buffer* ins, int nins) {
  for (int i = 0; i < nouts; ++i) {
    for (int j = 0; j < nins; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
    for (int j = i + 1; j < nouts; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
  }
  return false;
}

// Blocks along k, tiles and rows beyond the kernels' index ranges.
bool too_many(int64_t count, int64_t rows, int64_t k) {
  int64_t all;
  return k > ((int64_t)1 << 37) || !mul_ok(count, rows, &all) || all > ((int64_t)1 << 35);
}

nvfp4_status fp8_linear_sizes(int64_t m, int64_t n, int64_t k, Fp8Sizes* x, Fp8Sizes* w, int64_t* y_bytes) {
  nvfp4_status st;
  if (n <= 0) return NVFP4_ERR_SHAPE;
  if ((st = fp8_sizes(1, m, k, 1, x)) != NVFP4_OK || (st = fp8_sizes(1, n, k, 128, w)) != NVFP4_OK) return st;
  int64_t ye;
  if (!mul_ok(m, n, &ye) || !mul_ok(ye, 8, y_bytes)) return NVFP4_ERR_SHAPE;
  *y_bytes = 2 * ye;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_fp8_quantize(const uint16_t* w, int64_t count, int64_t rows, int64_t k, int64_t block_rows,
                                uint8_t* codes, float* scales, void* stream) {
  if (block_rows != 1 && block_rows != 128) return NVFP4_ERR_UNSUPPORTED;
  Fp8Sizes sz;
  nvfp4_status st = fp8_sizes(count, rows, k, block_rows, &sz);
  if (st != NVFP4_OK) return st;
  if (sz.codes == 0) return NVFP4_OK;
  if (!w || !codes || !scales) return NVFP4_ERR_NULL;
  if (too_many(count, rows, k)) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales)) return NVFP4_ERR_ALIGN;
  const Buffer outs[2] = {{codes, sz.codes}, {scales, sz.scales}}, in = {w, sz.bf16};
  if (clash(outs, 2, &in, 1)) return NVFP4_ERR_ALIAS;
  if ((st = check_device()) != NVFP4_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (block_rows == 1) nvfp4::launch_fp8_quantize_rows(w, count * rows, k, codes, scales, s);
  else nvfp4::launch_fp8_quantize_tiles(w, count, rows, k, codes, scales, s);
  return launch_status();
}

nvfp4_status nvfp4_rmsnorm_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                               int64_t rows, int64_t k, uint16_t* residual_out, uint8_t* codes, float* scales,
                               void* stream) {
  Fp8Sizes sz;
  nvfp4_status st = fp8_sizes(1, rows, k, 1, &sz);
  if (st != NVFP4_OK) return st;
  if (!(eps >= FLT_MIN && eps <= FLT_MAX)) return NVFP4_ERR_UNSUPPORTED;
  if (rows == 0) return NVFP4_OK;
  if (!x || !weight || !codes || !scales || (residual == nullptr) != (residual_out == nullptr)) return NVFP4_ERR_NULL;
  if (too_many(1, rows, k)) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) || !aligned16(codes) ||
      !aligned16(scales))
    return NVFP4_ERR_ALIGN;
  const bool in_place = residual_out != nullptr && residual_out == residual;
  const Buffer outs[3] = {{codes, sz.codes}, {scales, sz.scales}, {residual_out, residual_out ? sz.bf16 : 0}};
  const Buffer ins[3] = {{x, sz.bf16}, {weight, 2 * k}, {residual, residual && !in_place ? sz.bf16 : 0}};
  if (clash(outs, 3, ins, 3)) return NVFP4_ERR_ALIAS;
  if ((st = check_device()) != NVFP4_OK) return st;
  nvfp4::launch_rmsnorm_fp8(x, residual, weight, eps, rows, k, residual_out, codes, scales,
                            static_cast<hipStream_t>(stream));
  return launch_status();
}

nvfp4_status nvfp4_silu_mul_fp8(const uint16_t* gate_up, int64_t rows, int64_t n, uint8_t* codes, float* scales,
                                void* stream) {
  Fp8Sizes sz;
  nvfp4_status st = fp8_sizes(1, rows, n, 1, &sz);
  if (st != NVFP4_OK) return st;
  if (rows == 0) return NVFP4_OK;
  if (!gate_up || !codes || !scales) return NVFP4_ERR_NULL;
  if (too_many(1, rows, n)) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(gate_up) || !aligned16(codes) || !aligned16(scales)) return NVFP4_ERR_ALIGN;
  const Buffer outs[2] = {{codes, sz.codes}, {scales, sz.scales}}, in = {gate_up, 2 * sz.bf16};
  if (clash(outs, 2, &in, 1)) return NVFP4_ERR_ALIAS;
  if ((st = check_device()) != NVFP4_OK) return st;
  nvfp4::launch_silu_mul_fp8(gate_up, rows, n, codes, scales, static_cast<hipStream_t>(stream));
  return launch_status();
}

int64_t nvfp4_fp8_linear_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  Fp8Sizes x, w;
  int64_t yb;
  if (fp8_linear_sizes(m, n, k, &x, &w, &yb) != NVFP4_OK) return -1;
  return m == 0 || !nvfp4::fp8_linear_supported(m, n, k) ? 0 : nvfp4::fp8_linear_workspace_bytes(m, n, k);
}

nvfp4_status nvfp4_fp8_linear(const uint8_t* xq, const float* xs, int64_t m, int64_t n, int64_t k, const uint8_t* wq,
                              const float* ws, uint16_t* y, void* workspace, int64_t workspace_bytes, void* stream) {
  Fp8Sizes x, w;
  int64_t yb;
  nvfp4_status st = fp8_linear_sizes(m, n, k, &x, &w, &yb);
  if (st != NVFP4_OK) return st;
  if (workspace_bytes < 0) return NVFP4_ERR_SHAPE;
  if (!wq || !ws || (m != 0 && (!xq || !xs || !y))) return NVFP4_ERR_NULL;
  if (m == 0) return NVFP4_OK;
  if (!nvfp4::fp8_linear_supported(m, n, k)) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(wq) || !aligned16(ws) || !aligned16(y) || !aligned16(workspace))
    return NVFP4_ERR_ALIGN;
  const int64_t need = nvfp4::fp8_linear_workspace_bytes(m, n, k);
  if (workspace == nullptr || workspace_bytes < need) workspace = nullptr;
  const Buffer outs[2] = {{y, yb}, {workspace, workspace ? need : 0}};
  const Buffer ins[4] = {{xq, x.codes}, {xs, x.scales}, {wq, w.codes}, {ws, w.scales}};
  if (clash(outs, 2, ins, 4)) return NVFP4_ERR_ALIAS;
  if ((st = check_device()) != NVFP4_OK) return st;
  nvfp4::launch_fp8_linear(xq, xs, m, n, k, wq, ws, y, need > 0 ? workspace : nullptr,
                           static_cast<hipStream_t>(stream));
  return launch_status();
}

int64_t nvfp4_fp8_linear_grouped_workspace_bytes(int64_t t_count, int64_t topk, int64_t e) {
  int64_t pairs;
  if (t_count < 0 || topk < 1 || e < 1 || !mul_ok(t_count, topk, &pairs) || pairs > INT64_MAX / 8 ||
      e > INT64_MAX / 32)
    return -1;
  return nvfp4::grouped_workspace_bytes(pairs, e);
}

nvfp4_status nvfp4_fp8_linear_grouped(const uint8_t* xq, const float* xs, int64_t t_count, int64_t topk,
                                      const int32_t* route, int64_t e, int64_t n, int64_t k, const uint8_t* wq,
                                      const float* ws, uint16_t* y, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
  if (e < 1 || n <= 0) return NVFP4_ERR_SHAPE;
  const int64_t need = nvfp4_fp8_linear_grouped_workspace_bytes(t_count, topk, e);
  if (need < 0) return NVFP4_ERR_SHAPE;
  Fp8Sizes x, w;
  nvfp4_status st;
  if ((st = fp8_sizes(1, t_count, k, 1, &x)) != NVFP4_OK || (st = fp8_sizes(e, n, k, 128, &w)) != NVFP4_OK) return st;
  const int64_t pairs = t_count * topk;
  int64_t ye, yb;
  if (!mul_ok(pairs, n, &ye) || !mul_ok(ye, 2, &yb)) return NVFP4_ERR_SHAPE;
  if (!wq || !ws || (t_count != 0 && (!xq || !xs || !route || !y || !workspace))) return NVFP4_ERR_NULL;
  if (t_count == 0) return NVFP4_OK;
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  if (!nvfp4::fp8_grouped_supported(t_count, topk, e, n, k)) return NVFP4_ERR_UNSUPPORTED;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(wq) || !aligned16(ws) || !aligned16(y) ||
      !aligned16(workspace) || !aligned4(route))
    return NVFP4_ERR_ALIGN;
  const Buffer outs[2] = {{y, yb}, {workspace, need}};
  const Buffer ins[5] = {{xq, x.codes}, {xs, x.scales}, {wq, w.codes}, {ws, w.scales}, {route, 4 * pairs}};
  if (clash(outs, 2, ins, 5)) return NVFP4_ERR_ALIAS;
  if ((st = check_device()) != NVFP4_OK) return st;
  nvfp4::launch_fp8_linear_grouped(xq, xs, t_count, topk, route, e, n, k, wq, ws, y, workspace,
                                   static_cast<hipStream_t>(stream));
  return launch_status();
}

}  // extern "C"
