// C-ABI entry points of the 8-bit floating-point setting (declared in
// include/svdq.h).  Arguments are validated on the host before any HIP call.
#include <algorithm>

#include "checks.h"
#include "internal.h"

using namespace svdq;

namespace {

// y's type without the choice of its sums (any other value as it is: check_y refuses it).
int y_type(int y_dtype) { return y_dtype == (SVDQ_OUT_BF16 | SVDQ_FP8_FAST_SUMS) ? SVDQ_OUT_BF16 : y_dtype; }

int check_dims(int m, int n) {
  REQUIRE(m >= 1 && n >= 1, SVDQ_ERR_INVALID_ARG, "m and n must be >= 1 (got m=%d n=%d)", m, n);
  REQUIRE(m <= SVDQ_MAX_DIM && n <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "m and n must be <= %d (got m=%d n=%d)",
          SVDQ_MAX_DIM, m, n);
  return SVDQ_OK;
}

int check_weights(const uint8_t* qw, const uint8_t* wscale, const uint16_t* bias) {
  REQUIRE(qw && wscale, SVDQ_ERR_INVALID_ARG, "layer qw / wscale must not be NULL");
  REQUIRE(aligned16(qw), SVDQ_ERR_ALIGNMENT, "layer qw must be 16-byte aligned");
  REQUIRE(((uintptr_t)bias & 1u) == 0, SVDQ_ERR_ALIGNMENT, "layer bias must be 2-byte aligned");
  return SVDQ_OK;
}

int check_codes(const uint8_t* qx, const uint8_t* ascale) {
  REQUIRE(qx && ascale, SVDQ_ERR_INVALID_ARG, "qx and ascale must not be NULL");
  REQUIRE(aligned16(qx), SVDQ_ERR_ALIGNMENT, "qx must be 16-byte aligned");
  return SVDQ_OK;
}

int check_x(const uint16_t* x, int rows, int m) {
  REQUIRE(x != nullptr, SVDQ_ERR_INVALID_ARG, "x must not be NULL");
  REQUIRE(((uintptr_t)x & 1u) == 0, SVDQ_ERR_ALIGNMENT, "x must be 2-byte aligned");
  REQUIRE(launch_fits(fp8_act_grid(rows, m), 256), SVDQ_ERR_UNSUPPORTED, "x is too large (%d rows of %d)", rows, m);
  return SVDQ_OK;
}

// The layer, rows, output and epilogue of a product; a layer of no rows is done
// once its dimensions are right.
int check_product(const svdq_fp8_layer* L, const svdq_epilogue* epi, int b, void* y, int y_dtype, EpiArgs* ep) {
  REQUIRE(L != nullptr, SVDQ_ERR_INVALID_ARG, "layer is NULL");
  int st = check_dims(L->m, L->n);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_type(y_dtype), b);
  if (!st) st = check_epilogue(epi, b, L->n, y, y_type(y_dtype), ep);
  if (st || b == 0) return st;
  st = check_weights(L->qw, L->wscale, L->bias);
  if (st) return st;
  const Fp8Plan plan = fp8_plan(b, L->n, L->m, 0, y_dtype);
  REQUIRE(launch_fits(plan.split.grid, plan.threads), SVDQ_ERR_UNSUPPORTED, "too many output tiles (b=%d, n=%d)", b,
          L->n);
  return SVDQ_OK;
}

int check_grouped_product(const svdq_fp8_grouped_layer* L, const svdq_epilogue* epi, int x_rows,
                          const int32_t* row_index, const int32_t* offsets, int b, void* y, int y_dtype, EpiArgs* ep) {
  REQUIRE(L != nullptr, SVDQ_ERR_INVALID_ARG, "layer is NULL");
  REQUIRE(L->experts >= 1, SVDQ_ERR_INVALID_ARG, "experts must be >= 1 (got %d)", L->experts);
  REQUIRE(L->experts <= SVDQ_MAX_EXPERTS, SVDQ_ERR_UNSUPPORTED, "experts must be <= %d (got %d)", SVDQ_MAX_EXPERTS,
          L->experts);
  int st = check_dims(L->m, L->n);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_type(y_dtype), b);
  REQUIRE(st || !epi || (!epi->gate && !epi->residual), SVDQ_ERR_UNSUPPORTED,
          "a grouped product takes no gate and no residual");
  if (!st) st = check_epilogue(epi, b, L->n, y, y_type(y_dtype), ep);
  if (st || b == 0) return st;
  REQUIRE(offsets != nullptr, SVDQ_ERR_INVALID_ARG, "offsets must not be NULL");
  REQUIRE(((uintptr_t)offsets & 3u) == 0 && ((uintptr_t)row_index & 3u) == 0, SVDQ_ERR_ALIGNMENT,
          "offsets and row_index must be 4-byte aligned");
  REQUIRE(x_rows >= 1 && (row_index || x_rows >= b), SVDQ_ERR_INVALID_ARG,
          "x_rows must be >= 1, and >= b without a row_index (got %d)", x_rows);
  REQUIRE(x_rows <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "x_rows must be <= %d (got %d)", SVDQ_MAX_DIM, x_rows);
  st = check_weights(L->qw, L->wscale, L->bias);
  if (st) return st;
  const Fp8Plan plan = fp8_plan(b, L->n, L->m, L->experts, y_dtype);
  REQUIRE(launch_fits(plan.split.grid, plan.threads), SVDQ_ERR_UNSUPPORTED,
          "too many output tiles (b=%d, n=%d, experts=%d)", b, L->n, L->experts);
  return SVDQ_OK;
}

// The product's workspace, whatever its output's type and sums.
size_t fp8_gemm_ws_bytes(int b, int n, int m) {
  return std::max(fp8_plan(b, n, m, 0, SVDQ_OUT_BF16).ws_bytes,
                  fp8_plan(b, n, m, 0, SVDQ_OUT_BF16 | SVDQ_FP8_FAST_SUMS).ws_bytes);
}

// Codes, scales and the product's share of a whole layer's workspace.
struct Fp8Workspace {
  size_t as_off, gemm_off, total;
};
Fp8Workspace fp8_ws_layout(int rows, int m, size_t gemm) {
  const size_t G = (size_t)fp8_blocks(m);
  Fp8Workspace w;
  w.as_off = round_up(G * (size_t)rows * 128, kAlign);
  w.gemm_off = round_up(w.as_off + G * (size_t)rows, kAlign);
  w.total = w.gemm_off + gemm;
  return w;
}

// Whether no element of y lies in x's span of memory.
bool apart_from_x(const uint16_t* x, int b, int m, const EpiArgs& ep, int n, int y_dtype) {
  const uintptr_t px = (uintptr_t)x, py = (uintptr_t)ep.y;
  const uintptr_t bytes_y = ((uintptr_t)(b - 1) * ep.ldy + n) * (y_dtype == SVDQ_OUT_F32 ? 4 : 2);
  return px + (uintptr_t)b * m * 2 <= py || py + bytes_y <= px;
}

Fp8Args product_args(const uint8_t* qx, const uint8_t* ascale, const svdq_fp8_layer& L, int b, const EpiArgs& ep) {
  return Fp8Args{qx, ascale, L.qw, L.wscale, L.bias, nullptr, b, b, L.n, fp8_blocks(L.m), {nullptr, 0}, ep};
}
Fp8Args grouped_args(const uint8_t* qx, const uint8_t* ascale, int x_rows, const int32_t* row_index,
                     const int32_t* offsets, const svdq_fp8_grouped_layer& L, int b, const EpiArgs& ep) {
  return Fp8Args{qx, ascale, L.qw, L.wscale, L.bias, row_index, b, x_rows, L.n, fp8_blocks(L.m), {offsets, L.experts}, ep};
}

}  // namespace

extern "C" {

int svdq_fp8_quantize_weights(const void* W, int w_dtype, int experts, int m, int n, int transposed, uint8_t* qw,
                              uint8_t* wscale, void* stream) {
  clear_error();
  int st = check_dims(m, n);
  if (st) return st;
  REQUIRE(experts >= 1, SVDQ_ERR_INVALID_ARG, "experts must be >= 1 (got %d)", experts);
  REQUIRE(w_dtype == SVDQ_OUT_BF16 || w_dtype == SVDQ_OUT_F32, SVDQ_ERR_INVALID_ARG, "unknown w_dtype %d", w_dtype);
  REQUIRE(W && qw && wscale, SVDQ_ERR_INVALID_ARG, "W, qw and wscale must not be NULL");
  REQUIRE(element_aligned(W, w_dtype), SVDQ_ERR_ALIGNMENT, "W must be element-aligned");
  REQUIRE(aligned16(qw), SVDQ_ERR_ALIGNMENT, "qw must be 16-byte aligned");
  // a workgroup of 256 threads for each block of 16 KB of codes
  REQUIRE(experts <= SVDQ_MAX_DIM &&
              launch_fits(std::min((long long)fp8_blocks(m) * fp8_blocks(n), 1LL << 30) * experts, 256),
          SVDQ_ERR_UNSUPPORTED, "too many weights (experts=%d, m=%d, n=%d)", experts, m, n);
  return hip_status(launch_fp8_weights(W, w_dtype, experts, m, n, transposed != 0, qw, wscale, stream),
                    "fp8_quantize_weights");
}

int svdq_fp8_quantize_act(const uint16_t* x, int b, int m, uint8_t* qx, uint8_t* ascale, void* stream) {
  clear_error();
  int st = check_dims(m, 1);
  if (!st) st = check_rows(b);
  if (st || b == 0) return st;
  st = check_x(x, b, m);
  if (!st) st = check_codes(qx, ascale);
  if (st) return st;
  return hip_status(launch_fp8_act(x, b, m, qx, ascale, stream), "fp8_quantize_act");
}

size_t svdq_fp8_gemm_workspace_size(int b, int n, int m) {
  if (b <= 0 || b > SVDQ_MAX_DIM || n <= 0 || n > SVDQ_MAX_DIM || m <= 0 || m > SVDQ_MAX_DIM) return 0;
  return fp8_gemm_ws_bytes(b, n, m);
}

int svdq_fp8_gemm(const uint8_t* qx, const uint8_t* ascale, const svdq_fp8_layer* layer, const svdq_epilogue* epi, int b,
                  void* y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_product(layer, epi, b, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_codes(qx, ascale);
  const Fp8Plan plan = fp8_plan(b, layer->n, layer->m, 0, y_dtype);
  if (!st) st = check_workspace(workspace, workspace_bytes, fp8_gemm_ws_bytes(b, layer->n, layer->m), 16);
  if (st) return st;
  return hip_status(launch_fp8_gemm(product_args(qx, ascale, *layer, b, ep), plan, y_type(y_dtype), workspace, stream),
                    "fp8_gemm");
}

size_t svdq_fp8_linear_workspace_size(int b, int m, int n) {
  if (b <= 0 || b > SVDQ_MAX_DIM || n <= 0 || n > SVDQ_MAX_DIM || m <= 0 || m > SVDQ_MAX_DIM) return 0;
  return fp8_ws_layout(b, m, fp8_gemm_ws_bytes(b, n, m)).total;
}

int svdq_fp8_linear(const uint16_t* x, const svdq_fp8_layer* layer, const svdq_epilogue* epi, int b, void* y,
                    int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_product(layer, epi, b, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_x(x, b, layer->m);
  const Fp8Plan plan = fp8_plan(b, layer->n, layer->m, 0, y_dtype);
  const Fp8Workspace w = fp8_ws_layout(b, layer->m, fp8_gemm_ws_bytes(b, layer->n, layer->m));
  if (!st) st = check_workspace(workspace, workspace_bytes, w.total, kAlign);
  if (st) return st;
  uint8_t* ws = (uint8_t*)workspace;
  const int type = y_type(y_dtype);
  // few blocks of x: every workgroup of the product quantizes them itself, unless y is
  // written where x may still be read
  if (plan.rb == 1 && b <= 16 && fp8_blocks(layer->m) * b <= kFp8FusedBlocks && apart_from_x(x, b, layer->m, ep, layer->n, type))
    return hip_status(launch_fp8_rows_x(product_args(ws, ws + w.as_off, *layer, b, ep), x, layer->m, plan, type, stream),
                      "fp8_gemm");
  st = hip_status(launch_fp8_act(x, b, layer->m, ws, ws + w.as_off, stream), "fp8_quantize_act");
  if (st) return st;
  return hip_status(launch_fp8_gemm(product_args(ws, ws + w.as_off, *layer, b, ep), plan, type, ws + w.gemm_off, stream),
                    "fp8_gemm");
}

int svdq_fp8_grouped_gemm(const uint8_t* qx, const uint8_t* ascale, int x_rows, const int32_t* row_index,
                          const int32_t* offsets, const svdq_fp8_grouped_layer* layer, const svdq_epilogue* epi, int b,
                          void* y, int y_dtype, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_grouped_product(layer, epi, x_rows, row_index, offsets, b, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_codes(qx, ascale);
  if (st) return st;
  return hip_status(launch_fp8_gemm(grouped_args(qx, ascale, x_rows, row_index, offsets, *layer, b, ep),
                                    fp8_plan(b, layer->n, layer->m, layer->experts, y_dtype), y_type(y_dtype), nullptr,
                                    stream),
                    "fp8_grouped_gemm");
}

size_t svdq_fp8_grouped_linear_workspace_size(int b, int x_rows, int experts, int m, int n) {
  if (b <= 0 || b > SVDQ_MAX_DIM || x_rows <= 0 || x_rows > SVDQ_MAX_DIM || experts < 1 || experts > SVDQ_MAX_EXPERTS ||
      n <= 0 || n > SVDQ_MAX_DIM || m <= 0 || m > SVDQ_MAX_DIM)
    return 0;
  return fp8_ws_layout(x_rows, m, 0).total;
}

int svdq_fp8_grouped_linear(const uint16_t* x, int x_rows, const int32_t* row_index, const int32_t* offsets,
                            const svdq_fp8_grouped_layer* layer, const svdq_epilogue* epi, int b, void* y, int y_dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_grouped_product(layer, epi, x_rows, row_index, offsets, b, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_x(x, x_rows, layer->m);
  const Fp8Workspace w = fp8_ws_layout(x_rows, layer->m, 0);
  if (!st) st = check_workspace(workspace, workspace_bytes, w.total, kAlign);
  if (st) return st;
  uint8_t* ws = (uint8_t*)workspace;
  st = hip_status(launch_fp8_act(x, x_rows, layer->m, ws, ws + w.as_off, stream), "fp8_quantize_act");
  if (st) return st;
  return hip_status(launch_fp8_gemm(grouped_args(ws, ws + w.as_off, x_rows, row_index, offsets, *layer, b, ep),
                                    fp8_plan(b, layer->n, layer->m, layer->experts, y_dtype), y_type(y_dtype), nullptr,
                                    stream),
                    "fp8_grouped_gemm");
}

}  // extern "C"
