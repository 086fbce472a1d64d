// C-ABI entry points of the products with an epilogue, the layers grouped by
// expert and the combination of their rows (declared in include/svdq.h).
// Arguments are validated on the host before any HIP call or any write.
#include <algorithm>

#include "checks.h"
#include "internal.h"

using namespace svdq;

namespace {

bool element_aligned(const void* p, int dtype) {
  return ((uintptr_t)p & (dtype == SVDQ_OUT_F32 ? 3u : 1u)) == 0;
}

// Whether two row-major matrices of `rows` rows of n elements share an element
// (a, b: addresses; lda, ldb: row strides; size: bytes per element).
bool overlap(const void* a, int lda, const void* b, int ldb, int rows, int n, int size) {
  const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
  const uintptr_t bytes_a = ((uintptr_t)(rows - 1) * lda + n) * size, bytes_b = ((uintptr_t)(rows - 1) * ldb + n) * size;
  if (pa + bytes_a <= pb || pb + bytes_b <= pa) return false;
  if (lda != ldb) return true;
  // one stride: apart if the column ranges are (column slices of one tensor)
  const uintptr_t row = (uintptr_t)lda * size, off = (pa > pb ? pa - pb : pb - pa) % row, width = (uintptr_t)n * size;
  return off < width || row - off < width;
}

// Checks an epilogue for an output of b x n and fills the kernels' arguments.
int check_epilogue(const svdq_epilogue* epi, int b, int n, void* y, int y_dtype, EpiArgs* out) {
  const svdq_epilogue e = epi ? *epi : svdq_epilogue{SVDQ_ACT_NONE, 0, 0, 0, 0, nullptr, nullptr};
  REQUIRE(e.act >= SVDQ_ACT_NONE && e.act <= SVDQ_ACT_RELU, SVDQ_ERR_INVALID_ARG, "unknown activation %d", e.act);
  REQUIRE(e.act_begin >= 0 && e.act_begin <= n, SVDQ_ERR_INVALID_ARG, "act_begin must be in [0, %d] (got %d)", n,
          e.act_begin);
  REQUIRE(e.gate_rows >= 0, SVDQ_ERR_INVALID_ARG, "gate_rows must be >= 0 (got %d)", e.gate_rows);
  REQUIRE(e.ldy == 0 || (e.ldy >= n && e.ldy <= SVDQ_MAX_DIM), SVDQ_ERR_INVALID_ARG,
          "ldy must be 0 or in [%d, %d] (got %d)", n, SVDQ_MAX_DIM, e.ldy);
  REQUIRE(e.ldr == 0 || (e.ldr >= n && e.ldr <= SVDQ_MAX_DIM), SVDQ_ERR_INVALID_ARG,
          "ldr must be 0 or in [%d, %d] (got %d)", n, SVDQ_MAX_DIM, e.ldr);
  const int ldy = e.ldy ? e.ldy : n, ldr = e.ldr ? e.ldr : n;
  REQUIRE(((uintptr_t)e.gate & 1u) == 0, SVDQ_ERR_ALIGNMENT, "gate must be 2-byte aligned");
  REQUIRE(element_aligned(e.residual, y_dtype), SVDQ_ERR_ALIGNMENT, "residual must be element-aligned");
  const int size = y_dtype == SVDQ_OUT_F32 ? 4 : 2;
  if (e.residual && b > 0 && !(e.residual == y && (ldr == ldy || b == 1)))
    REQUIRE(!overlap(e.residual, ldr, y, ldy, b, n, size), SVDQ_ERR_INVALID_ARG,
            "residual overlaps y without being y itself");
  out->gate = e.gate;
  out->residual = e.residual;
  out->y = y;
  out->act = e.act_begin < n ? e.act : SVDQ_ACT_NONE;
  out->act_begin = e.act_begin;
  out->gate_rows = e.gate_rows ? e.gate_rows : std::max(b, 1);
  out->ldr = ldr;
  out->ldy = ldy;
  return SVDQ_OK;
}

int check_rows(int b) {
  REQUIRE(b >= 0, SVDQ_ERR_INVALID_ARG, "b must be >= 0 (got %d)", b);
  REQUIRE(b <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "b must be <= %d (got %d)", SVDQ_MAX_DIM, b);
  return SVDQ_OK;
}

int check_workspace(const void* ws, size_t have, size_t need, uintptr_t align) {
  if (need == 0) return SVDQ_OK;
  REQUIRE(ws != nullptr && have >= need, SVDQ_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need,
          ws ? have : (size_t)0);
  REQUIRE(((uintptr_t)ws & (align - 1)) == 0, SVDQ_ERR_ALIGNMENT, "workspace must be %zu-byte aligned", (size_t)align);
  return SVDQ_OK;
}

// The product's activation-side operands.
int check_operands(const void* qx, const void* ascale, const float* z, int rank, uintptr_t scale_align) {
  REQUIRE(qx && ascale, SVDQ_ERR_INVALID_ARG, "qx and ascale must not be NULL");
  REQUIRE(aligned16(qx), SVDQ_ERR_ALIGNMENT, "qx must be 16-byte aligned");
  REQUIRE(((uintptr_t)ascale & (scale_align - 1)) == 0, SVDQ_ERR_ALIGNMENT, "ascale must be %zu-byte aligned",
          (size_t)scale_align);
  if (rank > 0) {
    REQUIRE(z != nullptr, SVDQ_ERR_INVALID_ARG, "z must not be NULL when rank > 0");
    REQUIRE(((uintptr_t)z & 3u) == 0, SVDQ_ERR_ALIGNMENT, "z must be 4-byte aligned");
  }
  return SVDQ_OK;
}

// What the whole layers need besides the product.
int check_input(const uint16_t* x, const float* smooth_inv, const uint16_t* l1, int rank) {
  REQUIRE(x != nullptr, SVDQ_ERR_INVALID_ARG, "x must not be NULL");
  REQUIRE(aligned16(x), SVDQ_ERR_ALIGNMENT, "x must be 16-byte aligned");
  REQUIRE(aligned16(smooth_inv), SVDQ_ERR_ALIGNMENT, "smooth_inv must be 16-byte aligned");
  if (rank > 0) {
    REQUIRE(l1 != nullptr, SVDQ_ERR_INVALID_ARG, "layer l1 must not be NULL when rank > 0");
    REQUIRE(aligned16(l1), SVDQ_ERR_ALIGNMENT, "layer l1 must be 16-byte aligned");
  }
  return SVDQ_OK;
}

// Dimensions of an experts' layer; the tensors are checked where they are used.
int check_grouped(const svdq_grouped_layer* L) {
  REQUIRE(L != nullptr, SVDQ_ERR_INVALID_ARG, "layer is NULL");
  REQUIRE(L->experts >= 1, SVDQ_ERR_INVALID_ARG, "experts must be >= 1 (got %d)", L->experts);
  REQUIRE(L->experts <= SVDQ_MAX_EXPERTS, SVDQ_ERR_UNSUPPORTED, "experts must be <= %d (got %d)", SVDQ_MAX_EXPERTS,
          L->experts);
  int st = check_group(L->m, L->group);
  if (st) return st;
  REQUIRE(L->n >= 1, SVDQ_ERR_INVALID_ARG, "n must be >= 1 (got %d)", L->n);
  REQUIRE(L->n <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "n must be <= %d (got %d)", SVDQ_MAX_DIM, L->n);
  REQUIRE(L->rank >= 0 && L->rank <= SVDQ_MAX_RANK, SVDQ_ERR_UNSUPPORTED, "rank must be in [0, %d] (got %d)",
          SVDQ_MAX_RANK, L->rank);
  return SVDQ_OK;
}

int check_grouped_act(const uint16_t* x, int x_rows, const int32_t* row_index, const int32_t* offsets,
                      const svdq_grouped_layer* L, int b) {
  REQUIRE(offsets != nullptr, SVDQ_ERR_INVALID_ARG, "offsets must not be NULL");
  REQUIRE(((uintptr_t)offsets & 3u) == 0 && ((uintptr_t)row_index & 3u) == 0, SVDQ_ERR_ALIGNMENT,
          "offsets and row_index must be 4-byte aligned");
  REQUIRE(x_rows >= 1 && (row_index || x_rows >= b), SVDQ_ERR_INVALID_ARG,
          "x_rows must be >= 1, and >= b without a row_index (got %d)", x_rows);
  REQUIRE(x_rows <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "x_rows must be <= %d (got %d)", SVDQ_MAX_DIM, x_rows);
  return check_input(x, L->smooth_inv, L->l1, L->rank);
}

int check_grouped_gemm(const int32_t* offsets, const svdq_grouped_layer* L, const svdq_epilogue* epi, int b, void* y,
                       int y_dtype, EpiArgs* ep) {
  REQUIRE(offsets != nullptr, SVDQ_ERR_INVALID_ARG, "offsets must not be NULL");
  REQUIRE(((uintptr_t)offsets & 3u) == 0, SVDQ_ERR_ALIGNMENT, "offsets must be 4-byte aligned");
  REQUIRE(L->qw && L->wscale, SVDQ_ERR_INVALID_ARG, "layer qw / wscale must not be NULL");
  REQUIRE(aligned16(L->qw), SVDQ_ERR_ALIGNMENT, "layer qw must be 16-byte aligned");
  REQUIRE(((uintptr_t)L->wscale & 1u) == 0, SVDQ_ERR_ALIGNMENT, "layer wscale must be 2-byte aligned");
  REQUIRE(L->rank == 0 || L->l2, SVDQ_ERR_INVALID_ARG, "layer l2 must not be NULL when rank > 0");
  REQUIRE(((uintptr_t)L->l2 & 1u) == 0 && ((uintptr_t)L->bias & 1u) == 0, SVDQ_ERR_ALIGNMENT,
          "layer l2 and bias must be 2-byte aligned");
  REQUIRE(!epi || (!epi->gate && !epi->residual), SVDQ_ERR_UNSUPPORTED,
          "a grouped product takes no gate and no residual");
  // (fewer than 2^32 threads are fewer than 2^26 tiles: 32-bit tile numbers serve)
  const GroupedPlan plan = grouped_plan(b, L->n, L->m, L->experts);
  REQUIRE(launch_fits(plan.grid, plan.threads), SVDQ_ERR_UNSUPPORTED,
          "too many output tiles (b=%d, n=%d, experts=%d)", b, L->n, L->experts);
  return check_epilogue(epi, b, L->n, y, y_dtype, ep);
}

struct GroupedWorkspace {
  size_t as_off, z_off, total;
};
GroupedWorkspace grouped_ws_layout(int b, int m, int rank) {
  GroupedWorkspace w;
  const size_t G = (size_t)(m / SVDQ_GROUP);
  w.as_off = round_up(G * (size_t)b * 32, kAlign);
  w.z_off = round_up(w.as_off + G * (size_t)b * 2, kAlign);
  w.total = round_up(w.z_off + (size_t)b * (size_t)rank * 4, kAlign);
  return w;
}

// The INT4 activation kernels of svdq_linear on its workspace layout.
int run_act4(const uint16_t* x, const svdq_layer* layer, int b, char* ws, const LinearWorkspace& w, void* stream) {
  const int m = layer->m, rank = layer->rank;
  const ActPlan p = act_plan(b, m, rank);
  float* z = rank > 0 ? (float*)(ws + w.z_off) : nullptr;
  float* zpart = (rank > 0 && p.splits > 1) ? (float*)(ws + w.zpart_off) : z;
  int st = hip_status(launch_act_quant_down(x, b, m, rank, layer->smooth_inv, layer->l1, (uint8_t*)(ws + w.qx_off),
                                            (uint16_t*)(ws + w.as_off), zpart, p, kActQuantInt4, 1.0f, stream),
                      "act_quant_lowrank_down");
  if (st || rank == 0 || p.splits <= 1) return st;
  return hip_status(launch_z_reduce(zpart, p.splits, b, rank, z, stream), "z_reduce");
}

// INT4 and NVFP4: the row kernel takes no workspace.
size_t gemm_epi_ws_bytes(int b, int n, int m) { return b <= kRowsMax ? 0 : gemm_ws_bytes(b, n, m); }
size_t linear_epi_ws_bytes(const LinearWorkspace& w, int b) { return b <= kRowsMax ? w.gemm_off : w.total; }

bool linear_dims_ok(int b, int m, int n, int rank) {
  return b > 0 && b <= SVDQ_MAX_DIM && n > 0 && n <= SVDQ_MAX_DIM && m >= SVDQ_GROUP && m % SVDQ_GROUP == 0 &&
         rank >= 0 && rank <= SVDQ_MAX_RANK;
}

}  // namespace

extern "C" {

size_t svdq_gemm_epi_workspace_size(int b, int n, int m) {
  if (b <= 0 || b > SVDQ_MAX_DIM || n <= 0 || n > SVDQ_MAX_DIM || m < SVDQ_GROUP || m % SVDQ_GROUP) return 0;
  return gemm_epi_ws_bytes(b, n, m);
}

int svdq_gemm_w4a4_lowrank_up_epi(const uint8_t* qx, const uint16_t* ascale, const float* z, const svdq_layer* layer,
                                  const svdq_epilogue* epi, int b, void* y, int y_dtype, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_layer(layer);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_dtype, b);
  if (!st) st = check_epilogue(epi, b, layer->n, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_operands(qx, ascale, z, layer->rank, 2);
  if (!st) st = check_workspace(workspace, workspace_bytes, gemm_epi_ws_bytes(b, layer->n, layer->m), 16);
  if (st) return st;
  return hip_status(launch_gemm_epi(qx, ascale, z, *layer, b, y_dtype, ep, workspace, stream), "gemm_w4a4_epi");
}

int svdq_w8a8_gemm_lowrank_up_epi(const int8_t* qx, const uint16_t* ascale, const float* z,
                                  const svdq_w8a8_layer* layer, const svdq_epilogue* epi, int b, void* y, int y_dtype,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_layer8(layer);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_dtype, b);
  if (!st) st = check_epilogue(epi, b, layer->n, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_operands(qx, ascale, z, layer->rank, 2);
  if (!st) st = check_workspace(workspace, workspace_bytes, gemm_ws_bytes(b, layer->n, layer->m), 16);
  if (st) return st;
  return hip_status(launch_gemm8_epi(qx, ascale, z, *layer, b, y_dtype, ep, workspace, stream), "gemm_w8a8_epi");
}

int svdq_fp4_gemm_lowrank_up_epi(const uint8_t* qx, const uint8_t* ascale, const float* z, const svdq_fp4_layer* layer,
                                 const svdq_epilogue* epi, int b, void* y, int y_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_layer_fp4(layer);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_dtype, b);
  if (!st) st = check_epilogue(epi, b, layer->n, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_operands(qx, ascale, z, layer->rank, 2);
  if (!st) st = check_workspace(workspace, workspace_bytes, gemm_epi_ws_bytes(b, layer->n, layer->m), 16);
  if (st) return st;
  return hip_status(launch_gemm_fp4_epi(qx, ascale, z, *layer, b, y_dtype, ep, workspace, stream), "gemm_fp4_epi");
}

size_t svdq_linear_epi_workspace_size(int b, int m, int n, int rank) {
  return linear_dims_ok(b, m, n, rank) ? linear_epi_ws_bytes(linear_ws_layout(b, m, n, rank), b) : 0;
}

size_t svdq_fp4_linear_epi_workspace_size(int b, int m, int n, int rank) {
  return linear_dims_ok(b, m, n, rank) ? linear_epi_ws_bytes(linear_fp4_ws_layout(b, m, n, rank), b) : 0;
}

int svdq_linear_epi(const uint16_t* x, const svdq_layer* layer, const svdq_epilogue* epi, int b, void* y, int y_dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  bool done = false;
  EpiArgs ep;
  int st = check_linear(x, layer, b, y, y_dtype, &done);
  if (!st) st = check_epilogue(epi, b, layer->n, y, y_dtype, &ep);
  if (st || done) return st;
  const LinearWorkspace w = linear_ws_layout(b, layer->m, layer->n, layer->rank);
  st = check_workspace(workspace, workspace_bytes, linear_epi_ws_bytes(w, b), kAlign);
  if (st) return st;
  char* ws = (char*)workspace;
  st = run_act4(x, layer, b, ws, w, stream);
  if (st) return st;
  return hip_status(launch_gemm_epi((uint8_t*)(ws + w.qx_off), (uint16_t*)(ws + w.as_off),
                                    layer->rank > 0 ? (float*)(ws + w.z_off) : nullptr, *layer, b, y_dtype, ep,
                                    ws + w.gemm_off, stream),
                    "gemm_w4a4_epi");
}

int svdq_w8a8_linear_epi(const uint16_t* x, const svdq_w8a8_layer* layer, const svdq_epilogue* epi, int b, void* y,
                         int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_layer8(layer);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_dtype, b);
  if (!st) st = check_epilogue(epi, b, layer->n, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_input(x, layer->smooth_inv, layer->l1, layer->rank);
  if (st) return st;
  const LinearWorkspace w = linear8_ws_layout(b, layer->m, layer->n, layer->rank);
  st = check_workspace(workspace, workspace_bytes, w.total, kAlign);
  if (st) return st;
  char* ws = (char*)workspace;
  int8_t* qx = (int8_t*)(ws + w.qx_off);
  uint16_t* as = (uint16_t*)(ws + w.as_off);
  float* z = layer->rank > 0 ? (float*)(ws + w.z_off) : nullptr;
  st = run_act8(x, b, layer->m, layer->rank, layer->smooth_inv, layer->l1, qx, as, z, (float*)(ws + w.zpart_off), stream);
  if (st) return st;
  return hip_status(launch_gemm8_epi(qx, as, z, *layer, b, y_dtype, ep, ws + w.gemm_off, stream), "gemm_w8a8_epi");
}

int svdq_fp4_linear_epi(const uint16_t* x, const svdq_fp4_layer* layer, const svdq_epilogue* epi, int b, void* y,
                        int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_layer_fp4(layer);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_dtype, b);
  if (!st) st = check_epilogue(epi, b, layer->n, y, y_dtype, &ep);
  if (st || b == 0) return st;
  st = check_input(x, layer->smooth_inv, layer->l1, layer->rank);
  if (st) return st;
  const LinearWorkspace w = linear_fp4_ws_layout(b, layer->m, layer->n, layer->rank);
  st = check_workspace(workspace, workspace_bytes, linear_epi_ws_bytes(w, b), kAlign);
  if (st) return st;
  char* ws = (char*)workspace;
  uint8_t* qx = (uint8_t*)(ws + w.qx_off);
  uint8_t* as = (uint8_t*)(ws + w.as_off);
  float* z = layer->rank > 0 ? (float*)(ws + w.z_off) : nullptr;
  st = run_act_fp4(x, b, layer->m, layer->rank, layer->smooth_inv, layer->l1, layer->t_x, qx, as, z,
                   (float*)(ws + w.zpart_off), stream);
  if (st) return st;
  return hip_status(launch_gemm_fp4_epi(qx, as, z, *layer, b, y_dtype, ep, ws + w.gemm_off, stream), "gemm_fp4_epi");
}

int svdq_grouped_quantize_act_lowrank_down(const uint16_t* x, int x_rows, const int32_t* row_index,
                                           const int32_t* offsets, const svdq_grouped_layer* layer, int b, uint8_t* qx,
                                           uint16_t* ascale, float* z, void* stream) {
  clear_error();
  int st = check_grouped(layer);
  if (!st) st = check_rows(b);
  if (st || b == 0) return st;
  st = check_grouped_act(x, x_rows, row_index, offsets, layer, b);
  if (!st) st = check_operands(qx, ascale, z, layer->rank, 2);
  if (st) return st;
  return hip_status(launch_grouped_act(x, x_rows, row_index, offsets, *layer, b, qx, ascale, z, stream),
                    "grouped_act_quant");
}

int svdq_grouped_gemm_w4a4_lowrank_up(const uint8_t* qx, const uint16_t* ascale, const float* z,
                                      const int32_t* offsets, const svdq_grouped_layer* layer,
                                      const svdq_epilogue* epi, int b, void* y, int y_dtype, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_grouped(layer);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_dtype, b);
  if (st || b == 0) return st;
  st = check_grouped_gemm(offsets, layer, epi, b, y, y_dtype, &ep);
  if (!st) st = check_operands(qx, ascale, z, layer->rank, 2);
  if (st) return st;
  return hip_status(launch_grouped_gemm(qx, ascale, z, *layer, offsets, b, y_dtype, ep, stream), "grouped_gemm_w4a4");
}

size_t svdq_grouped_linear_workspace_size(int b, int experts, int m, int n, int rank) {
  if (b <= 0 || b > SVDQ_MAX_DIM || experts < 1 || n < 1 || m < SVDQ_GROUP || m % SVDQ_GROUP || rank < 0 ||
      rank > SVDQ_MAX_RANK)
    return 0;
  return grouped_ws_layout(b, m, rank).total;
}

int svdq_grouped_linear(const uint16_t* x, int x_rows, const int32_t* row_index, const int32_t* offsets,
                        const svdq_grouped_layer* layer, const svdq_epilogue* epi, int b, void* y, int y_dtype,
                        void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  EpiArgs ep;
  int st = check_grouped(layer);
  if (!st) st = check_rows(b);
  if (!st) st = check_y(y, y_dtype, b);
  if (st || b == 0) return st;
  st = check_grouped_act(x, x_rows, row_index, offsets, layer, b);
  if (!st) st = check_grouped_gemm(offsets, layer, epi, b, y, y_dtype, &ep);
  if (st) return st;
  const GroupedWorkspace w = grouped_ws_layout(b, layer->m, layer->rank);
  st = check_workspace(workspace, workspace_bytes, w.total, kAlign);
  if (st) return st;
  char* ws = (char*)workspace;
  uint8_t* qx = (uint8_t*)ws;
  uint16_t* as = (uint16_t*)(ws + w.as_off);
  float* z = layer->rank > 0 ? (float*)(ws + w.z_off) : nullptr;
  st = hip_status(launch_grouped_act(x, x_rows, row_index, offsets, *layer, b, qx, as, z, stream), "grouped_act_quant");
  if (st) return st;
  return hip_status(launch_grouped_gemm(qx, as, z, *layer, offsets, b, y_dtype, ep, stream), "grouped_gemm_w4a4");
}

int svdq_combine_rows(const void* rows, int R, int n, int dtype, const int32_t* index, const float* weight, int t,
                      int k, const void* residual, void* y, void* stream) {
  clear_error();
  REQUIRE(R >= 0 && n >= 1 && t >= 0 && k >= 1, SVDQ_ERR_INVALID_ARG,
          "need R >= 0, n >= 1, t >= 0 and k >= 1 (got R=%d n=%d t=%d k=%d)", R, n, t, k);
  REQUIRE(R <= SVDQ_MAX_DIM && n <= SVDQ_MAX_DIM && t <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "R, n and t must be <= %d",
          SVDQ_MAX_DIM);
  REQUIRE(k <= SVDQ_MAX_EXPERTS, SVDQ_ERR_UNSUPPORTED, "k must be <= %d (got %d)", SVDQ_MAX_EXPERTS, k);
  int st = check_y(y, dtype, t);
  if (st || t == 0) return st;
  REQUIRE((rows || R == 0) && index, SVDQ_ERR_INVALID_ARG, "rows and index must not be NULL");
  REQUIRE(element_aligned(rows, dtype) && element_aligned(residual, dtype), SVDQ_ERR_ALIGNMENT,
          "rows and residual must be element-aligned");
  REQUIRE((((uintptr_t)index | (uintptr_t)weight) & 3u) == 0, SVDQ_ERR_ALIGNMENT,
          "index and weight must be 4-byte aligned");
  // 512 G elements: more than any device's memory
  REQUIRE((long long)t * n <= 1LL << 39, SVDQ_ERR_UNSUPPORTED, "t x n is too large (t=%d, n=%d)", t, n);
  const int size = dtype == SVDQ_OUT_F32 ? 4 : 2;
  const uintptr_t row = (uintptr_t)n * size, py = (uintptr_t)y, pr = (uintptr_t)rows, ps = (uintptr_t)residual;
  const uintptr_t end = py + (uintptr_t)t * row;
  REQUIRE(R == 0 || pr + (uintptr_t)R * row <= py || end <= pr, SVDQ_ERR_INVALID_ARG, "y overlaps rows");
  REQUIRE(!residual || ps == py || ps + (uintptr_t)t * row <= py || end <= ps, SVDQ_ERR_INVALID_ARG,
          "residual overlaps y without being y itself");
  return hip_status(launch_combine(rows, R, n, dtype, index, weight, t, k, residual, y, stream), "combine_rows");
}

}  // extern "C"
