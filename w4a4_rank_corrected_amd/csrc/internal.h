// Internal declarations shared by the C-ABI layer, the host preparation code and
// the HIP kernel launchers.  Not part of the public ABI (include/svdq.h is).
#pragma once

#include <cstddef>
#include <cstdint>
#include <vector>

#include "svdq.h"

namespace svdq {

// ---- per-thread error message (svdq_last_error) -------------------------------
void set_error(const char* fmt, ...) __attribute__((format(printf, 1, 2)));
void clear_error();

// ---- scalar format conversions on the host (round to nearest, ties to even) ----
uint16_t f32_to_f16_sat(float f);   // fp16, saturated at +-65504
float f16_to_f32(uint16_t h);
uint16_t f64_to_bf16(double x);     // one rounding straight from fp64
float bf16_to_f32(uint16_t b);

// ---- host preparation (prep.cpp) ----------------------------------------------
// Smoothing scales of Eq.(4); lam32 / inv32 as fp32.  act_amax may be NULL.
void smoothing_lambda(const float* W, const float* act_amax, int m, int n, double alpha,
                      float* lam32, float* inv32);
// Rank-r truncated SVD of Wt (m x n, row-major fp64): L1 = U_r Sigma_r (m x r,
// row-major), L2 = V_r^T (r x n, row-major).  Returns false if it failed.
bool truncated_svd(const double* Wt, int m, int n, int r, double* L1, double* L2);
// QL iterations the SVD's eigen-solver may spend on one eigenvalue, and the
// test hook that changes it (limit < 0 restores the default); returns the
// previous limit.
constexpr int kEigIterationLimit = 60;
int set_eig_iteration_limit(int limit);
// INT4 group quantization of R (fp32 [m][n]) into group-major records.
void quantize_residual(const float* R, int m, int n, uint8_t* qw, uint16_t* wscale);
// INT8 quantization of each column of R (fp32 [m][n]) into 64-byte group-major
// records [m/64][n][64] and one fp16 scale per column.
void quantize_residual8(const float* R, int m, int n, int8_t* qw, uint16_t* wscale);
// NVFP4 quantization of each column of R (fp32 [m][n]) in blocks of 16 input
// channels with power-of-two tensor scale t: codes [m/64][n][32], E4M3 block
// scales [m/64][n][4].
void quantize_residual_fp4(const float* R, int m, int n, double t, uint8_t* qw, uint8_t* wscale);
// 2^ceil(log2(amax / (6 * 448))) (1 when amax is 0): the NVFP4 tensor scale.
double fp4_tensor_scale(double amax);

// One candidate protected layer on the host ([Review] Algorithm 1 steps 2-5).
struct HostLayer {
  double alpha = 0.5;
  std::vector<float> lam32, inv32;    // [m]
  std::vector<double> wt;             // W~ = diag(lambda) W, [m][n]
  std::vector<uint16_t> l1b, l2b;     // bf16 factors, L1 [m][r], L2 [r][n] (row-major)
  std::vector<float> r32;             // residual R = W~ - L1 L2, [m][n]
  std::vector<uint8_t> qw;            // INT4 codes of R, group-major [m/64][n][32]
  std::vector<uint16_t> wscale;       // fp16 scales [m/64][n]
};
// Steps 2-5 at migration strength alpha (act_amax NULL: lambda = 1).  Returns
// SVDQ_OK or SVDQ_ERR_NO_CONVERGENCE.
int build_layer(const float* W, const float* act_amax, int m, int n, int rank, double alpha, HostLayer& L);
// Steps 6-7: L1 L2 <- rank-r SVD of W~ - Q(R), then R and Q(R) again.
int refit_layer(int m, int n, int rank, HostLayer& L);
// Step 8's criterion: ||Y(X) - X W||_F^2 of the quantized layer on calibration
// rows x32 [b][m] (bf16 values), with X W given (fp64 [b][n]).
double layer_output_sq_error(const float* x32, int b, const double* yref, int m, int n, int rank,
                             const HostLayer& L);
// Y = X W in fp64 (x32 [b][m], W [m][n]).
void reference_output(const float* x32, int b, const float* W, int m, int n, double* y);
// Number of worker threads used by the preparation loops.
int host_threads();

// ---- device launch plan --------------------------------------------------------
// The act-quant kernel covers the rows in blocks of 64 (one 16-row strip per
// wave) and may split the channel groups of a block over `splits` workgroups;
// each split writes its own partial Z, summed in split order afterwards
// (deterministic).
// 16-column blocks of Z compiled for a rank (0, 1, 2, 3, 4, 8 or 16), and the
// LDS bytes one channel group takes in the act-quant kernel: 1/lambda (64 fp32)
// and 16 * blocks rows of L1 at a pitch of 72 bf16 (144 B, so the MFMA operand
// reads of 16 consecutive rows hit distinct banks).
constexpr int kActL1Pitch = 72;
constexpr int act_blocks(int rank) {
  return (rank + 15) / 16 <= 4 ? (rank + 15) / 16 : ((rank + 15) / 16 <= 8 ? 8 : 16);
}
constexpr int act_lds_group_bytes(int blocks) { return 256 + blocks * 16 * kActL1Pitch * 2; }
// Groups of activations each wave keeps in flight (a register ring), by the
// number of Z blocks: deeper for the light kernels, except two for ranks
// 17..32 (measured faster than four on the FLUX layers: a workgroup's first
// burst of activation loads delays the staging loads of the workgroups
// dispatched after it).
constexpr int act_depth(int blocks) { return blocks == 2 ? 2 : (blocks <= 4 ? 4 : (blocks == 8 ? 2 : 1)); }
// Groups staged in LDS at a time: the most (a multiple of the depth, at most
// 8) that fit in about 40 KB.
constexpr int act_chunk_fit(int blocks) {
  return 40960 / act_lds_group_bytes(blocks) < 8 ? 40960 / act_lds_group_bytes(blocks) : 8;
}
constexpr int act_chunk(int blocks) {
  return act_chunk_fit(blocks) - act_chunk_fit(blocks) % act_depth(blocks) > 0
             ? act_chunk_fit(blocks) - act_chunk_fit(blocks) % act_depth(blocks)
             : act_depth(blocks);
}

constexpr int kWideWavesPlan = 8;  // waves per workgroup of the wide act-quant kernel
struct ActPlan {
  int wide;              // 1: the wide kernel (16-row strips, waves over all groups, no splits)
  int strips;            // row blocks: ceil(b / 64), or ceil(b / 16) for the wide kernel
  int splits;            // workgroups per strip along the channel groups
  int groups_per_split;  // channel groups handled by one workgroup
};
ActPlan act_plan(int b, int m, int rank);

// ---- kernel launchers (HIP; return a hipError_t value, 0 = success) ------------
int launch_calibrate(const uint16_t* x, int b, int m, float* amax, int accumulate, void* stream);
// qmode: kActQuantNone (Z only), kActQuantInt4, kActQuantFp4 (tx: the power-of-
// two tensor scale of the FP4 block scales; unused otherwise).  For FP4, qx
// holds E2M1 codes in the INT4 record layout and ascale is read as bytes
// [m/64][b][4] (E4M3 block scales).
enum { kActQuantNone = 0, kActQuantInt4 = 1, kActQuantFp4 = 2 };
int launch_act_quant_down(const uint16_t* x, int b, int m, int rank, const float* smooth_inv,
                          const uint16_t* l1, uint8_t* qx, uint16_t* ascale, float* zpart,
                          const ActPlan& plan, int qmode, float tx, void* stream);
int launch_z_reduce(const float* zpart, int splits, int b, int rank, float* z, void* stream);
// Per-token INT8 codes and scales of the smoothed activations (one wave per row).
int launch_act8_quant(const uint16_t* x, int b, int m, const float* smooth_inv, int8_t* qx, uint16_t* ascale,
                      void* stream);
int launch_add(void* y, const void* t, size_t count, int y_dtype, void* stream);
int launch_lowrank_up(const float* z, const svdq_layer& L, int b, void* y, int y_dtype, void* stream);
// GEMM launch plan (plan.cpp): one tile per workgroup, or the last round's
// tiles split along the channel groups into pieces, one per workgroup, whose
// partial sums (in the workspace) a reduction kernel adds after the GEMM.
constexpr int kMaxCUs = 256;  // largest gfx950 part
struct GemmPlan {
  int tiles_m, tiles_n, G;
  int grid;             // workgroups launched
  int split;            // 1 = some tiles are split into pieces (split-K)
  int split_tiles;      // split tiles (linear tiles [0, split_tiles))
  int pieces;           // pieces per split tile
  int split_grid;       // split workgroups, split_tiles * pieces (dispatched first)
  int wg_per_cu;        // resident workgroups per CU of the kernel planned for
  int tile_n;           // output columns per tile: kGemmTileN, or kGemmTileNNarrow (INT4, few rows)
  size_t partial_bytes; // partial-sum area at the start of the workspace
  size_t ws_bytes;      // workspace bound for the shape (0 when m has too few groups to split)
};
// Operand formats of the GEMM kernel body (INT4 codes, the 8-bit setting, the
// NVFP4 setting); each has its own resident workgroups per CU.
enum GemmFormat { kFmtInt4 = 0, kFmtInt8 = 1, kFmtFp4 = 2 };
// Output tile of every GEMM build, and the resident workgroups per CU of each
// format's kernel (the same with and without split tiles).
constexpr int kGemmTileM = 128, kGemmTileN = 128;
// INT4 tiles for few rows (the wide tiles would not fill one round of slots)
constexpr int kGemmTileNNarrow = 64;
constexpr int kGemmWgPerCu[3] = {3, 3, 3};
// Split-K: pieces per split tile when full rounds of whole tiles run too
// (kMinPieces .. kMaxPieces) and when every tile is split (2 ..
// kMaxPiecesAll); each piece has at least kMinPieceGroups channel groups.
constexpr int kMinPieces = 3, kMaxPieces = 8, kMaxPiecesAll = 16, kMinPieceGroups = 8;
// The low-rank product's cost in groups: the piece that computes it (the last
// of its tile) gets this many groups fewer, so a tile's pieces end together.
constexpr int kLowRankPieceGroups = 4;
static_assert((kMaxPiecesAll - 1) * kLowRankPieceGroups < kMaxPiecesAll * (kMinPieceGroups - 1),
              "the last piece keeps at least one group");
// cus <= 0 gives the device-independent upper bound used to size workspaces
// (valid for every format); fmt selects the kernel whose residency is planned.
GemmPlan gemm_plan(int b, int n, int m, int cus, int fmt = kFmtInt4);
int device_cus();
int launch_gemm_up(const uint8_t* qx, const uint16_t* ascale, const float* z, const svdq_layer& L,
                   int b, void* y, int y_dtype, void* ws, void* stream);
int launch_gemm8_up(const int8_t* qx, const uint16_t* ascale, const float* z, const svdq_w8a8_layer& L,
                    int b, void* y, int y_dtype, void* ws, void* stream);
int launch_gemm_fp4_up(const uint8_t* qx, const uint8_t* ascale, const float* z, const svdq_fp4_layer& L, int b,
                       void* y, int y_dtype, void* ws, void* stream);
const char* hip_error_name(int err);

// ---- products with an epilogue, and grouped by expert --------------------------
// What the epilogue of a product needs, as the kernels take it: svdq_epilogue
// with its strides filled in.
struct EpiArgs {
  const uint16_t* gate;  // bf16 [ceil(b / gate_rows)][n] or NULL
  const void* residual;  // y's type, row stride ldr, or NULL
  void* y;               // row stride ldy
  int act, act_begin, gate_rows, ldr, ldy;
};
// The experts' rows of a grouped product.
struct Groups {
  const int32_t* offsets;  // device, [experts + 1]
  int experts;
};
// The most row blocks of `rows` rows that b rows sorted into `experts` experts
// can make: sum_e ceil(c_e / rows) with sum_e c_e <= b.
constexpr long long grouped_row_blocks(long long b, long long experts, long long rows) {
  const long long full = (b + experts * (rows - 1)) / rows;
  return full < b ? full : b;
}
// Rows up to which the INT4 and NVFP4 products with an epilogue use the row kernel.
constexpr int kRowsMax = 64;
// A launch of 2^32 threads or more is cut short without an error.
constexpr bool launch_fits(long long grid, long long threads) { return grid * threads < 0x100000000LL; }
// How a row kernel's workgroup is cut: nwk waves split the channel groups of the
// same columns, nwc take neighbouring column blocks.
struct RowsSplit {
  int nwk, nwc;
  long long grid;
};
RowsSplit rows_split(long long row_blocks, int n, int G, int rb);
// The kernel of a grouped product: the row kernel (rb 16-row blocks a workgroup),
// or tiles of tile_m rows x 128 columns (rb = 0); its largest launch.
struct GroupedPlan {
  int rb, tile_m;
  long long grid;
  int threads;
};
GroupedPlan grouped_plan(int b, int n, int m, int experts);
int launch_gemm_epi(const uint8_t* qx, const uint16_t* ascale, const float* z, const svdq_layer& L, int b,
                    int y_dtype, const EpiArgs& ep, void* ws, void* stream);
int launch_gemm8_epi(const int8_t* qx, const uint16_t* ascale, const float* z, const svdq_w8a8_layer& L, int b,
                     int y_dtype, const EpiArgs& ep, void* ws, void* stream);
int launch_gemm_fp4_epi(const uint8_t* qx, const uint8_t* ascale, const float* z, const svdq_fp4_layer& L, int b,
                        int y_dtype, const EpiArgs& ep, void* ws, void* stream);
int launch_grouped_gemm(const uint8_t* qx, const uint16_t* ascale, const float* z, const svdq_grouped_layer& L,
                        const int32_t* offsets, int b, int y_dtype, const EpiArgs& ep, void* stream);
// The row kernel (rows_kernels.hip), for one layer (groups.offsets NULL) or
// grouped by expert; rb = 16-row blocks per workgroup (1, 2, or 4 without groups).
struct RowsArgs {
  const uint8_t* qx;
  const uint16_t* ascale;
  const float* z;
  const uint8_t* qw;
  const uint16_t* wscale;
  const uint16_t* l2;
  const uint16_t* bias;
  int b, n, G, rank;
  Groups groups;
  EpiArgs ep;
  float txw;  // NVFP4: the product of the tensor scales
};
int launch_gemm_rows(const RowsArgs& a, int rb, int y_dtype, int fmt, void* stream);
int launch_grouped_act(const uint16_t* x, int x_rows, const int32_t* row_index, const int32_t* offsets,
                       const svdq_grouped_layer& L, int b, uint8_t* qx, uint16_t* ascale, float* z, void* stream);
int launch_combine(const void* rows, int R, int n, int dtype, const int32_t* index, const float* weight, int t, int k,
                   const void* residual, void* y, void* stream);

// ---- the routing of rows to experts ----------------------------------------------
// The sort's chunks of slots, one per workgroup (a multiple of its threads each).
constexpr int kSortThreads = 512, kSortChunk = 8 * kSortThreads;
struct SortPlan {
  int chunk, chunks;
};
SortPlan sort_plan(int b);
int launch_sort_rows(const int32_t* expert, int b, int k, int experts, int32_t* offsets, int32_t* row_index,
                     int32_t* index, void* ws, void* stream);
// The dispatch of rows x to drows (rows, dweight NULL), or the weights' gradient alone (drows NULL).
int launch_scatter_rows(const void* x, int t, int n, int dtype, const int32_t* index, const float* weight, int k,
                        const void* rows, int R, void* drows, float* dweight, void* stream);
// Workgroups of the rows' gradient, `per` rows each.
struct GradPlan {
  int per, blocks;
};
GradPlan grad_plan(int R);
// drows NULL: the weights' gradient only; dweight NULL: the rows' only.
int launch_combine_grad(const void* dy, int t, int n, int dtype, const int32_t* index, const float* weight, int k,
                        const void* rows, int R, void* drows, float* dweight, void* stream);

// ---- the 8-bit floating-point setting --------------------------------------------
constexpr int fp8_blocks(int d) { return (d + SVDQ_FP8_BLOCK - 1) / SVDQ_FP8_BLOCK; }
// Workgroups of the activation kernel: 16 rows and kFp8ActBlocks blocks of each.
constexpr int kFp8ActBlocks = 4;
constexpr long long fp8_act_grid(int b, int m) {
  return (long long)((b + 15) / 16) * ((fp8_blocks(m) + kFp8ActBlocks - 1) / kFp8ActBlocks);
}
// A product of b rows, row i's codes being row row_index[i] (or i) of the x_rows of qx.
struct Fp8Args {
  const uint8_t* qx;
  const uint8_t* ascale;
  const uint8_t* qw;
  const uint8_t* wscale;
  const uint16_t* bias;
  const int32_t* row_index;
  int b, x_rows, n, G;
  Groups groups;  // offsets NULL: one layer
  EpiArgs ep;
};
// The kernel of a product (experts 0: one layer) and its largest launch: the row
// kernel with rb 16-row blocks a workgroup; or (rb 0) tiles of 128 x 128, in `pieces`
// along the channels; or (small) of 64 x 128; or (big) the first `full` tiles of 256 x 256 and the others in
// `parts` (1: there are no others).
// fast: tiles by the 8-bit matrix instruction (SVDQ_FP8_FAST_SUMS asked for), otherwise by
// the bf16 one.  y_dtype as the C ABI takes it, flag and all; y_dtype of the launchers
// without the flag.
struct Fp8Plan {
  int rb, big, small, full, parts, pieces, threads;
  RowsSplit split;
  size_t ws_bytes;
  bool fast;
};
Fp8Plan fp8_plan(int b, int n, int m, int experts, int y_dtype);
int launch_fp8_act(const uint16_t* x, int b, int m, uint8_t* qx, uint8_t* ascale, void* stream);
int launch_fp8_weights(const void* w, int dtype, int experts, int m, int n, bool transposed, uint8_t* qw,
                       uint8_t* wscale, void* stream);
int launch_fp8_rows(const Fp8Args& a, const Fp8Plan& plan, int y_dtype, void* stream);
int launch_fp8_tiles(const Fp8Args& a, const Fp8Plan& plan, int y_dtype, void* ws, void* stream);
// The row kernel on x itself: up to 16 rows of one layer, at most kFp8FusedBlocks blocks (four
// or fewer for each 16 lanes of a workgroup, 8 KB of LDS).
constexpr int kFp8FusedBlocks = 64;
int launch_fp8_rows_x(const Fp8Args& a, const uint16_t* x, int m, const Fp8Plan& plan, int y_dtype, void* stream);
int launch_fp8_gemm(const Fp8Args& a, const Fp8Plan& plan, int y_dtype, void* ws, void* stream);
// Launcher status (not a hipError_t) of a kernel that would use scratch memory.
constexpr int kErrKernelScratch = -1000;

// Device scratch of the allocation-free entry point (scratch.hip): the
// current device's copy of a file-scope device array of kScratchBytes, its
// address looked up once per device.  Returns a hipError_t value (0 = success).
constexpr size_t kScratchBytes = (size_t)128 << 20;
int scratch_buffer(void** out);

}  // namespace svdq
