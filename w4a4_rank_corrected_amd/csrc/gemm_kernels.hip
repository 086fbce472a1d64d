// Fused W4A4 GEMM + low-rank up-projection (second fused pair of Nunchaku).
//
// [Review] = "SVDQuant: How a Small High-Precision Branch Makes 4-Bit Diffusion
// Practical" (technical review of arXiv:2411.05007v4): sec. 4.2 Eq.(7),
// sec. 6.1 Algorithm 2 steps 4-8 and Fig. 4 second pair.
// [Nunchaku] = "SVDQuant: 4-bit Quantization Enables Efficient Diffusion Model
// Inference on Consumer GPUs", section "Nunchaku": two 4-bit values per byte,
// unpacked with bit operations.
//
// Y[i,j] = sum_g sx[g,i] sw[g,j] isum[i,j,g] + (bf16(Z) L2)[i,j] + bias[j]
//
// Exact per-group integer sums on i8 MFMA: a nibble is unpacked to the byte
// 16*q (mask for the high nibble, shift-and-mask for the low one), so one
// v_mfma_i32_16x16x64_i8 over exactly one 64-channel group yields 256*isum.
// The MFMA accumulator is seeded with the bits of 1.5*2^23, so the result read
// as a float is 1.5*2^23 + 256*isum exactly (|256*isum| <= 802816 < 2^22).  Two
// FMAs then apply the scales:
//   t   = fma(r, sx/256, -1.5*2^23 * sx/256) = isum * sx   (exact: <= 23 bits)
//   acc = fma(t, sw, acc)                                 (one rounding)
// The low-rank branch initialises the accumulators with bf16 MFMAs.
//
// The two FMAs per (output element, group) make the kernel VALU-bound on
// gfx950 (a 16x16x64 i8 MFMA covers 256 element-groups in 16 cycles; their 8
// wave64 FMAs need 32), and only about 40 % of an MFMA's time overlaps VALU
// work, whether the two come from one wave or from different waves (measured
// with a microbenchmark).  The work decomposition therefore aims at keeping
// the VALU busy: three waves per SIMD to cover each other's latencies,
// unpacking each code once per workgroup, few LDS reads of scales, and few
// barriers.
//
// Work decomposition (gfx950: 256 CUs in 8 XCDs, 4 SIMDs per CU, wave64),
// parameterised by GemmCfg:
//   a workgroup computes TM x TN tiles of Y (rows x columns) with
//   (TM/WM) x (TN/WN) waves, each owning a WM x WN sub-tile of 16x16 MFMA
//   blocks.  Per 64-channel group it loads the packed activation and weight
//   records (contiguous in the group-major layout) with buffer loads, unpacks
//   them once into LDS (double-buffered), and every wave reads its MFMA
//   operands from there.  Global loads run DEPTH groups ahead in registers.
//   Measured alternatives that were not faster on gfx950: 256 x 256 and
//   128 x 256 tiles (register spills or fewer resident waves), 128 x 64 tiles
//   at three or four waves per SIMD (more staging and LDS traffic per output),
//   and explicit MFMA/FMA interleaving hints (the resident workgroups
//   already interleave).
//
// Schedules (tile = TM x TN outputs over all G groups; slots = the resident
// workgroups of all CUs, three per CU):
//   * one whole tile per workgroup, when the tiles fill whole rounds of slots
//     or their last round is more than a third full;
//   * otherwise the tiles of the last round are split along the channel
//     groups into k pieces each, one piece per workgroup (split workgroups
//     first in the grid, then the full rounds of whole tiles).  A piece
//     stores its sums in a partial slot of the workspace and ends; a
//     reduction kernel launched next on the same stream adds each tile's k
//     slots in piece order, applies the epilogue and stores the tile.  No
//     workgroup waits for or signals another (the kernel boundary orders the
//     slots' stores before their loads), so correctness does not depend on
//     the order or residency in which workgroups are dispatched, and results
//     are deterministic for a shape and CU count.  Device-scope atomics and
//     coherent loads, the alternative inside one kernel, measured 4-5 us per
//     round trip here: the last piece of a 256-row FLUX tile spent 35 us
//     adding eight 64 KB slots.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_body.h"
#include "launch.h"

#pragma clang fp contract(off)

namespace svdq {
namespace {

using namespace dev;

template <class C, bool OUT_BF16, bool SK>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WPE, C::WPE))) void gemm_w4a4_up_kernel(
    const uint8_t* __restrict__ qx, const uint16_t* __restrict__ ascale,
    const float* __restrict__ z, const uint8_t* __restrict__ qw,
    const uint16_t* __restrict__ wscale, const uint16_t* __restrict__ l2t,
    const uint16_t* __restrict__ bias, int b, int n, int G, int rank, int tiles_m, int tiles_n,
    void* __restrict__ yout, SplitK sk, float txw) {
  gemm_up_body<C, OUT_BF16, kFmtInt4, SK>(qx, ascale, z, qw, wscale, l2t, bias, b, n, G, rank, tiles_m, tiles_n,
                                          yout, sk, txw);
}

template <class C, bool OUT_BF16, bool SK>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WPE, C::WPE))) void gemm_w8a8_up_kernel(
    const uint8_t* __restrict__ qx, const uint16_t* __restrict__ ascale,
    const float* __restrict__ z, const uint8_t* __restrict__ qw,
    const uint16_t* __restrict__ wscale, const uint16_t* __restrict__ l2t,
    const uint16_t* __restrict__ bias, int b, int n, int G, int rank, int tiles_m, int tiles_n,
    void* __restrict__ yout, SplitK sk, float txw) {
  gemm_up_body<C, OUT_BF16, kFmtInt8, SK>(qx, ascale, z, qw, wscale, l2t, bias, b, n, G, rank, tiles_m, tiles_n,
                                          yout, sk, txw);
}

template <class C, bool OUT_BF16, bool SK>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WPE, C::WPE))) void gemm_fp4_up_kernel(
    const uint8_t* __restrict__ qx, const uint16_t* __restrict__ ascale,
    const float* __restrict__ z, const uint8_t* __restrict__ qw,
    const uint16_t* __restrict__ wscale, const uint16_t* __restrict__ l2t,
    const uint16_t* __restrict__ bias, int b, int n, int G, int rank, int tiles_m, int tiles_n,
    void* __restrict__ yout, SplitK sk, float txw) {
  gemm_up_body<C, OUT_BF16, kFmtFp4, SK>(qx, ascale, z, qw, wscale, l2t, bias, b, n, G, rank, tiles_m, tiles_n,
                                         yout, sk, txw);
}

int g_num_cus = 0;
template <bool OUT_BF16, int FMT>
int launch_typed(const uint8_t* qx, const uint16_t* ascale, const float* z, const Operands& L, int b,
                 void* y, const GemmPlan& plan, void* ws, hipStream_t st, float txw = 1.0f) {
  SplitK sk{0, 0, 1, 0, nullptr};
  if (plan.split) {
    sk.P = plan.split_grid;
    sk.T = plan.split_tiles;
    sk.k = plan.pieces;
    // about one memory round trip of its loads, measured at 4-6 us, the time
    // of 4 groups at three workgroups per CU; (k - 1) lr < G - k holds since
    // every piece has at least kMinPieceGroups groups
    sk.lr = L.rank > 0 ? kLowRankPieceGroups : 0;
    sk.partials = reinterpret_cast<float*>(ws);
  }
#define SVDQ_GEMM_ARGS qx, ascale, z, L.qw, L.wscale, L.l2, L.bias, b, L.n, plan.G, L.rank, plan.tiles_m, \
                       plan.tiles_n, y, sk, txw
  int st_gemm;
  if constexpr (FMT == kFmtInt8) {
    st_gemm = plan.split
                  ? launch_checked(gemm_w8a8_up_kernel<Cfg8, OUT_BF16, true>, plan.grid, Cfg8::NT, st, SVDQ_GEMM_ARGS)
                  : launch_checked(gemm_w8a8_up_kernel<Cfg8, OUT_BF16, false>, plan.grid, Cfg8::NT, st, SVDQ_GEMM_ARGS);
  } else if constexpr (FMT == kFmtFp4) {
    // the planner never splits NVFP4 tiles (its split build exceeds the
    // register budget of three workgroups per CU)
    if (plan.split) return (int)hipErrorInvalidValue;
    st_gemm = launch_checked(gemm_fp4_up_kernel<CfgF4, OUT_BF16, false>, plan.grid, CfgF4::NT, st, SVDQ_GEMM_ARGS);
  } else if (plan.tile_n == CfgN::TN) {
    st_gemm = plan.split
                  ? launch_checked(gemm_w4a4_up_kernel<CfgN, OUT_BF16, true>, plan.grid, CfgN::NT, st, SVDQ_GEMM_ARGS)
                  : launch_checked(gemm_w4a4_up_kernel<CfgN, OUT_BF16, false>, plan.grid, CfgN::NT, st, SVDQ_GEMM_ARGS);
  } else {
    st_gemm = plan.split
                  ? launch_checked(gemm_w4a4_up_kernel<Cfg, OUT_BF16, true>, plan.grid, Cfg::NT, st, SVDQ_GEMM_ARGS)
                  : launch_checked(gemm_w4a4_up_kernel<Cfg, OUT_BF16, false>, plan.grid, Cfg::NT, st, SVDQ_GEMM_ARGS);
  }
#undef SVDQ_GEMM_ARGS
  if (st_gemm != 0 || !plan.split) return st_gemm;
  const int lr_slot = FMT == kFmtInt8 && L.rank > 0 ? 1 : 0;
  auto reduce = [&](auto cfg) {
    using C = decltype(cfg);
    constexpr int UNITS = C::TM * C::TN / 4;
    return launch_checked(splitk_reduce_kernel<C, FMT, OUT_BF16>, (int)(((long long)sk.T * UNITS + 255) / 256),
                          256, st, (const float*)sk.partials, sk.T, sk.k, plan.tiles_m, plan.tiles_n, b, L.n,
                          ascale, L.wscale, lr_slot, L.bias, y, EpiArgs{});
  };
  if constexpr (FMT == kFmtFp4) {
    return st_gemm;
  } else if constexpr (FMT == kFmtInt8) {
    return reduce(Cfg8{});
  } else {
    return plan.tile_n == CfgN::TN ? reduce(CfgN{}) : reduce(Cfg{});
  }
}

}  // namespace

// The launch plan (gemm_plan) is host logic in plan.cpp; the kernel builds
// here must match the tiling and residencies it plans for.
static_assert(Cfg::TM == kGemmTileM && Cfg::TN == kGemmTileN && CfgN::TM == kGemmTileM &&
                  CfgN::TN == kGemmTileNNarrow && CfgN::WG_PER_CU == Cfg::WG_PER_CU,
              "tile shapes");
static_assert(Cfg::TM == Cfg8::TM && Cfg::TN == Cfg8::TN && Cfg::TM == CfgF4::TM && Cfg::TN == CfgF4::TN,
              "one tiling for every setting");
static_assert(Cfg::WG_PER_CU == kGemmWgPerCu[kFmtInt4] && Cfg8::WG_PER_CU == kGemmWgPerCu[kFmtInt8] &&
                  CfgF4::WG_PER_CU == kGemmWgPerCu[kFmtFp4],
              "resident workgroups per CU of each build");

int device_cus() {
  if (g_num_cus == 0) {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) == hipSuccess &&
        hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && v > 0)
      g_num_cus = std::min(v, kMaxCUs);
    else
      g_num_cus = kMaxCUs;
  }
  return g_num_cus;
}

int launch_gemm_up(const uint8_t* qx, const uint16_t* ascale, const float* z, const svdq_layer& L,
                   int b, void* y, int y_dtype, void* ws, void* stream) {
  const GemmPlan plan = gemm_plan(b, L.n, L.m, device_cus());
  const Operands o{L.qw, L.wscale, L.l2, L.bias, L.n, L.rank};
  hipStream_t st = (hipStream_t)stream;
  if (y_dtype == SVDQ_OUT_BF16) return launch_typed<true, kFmtInt4>(qx, ascale, z, o, b, y, plan, ws, st);
  return launch_typed<false, kFmtInt4>(qx, ascale, z, o, b, y, plan, ws, st);
}

int launch_gemm8_up(const int8_t* qx, const uint16_t* ascale, const float* z, const svdq_w8a8_layer& L,
                    int b, void* y, int y_dtype, void* ws, void* stream) {
  const GemmPlan plan = gemm_plan(b, L.n, L.m, device_cus(), kFmtInt8);
  const Operands o{reinterpret_cast<const uint8_t*>(L.qw), L.wscale, L.l2, L.bias, L.n, L.rank};
  const uint8_t* a = reinterpret_cast<const uint8_t*>(qx);
  hipStream_t st = (hipStream_t)stream;
  if (y_dtype == SVDQ_OUT_BF16) return launch_typed<true, kFmtInt8>(a, ascale, z, o, b, y, plan, ws, st);
  return launch_typed<false, kFmtInt8>(a, ascale, z, o, b, y, plan, ws, st);
}

int launch_gemm_fp4_up(const uint8_t* qx, const uint8_t* ascale, const float* z, const svdq_fp4_layer& L, int b,
                       void* y, int y_dtype, void* ws, void* stream) {
  const GemmPlan plan = gemm_plan(b, L.n, L.m, device_cus(), kFmtFp4);
  const Operands o{L.qw, reinterpret_cast<const uint16_t*>(L.wscale), L.l2, L.bias, L.n, L.rank};
  const uint16_t* as = reinterpret_cast<const uint16_t*>(ascale);
  const float txw = L.t_x * L.t_w;  // powers of two: exact
  hipStream_t st = (hipStream_t)stream;
  if (y_dtype == SVDQ_OUT_BF16) return launch_typed<true, kFmtFp4>(qx, as, z, o, b, y, plan, ws, st, txw);
  return launch_typed<false, kFmtFp4>(qx, as, z, o, b, y, plan, ws, st, txw);
}

// The low-rank up-projection alone, y = bf16(z) L2 (the unfused path's
// separate kernel): the GEMM kernel with no channel groups and no bias.
int launch_lowrank_up(const float* z, const svdq_layer& L, int b, void* y, int y_dtype, void* stream) {
  const GemmPlan plan = gemm_plan(b, L.n, 0, device_cus());  // G = 0: one tile per workgroup
  const Operands o{nullptr, nullptr, L.l2, nullptr, L.n, L.rank};
  hipStream_t st = (hipStream_t)stream;
  if (y_dtype == SVDQ_OUT_BF16) return launch_typed<true, kFmtInt4>(nullptr, nullptr, z, o, b, y, plan, nullptr, st);
  return launch_typed<false, kFmtInt4>(nullptr, nullptr, z, o, b, y, plan, nullptr, st);
}

}  // namespace svdq
