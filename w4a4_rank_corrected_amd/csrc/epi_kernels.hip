// The tiled product (gemm_body.h) with the epilogue of epilogue.h, for one
// layer in the INT4, 8-bit and NVFP4 settings, and for INT4 layers grouped by
// expert; and the choice between it and the row kernel.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_body.h"
#include "launch.h"

#pragma clang fp contract(off)

namespace svdq {
namespace {

using namespace dev;

// INT4 is bound by the two FMAs per output and channel group that apply the
// scales (4096 x 1152 -> 4608 with GELU: 52.6 us, of which the 18 groups are 33 and
// y's write, Z L2 and GELU the rest).  8 bits with hundreds of rows: neither the
// vector nor the matrix units are busy (1000 x 4608 -> 1152: 14.8 us and 6.7 us of
// reduction, 0.34 M MFMAs are 2 us of them); the pieces fetch 52 MB past the L2s
// for 10 MB of codes, since every XCD's L2 takes its own copy, and write 19 MB of
// sums.  How much of the time that is, and how much the latency of the steps,
// is not told apart: 64 x 64 tiles (36 MB, no sums to write) take 21.8 us.
// NVFP4: the dequantization, which every wave does for its own operands (2304 x
// 1152 -> 4608 with GELU: 39.6 us; 128 vector instructions a group for it, 265 a
// group by the counters with staging, addresses and the epilogue, 45 % of the
// vector units' time, beside 33 MFMAs, 25 % of theirs), and 648 tiles on 256 CUs,
// 3 on the fullest (42.5 us with the block scales widened bit by bit, 44.9 us with
// 32 LDS reads a group instead of 10 as well).
template <class C, bool OUT_BF16, int FMT, bool SK>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WPE, C::WPE))) void gemm_epi_kernel(
    const uint8_t* __restrict__ qx, const uint16_t* __restrict__ ascale, const float* __restrict__ z, Operands L, int b,
    int G, int tiles_m, int tiles_n, SplitK sk, float txw, EpiArgs ep) {
  gemm_up_body<C, OUT_BF16, FMT, SK, kTileEpi>(qx, ascale, z, L.qw, L.wscale, L.l2, L.bias, b, L.n, G, L.rank, tiles_m,
                                               tiles_n, nullptr, sk, txw, ep);
}

// 8-bit codes, few tiles: 64 x 64 tiles, 4 waves of 32 x 32, loads three groups
// ahead (90 registers).
using Cfg8S = GemmCfg<64, 64, 32, 32, 4, 3>;
// NVFP4, split tiles: at most two workgroups a CU are launched, so two share its
// registers and loads run two groups ahead.
using CfgF4K = GemmCfg<128, 128, 64, 64, 2, 2>;
// Experts with few rows: 64 x 128 tiles, 4 waves of 64 x 32.
using CfgG = GemmCfg<64, 128, 64, 32, 3, 2>;

// One tile of one expert per workgroup; the workgroups past the last tile end.
// Bound as the dense INT4 product, plus the empty rows of each expert's last row
// block: 8192 rows of 8 experts, 1152 -> 4608: 98.8 us; 18006 rows of 64 experts,
// 2048 -> 1408: 118 us, 27 % more tile rows than rows.
template <class C, bool OUT_BF16>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WPE, C::WPE))) void gemm_grouped_kernel(
    const uint8_t* __restrict__ qx, const uint16_t* __restrict__ ascale, const float* __restrict__ z, Operands L, int b,
    int G, int tiles_n, Groups groups, EpiArgs ep) {
  const GroupTile g = find_tile<C::TM>(groups.offsets, groups.experts, b, tiles_n, (int)blockIdx.x,
                                       [](int d, int T) { return xcd_range(d, T); });
  if (!g.live) return;
  const size_t e = (size_t)g.expert;
  gemm_up_body<C, OUT_BF16, kFmtInt4, false, kTileGrouped>(
      qx, ascale, z, L.qw + e * G * L.n * 32, L.wscale + e * G * L.n, L.rank > 0 ? L.l2 + e * L.n * L.rank : nullptr,
      L.bias ? L.bias + e * L.n : nullptr, b, L.n, G, L.rank, 0, tiles_n, nullptr, SplitK{0, 0, 1, 0, nullptr}, 1.0f, ep,
      g);
}

template <bool OUT_BF16, int FMT>
int launch_tiles(const uint8_t* qx, const uint16_t* ascale, const float* z, const Operands& L, int b,
                 const GemmPlan& plan, const EpiArgs& ep, void* ws, hipStream_t st, float txw) {
  SplitK sk{0, 0, 1, 0, nullptr};
  if (plan.split) {
    sk.P = plan.split_grid;
    sk.T = plan.split_tiles;
    sk.k = plan.pieces;
    sk.lr = L.rank > 0 ? kLowRankPieceGroups : 0;
    sk.partials = reinterpret_cast<float*>(ws);
  }
  auto run = [&](auto cfg) {
    using C = decltype(cfg);
    auto gemm = [&](auto kernel) {
      return launch_checked(kernel, plan.grid, C::NT, st, qx, ascale, z, L, b, plan.G, plan.tiles_m, plan.tiles_n, sk,
                            txw, ep);
    };
    if (!plan.split) return gemm(gemm_epi_kernel<C, OUT_BF16, FMT, false>);
    if constexpr (std::is_same_v<C, Cfg8S>) {
      return (int)hipErrorInvalidValue;  // never split
    } else {
      using CS = std::conditional_t<FMT == kFmtFp4, CfgF4K, C>;
      const int status = gemm(gemm_epi_kernel<CS, OUT_BF16, FMT, true>);
      if (status != 0) return status;
      constexpr int UNITS = C::TM * C::TN / 4;
      // NVFP4 pieces are scaled sums: they add up like INT4's
      return launch_checked(splitk_reduce_kernel<C, FMT == kFmtFp4 ? kFmtInt4 : FMT, OUT_BF16, true>,
                            (int)(((long long)sk.T * UNITS + 255) / 256), 256, st, (const float*)sk.partials, sk.T, sk.k,
                            plan.tiles_m, plan.tiles_n, b, L.n, ascale, L.wscale,
                            FMT != kFmtInt4 && L.rank > 0 ? 1 : 0, L.bias, (void*)nullptr, ep);
    }
  };
  if constexpr (FMT == kFmtInt8) return plan.tile_n == Cfg8S::TN ? run(Cfg8S{}) : run(Cfg8{});
  if constexpr (FMT == kFmtFp4) return run(CfgF4{});
  if constexpr (FMT == kFmtInt4) return plan.tile_n == CfgN::TN ? run(CfgN{}) : run(Cfg{});
}

// One tile of TM x TN per workgroup, none split.
template <class C>
void whole_tiles(GemmPlan& p, int b, int n) {
  p.tiles_m = (b + C::TM - 1) / C::TM;
  p.tiles_n = (n + C::TN - 1) / C::TN;
  p.tile_n = C::TN;
  p.grid = p.tiles_m * p.tiles_n;
  p.split = p.split_tiles = p.split_grid = 0;
  p.pieces = 1;
}

// The plan of the plain product, except for few tiles.
// INT4, less than one round of tiles (768), T = wide (128 x 128) tiles:
//   * above half a round whole wide tiles, not narrow ones (rank 16, residual, us:
//     1500 x 1152 -> 4608, T = 432, 32.0 narrow / 29.6 wide; 2500 rows, T = 720,
//     42.3 / 37.0; 3000 x 2048 -> 2048, T = 384, 34.7 / 42.4);
//   * pieces only where they pay.  A narrow tile takes about half a microsecond a
//     group, so k pieces save G (1 - 1/k) / 2; they cost a launch and 64 KB of
//     traffic a piece, about 1.5 us + 0.013 us a piece (split / whole, us:
//     200 x 1152 -> 4608 16.4 / 14.5, 500 rows 22.4 / 19.5, 1000 x 2048 -> 2048
//     24.4 / 21.9; 500 x 2048 -> 2048 17.5 / 20.6, 256 x 4096 -> 8000 31.9 / 36.6,
//     1000 x 4608 -> 1152 24.7 / 39.9).
// 8 bits, up to 384 tiles (more keep the plain plan: 576, 2000 x 4608 -> 4608, 64
// us, 64 x 64 tiles 76): the quicker of
//   * 64 x 64 tiles, unsplit: 5.2 us + 0.155 us a group, and 0.42 of that again
//     for each further round of one tile a CU;
//   * as many pieces as give every CU one workgroup, two at the least: 8.5 us +
//     0.3 us a group of a piece + 0.02 us a piece (more pieces are slower: 1000 x
//     4608 -> 1152, 72 tiles, 3 pieces 21.0 us, 10 27.1).
// 64 x 64 / pieces, rank 16, gate, residual, us:
//   1 x 1152 -> 4608 7.3 / 11.7; 128 x 2048 -> 2048 10.2 / 12.1; 256 x 3008 -> 1152
//   13.6 / 13.4; 1 x 4032 -> 1152 13.0 / 10.8; 100 x 4032 -> 512 14.2 / 10.2; 256 x
//   4032 -> 1152 15.8 / 13.8; 400 x 4032 -> 1152 15.4 / 15.6; 256 x 4096 -> 2048
//   15.7 / 16.8; 256 x 4608 -> 1152 16.8 / 14.0; 500 x 4608 -> 1152 16.8 / 16.4; 500
//   x 4608 -> 2048 17.4 / 20.2; 65 x 8192 -> 2048 23.5 / 14.1; 1 x 8192 -> 8192 22.8 /
//   23.2; 1000 x 4608 -> 1152 (288 tiles of 64 x 64) 21.8 / 21.0; 600 x 8192 -> 2048
//   31.5 / 27.0; 1000 x 4096 -> 2048 23.0 / 28.5; 1500 x 4608 -> 2048 31.0 / 37.4.
// On 60 random shapes (1..3000 rows, 256..8960 -> 64..9216) the choice was within
// 7 % of the quicker side.
// NVFP4, which the plain product never splits: into as many pieces as two
// workgroups a CU take, where the 0.62 us a group that they save pay for the
// launch and for 0.03 us a piece (whole / split, us: 256 x 4608 -> 1152 51.6 /
// 16.4; 500 x 2048 -> 2048 27.1 / 18.7; 128 x 8192 -> 8192 89 / 33; 65 x 12288 ->
// 3000 128 / 25; 100 x 1152 -> 4608 17.9 / 16.0; not 256 x 1152 -> 4608, 18.2 /
// 18.8; up to 64 rows are the row kernel's).  Fewer pieces, where they cost least by that count, were up to 10 %
// slower.  The pieces stay within the workspace: k T <= two a CU, k within the
// limits it is sized for.
GemmPlan epi_plan(int b, int n, int m, int fmt) {
  GemmPlan p = gemm_plan(b, n, m, device_cus(), fmt);
  const long long T = (long long)p.tiles_m * p.tiles_n, slots = (long long)p.wg_per_cu * device_cus();
  if (fmt == kFmtInt4 && T < 2 * slots && p.tile_n == CfgN::TN) {
    const long long wide = (long long)p.tiles_m * ((n + Cfg::TN - 1) / Cfg::TN);
    if (2 * wide > slots + 32)
      whole_tiles<Cfg>(p, b, n);
    else if (p.split && 0.5 * p.G * (1.0 - 1.0 / p.pieces) <= 1.5 + 0.013 * (double)p.split_grid)
      whole_tiles<CfgN>(p, b, n);
  }
  if (fmt == kFmtFp4) {
    const long long two = CfgF4K::WG_PER_CU * (long long)device_cus();
    const long long k = std::min<long long>({kMaxPiecesAll, p.G / kMinPieceGroups, two / T});
    if (k >= 2 && 0.62 * p.G * (1.0 - 1.0 / (double)k) > 1.5 + 0.03 * (double)(T * k)) {
      p.pieces = (int)k;
      p.split = 1;
      p.split_tiles = (int)T;
      p.split_grid = p.grid = (int)(T * k);
    }
  }
  if (fmt == kFmtInt8) {
    const long long cus = device_cus();
    const long long small = (long long)((b + Cfg8S::TM - 1) / Cfg8S::TM) * ((n + Cfg8S::TN - 1) / Cfg8S::TN);
    const long long k = std::min<long long>(p.pieces, cus / T);
    const double whole = (5.2 + 0.155 * p.G) * (1.0 + 0.42 * (double)((small - 1) / cus));
    const double split = 8.5 + 0.3 * p.G / (double)std::max<long long>(k, 1) + 0.02 * (double)(T * k);
    if (T <= 384 && (k < 2 || whole <= split)) {
      whole_tiles<Cfg8S>(p, b, n);
    } else if (p.split && p.split_tiles == T) {
      p.pieces = (int)std::max<long long>(2, k);
      p.split_grid = p.grid = (int)T * p.pieces;
    }
  }
  return p;
}

template <int FMT>
int launch_tiles_typed(const uint8_t* qx, const uint16_t* ascale, const float* z, const Operands& L, int m, int b,
                       int y_dtype, const EpiArgs& ep, void* ws, void* stream, float txw) {
  const GemmPlan plan = epi_plan(b, L.n, m, FMT);
  hipStream_t st = (hipStream_t)stream;
  return y_dtype == SVDQ_OUT_BF16 ? launch_tiles<true, FMT>(qx, ascale, z, L, b, plan, ep, ws, st, txw)
                                  : launch_tiles<false, FMT>(qx, ascale, z, L, b, plan, ep, ws, st, txw);
}

template <class C>
int launch_grouped_tiles(const uint8_t* qx, const uint16_t* ascale, const float* z, const Operands& L, int G,
                         const Groups& groups, int b, int y_dtype, const EpiArgs& ep, const GroupedPlan& plan,
                         hipStream_t st) {
  static_assert(C::TN == kGemmTileN && C::NT == 256, "the plan's tiles");
  auto go = [&](auto kernel) {
    return launch_checked(kernel, plan.grid, C::NT, st, qx, ascale, z, L, b, G, (L.n + C::TN - 1) / C::TN, groups, ep);
  };
  return y_dtype == SVDQ_OUT_BF16 ? go(gemm_grouped_kernel<C, true>) : go(gemm_grouped_kernel<C, false>);
}

}  // namespace

int launch_gemm_epi(const uint8_t* qx, const uint16_t* ascale, const float* z, const svdq_layer& L, int b, int y_dtype,
                    const EpiArgs& ep, void* ws, void* stream) {
  if (b <= kRowsMax) {
    const RowsArgs a{qx, ascale, z, L.qw, L.wscale, L.l2, L.bias, b, L.n, L.m / SVDQ_GROUP, L.rank, Groups{nullptr, 0}, ep, 1.0f};
    return launch_gemm_rows(a, b <= 16 ? 1 : (b <= 32 ? 2 : 4), y_dtype, kFmtInt4, stream);
  }
  const Operands o{L.qw, L.wscale, L.l2, L.bias, L.n, L.rank};
  return launch_tiles_typed<kFmtInt4>(qx, ascale, z, o, L.m, b, y_dtype, ep, ws, stream, 1.0f);
}

int launch_gemm8_epi(const int8_t* qx, const uint16_t* ascale, const float* z, const svdq_w8a8_layer& L, int b,
                     int y_dtype, const EpiArgs& ep, void* ws, void* stream) {
  const Operands o{reinterpret_cast<const uint8_t*>(L.qw), L.wscale, L.l2, L.bias, L.n, L.rank};
  return launch_tiles_typed<kFmtInt8>(reinterpret_cast<const uint8_t*>(qx), ascale, z, o, L.m, b, y_dtype, ep, ws,
                                      stream, 1.0f);
}

int launch_gemm_fp4_epi(const uint8_t* qx, const uint8_t* ascale, const float* z, const svdq_fp4_layer& L, int b,
                        int y_dtype, const EpiArgs& ep, void* ws, void* stream) {
  const Operands o{L.qw, reinterpret_cast<const uint16_t*>(L.wscale), L.l2, L.bias, L.n, L.rank};
  if (b <= kRowsMax) {
    const RowsArgs a{qx, reinterpret_cast<const uint16_t*>(ascale), z, L.qw, o.wscale, L.l2, L.bias, b, L.n,
                     L.m / SVDQ_GROUP, L.rank, Groups{nullptr, 0}, ep, L.t_x * L.t_w};
    return launch_gemm_rows(a, b <= 16 ? 1 : (b <= 32 ? 2 : 4), y_dtype, kFmtFp4, stream);
  }
  return launch_tiles_typed<kFmtFp4>(qx, reinterpret_cast<const uint16_t*>(ascale), z, o, L.m, b, y_dtype, ep, ws,
                                     stream, L.t_x * L.t_w);
}

int launch_grouped_gemm(const uint8_t* qx, const uint16_t* ascale, const float* z, const svdq_grouped_layer& L,
                        const int32_t* offsets, int b, int y_dtype, const EpiArgs& ep, void* stream) {
  const Groups groups{offsets, L.experts};
  const int G = L.m / SVDQ_GROUP;
  const GroupedPlan plan = grouped_plan(b, L.n, L.m, L.experts);
  if (plan.rb > 0) {
    const RowsArgs a{qx, ascale, z, L.qw, L.wscale, L.l2, L.bias, b, L.n, G, L.rank, groups, ep, 1.0f};
    return launch_gemm_rows(a, plan.rb, y_dtype, kFmtInt4, stream);
  }
  const Operands o{L.qw, L.wscale, L.l2, L.bias, L.n, L.rank};
  hipStream_t st = (hipStream_t)stream;
  return plan.tile_m == Cfg::TM ? launch_grouped_tiles<Cfg>(qx, ascale, z, o, G, groups, b, y_dtype, ep, plan, st)
                                : launch_grouped_tiles<CfgG>(qx, ascale, z, o, G, groups, b, y_dtype, ep, plan, st);
}

}  // namespace svdq
