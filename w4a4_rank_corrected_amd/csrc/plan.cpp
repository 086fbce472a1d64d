// Launch plans of the GEMM kernels (host logic; the kernels are in
// gemm_kernels.hip, which checks its builds against the tiling and
// residencies declared in internal.h, epi_kernels.hip and rows_kernels.hip).
#include <algorithm>

#include "internal.h"

namespace svdq {

// Plan of the GEMM launch.  With T tiles of G groups and S = CUs * (resident
// workgroups per CU) slots, one tile per workgroup runs T / S full rounds and
// a last round of R = T mod S tiles, which leaves S - R slots idle for a whole
// tile's time.  Those R tiles are split instead, each into k pieces along the
// channel groups (one piece per workgroup, each of at least kMinPieceGroups
// groups), so the last round takes about 1/k of a tile's time:
//   * after full rounds, k = floor(S / R) capped at kMaxPieces, and only when
//     k >= kMinPieces: halves cost more in partial sums than they save
//     (measured on FLUX QKV and PixArt fc1);
//   * when every tile is in the last round (T < S, a few hundred rows), k =
//     floor(S / T) capped at kMaxPiecesAll, from k = 2: otherwise most CUs
//     idle (FLUX projections at 256 rows).
// NVFP4 tiles are never split: that build of its kernel does not fit the
// register budget of three workgroups per CU without spilling.
// Each piece stores its sums in a partial slot of the workspace and a
// reduction kernel adds them (plus, in the 8-bit setting, one slot per tile
// for the low-rank product).  Split workgroups come first in the
// grid, then the full rounds of whole tiles.  The workspace bound assumes the
// largest gfx950 part (256 CUs), so it does not depend on the device or the
// format.
GemmPlan gemm_plan(int b, int n, int m, int cus, int fmt) {
  const int ncu = cus > 0 ? cus : kMaxCUs;
  GemmPlan p;
  p.G = m / 64;
  p.tiles_m = (b + kGemmTileM - 1) / kGemmTileM;
  p.wg_per_cu = kGemmWgPerCu[fmt];
  const long long slots = (long long)p.wg_per_cu * ncu;
  // INT4 tiles narrow to 128 x 64 when the wide ones would not fill a round
  const long long T128 = (long long)p.tiles_m * ((n + kGemmTileN - 1) / kGemmTileN);  // wide tiles
  p.tile_n = fmt == kFmtInt4 && T128 < slots ? kGemmTileNNarrow : kGemmTileN;
  p.tiles_n = (n + p.tile_n - 1) / p.tile_n;
  const long long T = (long long)p.tiles_m * p.tiles_n;
  const long long full = T / slots, rest = T - full * slots;
  const long long cap = full == 0 ? kMaxPiecesAll : kMaxPieces, kmin = full == 0 ? 2 : kMinPieces;
  const long long k = rest > 0 ? std::min<long long>({slots / rest, cap, p.G / kMinPieceGroups}) : 0;
  p.split = fmt != kFmtFp4 && rest > 0 && k >= kmin;  // NVFP4: never (register budget)
  p.split_tiles = p.split ? (int)rest : 0;
  p.pieces = p.split ? (int)k : 1;
  p.split_grid = p.split_tiles * p.pieces;
  p.grid = (int)(p.split_grid + (T - p.split_tiles));
  // workspace: one slot per split workgroup (at most one round of slots on
  // the largest part) plus one low-rank slot per split tile (at most half a
  // round: k >= 2); none when m has too few groups to split on any device
  const int max_wg_per_cu = std::max({kGemmWgPerCu[kFmtInt4], kGemmWgPerCu[kFmtInt8], kGemmWgPerCu[kFmtFp4]});
  const long long round = (long long)max_wg_per_cu * kMaxCUs;
  const long long kcap = std::min<long long>(kMaxPiecesAll, p.G / kMinPieceGroups);
  // counted in wide tiles of 64 KB: a narrow plan's k * T narrow slots of 32 KB
  // stay within it, on any device (k * T <= one round, T <= 2 * T128)
  const long long max_slots = kcap >= 2 ? std::min(round, T128 * kcap) + std::min(T128, round / 2) : 0;
  p.partial_bytes = (size_t)max_slots * kGemmTileM * kGemmTileN * 4;
  p.ws_bytes = p.partial_bytes;
  return p;
}

// Waves to split the groups over: up to the 16 waves a CU that are resident
// together (more would wait for a second round), each with two groups at the
// least; then column blocks until a workgroup has four waves.
RowsSplit rows_split(long long row_blocks, int n, int G, int rb) {
  const long long tiles = row_blocks * ((n + 15) / 16);
  RowsSplit s{1, 1, 0};
  while (s.nwk < (rb == 4 ? 8 : 16) && tiles * s.nwk <= 2048 && G >= 4 * s.nwk) s.nwk *= 2;
  if (s.nwk < 4) s.nwc = 4 / s.nwk;
  s.grid = row_blocks * ((n + 16 * s.nwc - 1) / (16 * s.nwc));
  return s;
}

// The row kernel or tiles.  The row kernel's cost is the (16 RB rows) x (16
// columns) x group steps it takes; a tile's waves share the weights, but each
// tile walks all groups at about half a microsecond a step, so too few tiles
// leave the chip waiting.  Product alone, us, row kernel against 64 x 128 tiles:
//   mean rows 4   of 64 experts, 2048 -> 1408: 21 / 26;  mean 16: 38 / 33;  mean 32: 53 / 43
//   mean rows 16  of 8 experts,  1152 -> 4608: 14 / 18 (324 tiles);  mean 64: 25 / 19 (540 tiles)
//   mean rows 150 of 4 experts,  4608 -> 1152: 21 / 39 (117 tiles)
// and about the limits, where the slower side was taken by 10 % at the most:
//   mean 8  of 64 experts, 2048 -> 1408 (259 000 steps) 26.4 / 31.9;  mean 10 (282 000): 29.6 / 32.5
//   mean 24 of 8 experts,  1152 -> 4608 (360 tiles) 17.0 / 18.0;  mean 32 (396 tiles): 17.2 / 18.3
//   mean 200 of 4 experts, 4608 -> 1152 (145 000 steps) 26.6 / 38.1;  mean 128 of 8 (202 000): 37.6 / 38.4
//   mean 10 of 128 experts, 1152 -> 512 (584 tiles) 18.7 / 18.7
// 128 x 128 tiles do the most work per staged record, 64 x 128 tiles leave less
// of an expert's last row block empty and fill the chip with fewer rows: mean
// rows 64 of 64 experts (2048 -> 1408) 66 / 51 us, 128: 80 / 73, 281: 133 / 140;
// mean 256 of 8 experts, 4608 -> 1152 (207 wide tiles) 70 / 63.
GroupedPlan grouped_plan(int b, int n, int m, int experts) {
  const int G = m / 64;
  const long long mean = (b + experts - 1) / experts;  // rows of an expert; the real counts are on the device
  const long long cols = (n + kGemmTileN - 1) / kGemmTileN;
  GroupedPlan p{mean <= 16 ? 1 : 2, 0, 0, 0};
  const long long blocks = grouped_row_blocks(b, experts, 16 * p.rb), steps = blocks * ((n + 15) / 16) * G;
  const long long tiles = grouped_row_blocks(b, experts, 64) * cols;
  if (mean <= 8 || (tiles <= 384 && steps <= 160000)) {
    const RowsSplit s = rows_split(blocks, n, G, p.rb);
    p.grid = s.grid;
    p.threads = 64 * s.nwk * s.nwc;
    return p;
  }
  p.rb = 0;
  const long long wide = grouped_row_blocks(b, experts, 128) * cols;
  p.tile_m = mean >= 256 && wide >= 3 * kMaxCUs ? 128 : 64;
  p.grid = p.tile_m == 128 ? wide : tiles;
  p.threads = 256;
  return p;
}

}  // namespace svdq
