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

// The sort of the slots: 8 a thread, more where that would be over 256 chunks
// (every workgroup reads the counts of all chunks).
SortPlan sort_plan(int b) {
  const long long even = ((long long)b + 256LL * kSortThreads - 1) / (256LL * kSortThreads) * kSortThreads;
  SortPlan p;
  p.chunk = (int)std::max<long long>(kSortChunk, even);
  p.chunks = std::max((int)(((long long)b + p.chunk - 1) / p.chunk), 1);
  return p;
}

// The rows' gradient of the combination: two workgroups a CU, each reading the whole
// index once; 4096 rows at the most (8 bytes each in LDS, beside 16 KB of lists).
GradPlan grad_plan(int R) {
  GradPlan p;
  p.per = std::min(std::max((R + 2 * kMaxCUs - 1) / (2 * kMaxCUs), 1), 4096);
  p.blocks = (R + p.per - 1) / p.per;
  return p;
}

namespace {

// Microseconds of an 8-bit floating-point product by tiles of 128 x 128 in k pieces, as
// measured: a launch and a tile's ends 4, a step 0.6 with one workgroup on a CU and 0.96
// for both of two (exact, by the bf16 matrix instruction: 0.96 and 1.65); for pieces a second launch, and the
// sums, 64 KB a piece, written and read.
//   tiles x pieces, steps of all pieces, fast: 72 x 1, 36: 26.7; 72 x 2: 20.7; 72 x 4: 20.3;
//   18 x 1, 36: 21.0; x 2: 15.4; x 4: 12.5; x 8: 15.0;  80 x 1, 16: 11.7; x 2: 15.5;
//   128 x 1, 64: 43.7; x 2: 30.9; x 4: 27.7;  exact: 72 x 1, 36: 39.5; x 2: 26.4; x 4: 25.8
double fp8_tiles_us(long long tiles, int G, int k, bool exact) {
  const double units = (double)(tiles * k);
  const double step = units <= kMaxCUs ? (exact ? 0.96 : 0.6) : (exact ? 1.65 : 0.96);
  const double rounds = std::max(1.0, units / (2 * kMaxCUs));
  return (4.0 + ((G + k - 1) / k) * step) * rounds + (k > 1 ? 1.5 + 0.35 * k + 0.026 * units : 0.0);
}

// The same by tiles of 64 x 128, whole (128 x 128, in the best pieces, against it):
//   exact: 333 rows, 1000 -> 1500 13.5, 9.9; 512, 1152 -> 1152 12.6, 10.4; 1000, 2048 -> 2048
//   20.7, 16.1; 256, 1152 -> 6912 14.4, 11.0; 1000, 4608 -> 1152 22.9, 30.0; 2048, 2048 ->
//   2048 22.6, 23.6;  fast: 333, 1000 -> 1500 9.7, 7.8; 512, 2048 -> 2048 11.7, 10.5;
//   1000, 2048 -> 2048 11.8, 10.8; 256, 4608 -> 4608 18.2, 21.5; 2048, 2048 -> 2048 13.0, 14.8
double fp8_small_us(long long tiles, int G, bool exact) {
  const double units = (double)tiles;
  const double step = units <= kMaxCUs ? (exact ? 0.71 : 0.48) : (exact ? 1.2 : 0.66);
  return (4.0 + G * step) * std::max(1.0, units / (2 * kMaxCUs));
}

// The same by the row kernel, for `steps` of 16 rb rows x 16 columns x 128 channels:
//   one layer, us for rb 1 / 2 / 4: 64 rows, 2048 -> 2048 7.5 / 7.3 / 8.5; 179, 1344 -> 256
//   4.6 / 5.3 / 7.0; 333, 1000 -> 1500 11.8 / 11.9 / 11.4; 100, 2048 -> 2048 11.5 / 9.2 / 8.6;
//   64, 8192 -> 8192 62 / 48 / 43; 16 rows of it 19.3 with rb 1;
//   64 experts, 2048 -> 1408, mean rows 1: 21.7 (tiles 15.1), 8: 52.9 (21.9), 32: 110 (37);
//   8 experts, 4096 -> 1152, mean 1: 9.3 (18.9), 8: 16.1 (23.6), 16: 19.3 (23.5), 32: 27.4 (24.1)
//   (tiles with fast sums; exact ones: 64 experts, mean 2: 34.9 (43.9), 8: 52 (48), 16: 72 (48);
//   8 experts, mean 8: 15.4 (32.8), 32: 25.9 (33.3), 64: 41.2 (33.5), taken 41.6)
// of one layer with weights from memory, rows 1 / 4 / 8 / 16: 8192 -> 28672 47.6 / 48.0 / 53.4 / 64.0 (tiles
//   of 64 x 128 59-60); 4096 -> 14336 16.7 / 16.2 / 17.6 / 20.3; 4096 -> 128256 92 / 94 / 104 / 126 (102-103)
double fp8_rows_us(double steps, int rb, int b, bool grouped) {
  if (grouped) return 3.5 + (rb == 1 ? 0.00035 : 0.0006) * steps;
  if (rb == 1) return 3.5 + (0.00036 + 0.00014 * std::min(b, 16) / 16) * steps;
  return rb == 2 ? 4.0 + 0.0007 * steps : 6.3 + 0.0011 * steps;
}

// No tiles of one layer are quicker than a launch and the weights from memory (5.1 TB/s).
double fp8_memory_us(int n, int m) { return 4.0 + (double)n * m / 5.1e6; }

}  // namespace

// The 8-bit floating-point product of one layer (experts 0) or of experts' rows:
//   * fast sums of more than 128 rows of one layer with more than 128 tiles of 256 x 256 (fewer
//     rows leave half of each tile empty: 4096 -> 128256, 128 rows 125 against 111 by 128 x 128,
//     129 rows 123 against 158): those tiles, which take half the records from the L2s that
//     128 x 128 ones do (8192 x 8192 -> 8192 487 us against 377; these times without an
//     activation); their last round is cut smaller where the tiles left over are few:
//     4608 x 4608 -> 12288 (96 of 864 left) 212 whole, 204 in halves, 216 in quarters;
//     4096 x 1152 -> 4608 (32 of 288) 36.5, 31.5, 29.1; 4608 x 3072 -> 9216 (136 of 648)
//     112, 125, 132;
//   * the same for experts of 1024 rows on average and more (8 experts, 4096 -> 4096,
//     mean 2048: 314 by 128 x 128, 252; 1024: 150, 143; 512: 82, 95; 1152 -> 4608, mean
//     1024: 59.5, 56.7): below, half-empty last row blocks cost more;
//   * otherwise tiles of 128 x 128, one layer's in the pieces that are quickest, for one
//     layer tiles of 64 x 128, or the row kernel, whichever the estimates above say is
//     quickest.
Fp8Plan fp8_plan(int b, int n, int m, int experts, int y_dtype) {
  const int G = fp8_blocks(m);
  const bool exact = y_dtype != (SVDQ_OUT_BF16 | SVDQ_FP8_FAST_SUMS), grouped = experts > 0;
  Fp8Plan p{0, 0, 0, 0, 1, 1, 256, {1, 1, 0}, 0, !exact};
  const long long big = (long long)((b + 255) / 256) * ((n + 255) / 256);
  if (!grouped && !exact && b > 128 && big > 128) {
    p.big = 1;
    const long long full = big / kMaxCUs * kMaxCUs, left = big - full;
    p.parts = left == 0 || left > 128 ? 1 : (left > 64 ? 2 : 4);
    p.split.grid = p.parts == 1 ? big : full + left * p.parts;
    p.full = (int)(p.parts == 1 ? big : full);
    p.threads = 512;
    return p;
  }
  const long long mean = grouped ? (b + experts - 1) / experts : b;
  if (grouped && !exact && mean >= 1024) {
    p.big = 1;
    p.split.grid = grouped_row_blocks(b, experts, 256) * ((n + 255) / 256);
    p.threads = 512;
    return p;
  }
  const long long tiles = (grouped ? grouped_row_blocks(b, experts, 128) : (b + 127) / 128) * ((n + 127) / 128);
  const double least = grouped ? 0.0 : fp8_memory_us(n, m);
  double best = std::max(fp8_tiles_us(tiles, G, 1, exact), least);
  for (int k : {2, 3, 4, 6, 8}) {
    if (grouped || G < 2 * k) break;
    const double us = std::max(fp8_tiles_us(tiles, G, k, exact), least);
    if (us < best) best = us, p.pieces = k;
  }
  const long long small = (long long)((b + 63) / 64) * ((n + 127) / 128);
  if (!grouped) {
    const double us = std::max(fp8_small_us(small, G, exact), least);
    if (us < best) best = us, p.small = 1;
  }
  for (int rb : {1, 2, 4}) {
    if (grouped && rb != (mean <= 16 ? 1 : (mean <= 32 ? 2 : 4))) continue;
    const long long blocks = grouped ? grouped_row_blocks(b, experts, 16 * rb) : (b + 16 * rb - 1) / (16 * rb);
    const double us = fp8_rows_us((double)blocks * (double)((n + 15) / 16) * G, rb, b, grouped);
    if (us >= best) continue;
    best = us;
    p.rb = rb;
    p.split = rows_split(blocks, n, 2 * G, rb);
  }
  if (p.rb) {
    p.pieces = 1;
    p.small = 0;
    p.threads = 64 * p.split.nwk * p.split.nwc;
    return p;
  }
  if (p.small) {
    p.pieces = 1;
    p.split.grid = small;
    return p;
  }
  p.split.grid = tiles * p.pieces;
  p.ws_bytes = p.pieces > 1 ? (size_t)p.split.grid * (128 * 128 * 4) : 0;
  return p;
}

}  // namespace svdq
