// Tiles of rows that are sorted by expert (device code).
//
// Expert e owns rows offsets[e] .. offsets[e+1]-1 of the b rows.  Its rows are
// cut into blocks of TR rows from its first one, so every block has one
// expert; a row block and a column block make a tile.  The tiles are numbered
// expert by expert, and a workgroup finds its own by a prefix sum over the
// experts' tile counts: 64 experts per wave step, the offsets being a few cache
// lines that every workgroup reads.  The number of tiles is known on the device
// only; the launch covers the most there can be (grouped_row_blocks), and the
// workgroups past the last tile end at once.
//
// Offsets are clamped to [0, b] and an end before its start counts as no rows,
// so no contents of `offsets` lead a kernel outside its rows.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"

namespace svdq {
namespace dev {

struct GroupTile {
  int live;    // 0: no tile for this workgroup
  int expert;  // the tile's expert
  int lo, hi;  // the expert's rows
  int u;       // tile index among the expert's tiles
  int blocks;  // row blocks of the expert
};

// Workgroup d of T -> index below T: workgroups are dealt round-robin to the 8
// XCDs, so each XCD gets a contiguous range, whose workgroups then share
// records in its L2.
__device__ __forceinline__ int xcd_range(int d, int T) {
  const int xcd = d & 7, k = d >> 3;
  const int per = T >> 3, extra = T & 7;
  return xcd < extra ? xcd * (per + 1) + k : extra * (per + 1) + (xcd - extra) * per + k;
}

// Exclusive scan over the wave with DPP moves (shifts within rows of 16 lanes,
// then broadcasts of the rows' last lanes); `total` receives the sum.
__device__ __forceinline__ int wave_scan(int v, int& total) {
  int s = v;
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, true);   // row_shr:1
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, true);   // row_shr:2
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, true);   // row_shr:4
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, true);   // row_shr:8
  s += __builtin_amdgcn_update_dpp(0, s, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  s += __builtin_amdgcn_update_dpp(0, s, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  total = __builtin_amdgcn_readlane(s, 63);
  return s - v;
}

// Workgroup d's tile of row blocks of TR rows and tiles_n column blocks.
// spread(d, T) maps the workgroup to a tile index below T (d < T).
template <int TR, class F>
__device__ __forceinline__ GroupTile find_tile(const int32_t* __restrict__ offsets, int experts, int b, int tiles_n,
                                               int d, F&& spread) {
  const int lane = (int)(threadIdx.x & 63);
  auto rows_of = [&](int e, int& lo, int& hi) {
    lo = hi = 0;
    if (e < experts) {
      lo = min(max(offsets[e], 0), b);
      hi = min(max(offsets[e + 1], lo), b);
    }
  };
  GroupTile g{0, 0, 0, 0, 0, 0};
  int lo, hi, sum = 0, T = 0, before = 0;
  if (experts > 64) {  // the tile count first, then the chunk that holds the tile
    for (int e0 = 0; e0 < experts; e0 += 64) {
      rows_of(e0 + lane, lo, hi);
      wave_scan((hi - lo + TR - 1) / TR * tiles_n, sum);
      T += sum;
    }
  }
  int t = 0;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    rows_of(e0 + lane, lo, hi);
    const int blocks = (hi - lo + TR - 1) / TR;
    const int ex = wave_scan(blocks * tiles_n, sum) + before;
    if (e0 == 0) {
      if (experts <= 64) T = sum;
      if (d >= T) return g;
      t = spread(d, T);
    }
    const bool mine = t >= ex && t - ex < blocks * tiles_n;
    const uint64_t hit = __ballot(mine);
    if (hit != 0) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      g.live = 1;
      g.expert = e0 + src;
      g.lo = __builtin_amdgcn_readlane(lo, src);
      g.hi = __builtin_amdgcn_readlane(hi, src);
      g.u = t - __builtin_amdgcn_readlane(ex, src);
      g.blocks = __builtin_amdgcn_readlane(blocks, src);
      return g;
    }
    before += sum;
  }
  return g;
}

}  // namespace dev
}  // namespace svdq
