// The 8-bit floating-point product for many rows: tiles through LDS.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "epilogue.h"
#include "fp8.h"
#include "grouped.h"
#include "internal.h"
#include "launch.h"

#pragma clang fp contract(off)

namespace svdq {
namespace {

using namespace dev;

// 16 bytes a lane from memory to LDS: to + 16 lane, past the resource's end zeros.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t offset, void* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, offset, 0, 0, 0);
}

// Records in LDS: record r's 16-byte piece p lies at place p ^ key(r), so that the
// lanes of an operand read, which want one piece of 16 records, spread over the banks.
__device__ __forceinline__ int record_key(int r) { return r & 7; }

// W (4, or 8 of bf16) whole columns of a row from column j on, at any element's address.
template <int W, bool BF16>
__device__ __forceinline__ void load_whole(const void* row, int j, float (&v)[W]) {
  if constexpr (BF16 && W == 8) {
    const u32x4 w = *reinterpret_cast<const u32x4_loose*>(reinterpret_cast<const uint16_t*>(row) + j);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
  } else if constexpr (BF16) {
    const uint2 w = *reinterpret_cast<const uint2_loose*>(reinterpret_cast<const uint16_t*>(row) + j);
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
  } else {
    const f32x4 w = *reinterpret_cast<const f32x4_loose*>(reinterpret_cast<const float*>(row) + j);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = w[e];
  }
}
// The same where the row may end in them (n >= 1 columns): an element at a time, the last
// one for those behind it, so that all of the loads are under way together.
template <int W, bool BF16>
__device__ __forceinline__ void load_ragged(const void* row, int j, int n, float (&v)[W]) {
  if (j + W <= n) return load_whole<W, BF16>(row, j, v);
#pragma unroll
  for (int e = 0; e < W; ++e) {
    const int at = min(j + e, n - 1);
    v[e] = BF16 ? bf16_lo(reinterpret_cast<const uint16_t*>(row)[at]) : reinterpret_cast<const float*>(row)[at];
  }
}
template <int W, bool BF16>
__device__ __forceinline__ void store_whole(void* to, const float (&v)[W]) {
  if constexpr (BF16)
    *reinterpret_cast<u32x4_loose*>(to) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                                pack_bf16x2(v[6], v[7])};
  else
    *reinterpret_cast<f32x4_loose*>(to) = f32x4{v[0], v[1], v[2], v[3]};
}

// s_waitcnt's operand: at most vm loads and lgkm LDS accesses under way.
constexpr int wait_for(int vm, int lgkm) { return (vm & 15) | 0x70 | lgkm << 8 | (vm >> 4) << 14; }

// The first column of the four that block f of a lane's results holds.
template <bool OUT_BF16>
__device__ __forceinline__ int column_of(int jw, int c, int f) {
  return jw + (OUT_BF16 ? 32 * (f >> 1) + 8 * c + 4 * (f & 1) : 16 * f + 4 * c);
}

// The activation, gate and residual, and y's rounding, for a wave's 16 QB rows from
// row0 on and 64 columns from jw on.  A lane holds W neighbouring columns of a row in
// each of UNITS units; four lanes' are 64 bytes of y.  part: 32 x 272 bytes of LDS of
// the wave's own, not in use.
template <int QB, bool OUT_BF16>
__device__ __forceinline__ void finish_rows(const f32x4 (&acc)[4][QB], int row0, int row_end, int jw, int n,
                                            const EpiArgs& ep, uint8_t* part) {
  const int lane = (int)threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  constexpr int W = OUT_BF16 ? 8 : 4, UNITS = 16 / W;
  const int begin = ep.act == SVDQ_ACT_NONE ? n : ep.act_begin;
  if (jw >= n) return;
  if (jw + 64 <= n && (begin <= jw || begin >= jw + 64)) {
    // Whole columns, all with the activation or all without: straight code, one copy for
    // each case, so that a call's instructions lie together.
    auto finish = [&](auto A, auto MORE) {
      uint8_t* y = reinterpret_cast<uint8_t*>(row_of<OUT_BF16>(ep.y, row0 + r, ep.ldy)) + (jw + W * c) * (OUT_BF16 ? 2 : 4);
      const size_t next = (size_t)16 * ep.ldy * (OUT_BF16 ? 2 : 4);
      // The gate and the residual of a block of rows are loaded before the block before it
      // is stored (the compiler would wait for each: the residual may be y).
      float gv[2][UNITS][W], rv[2][UNITS][W];
      auto load_more = [&](int q) {
        const int i = min(row0 + 16 * q + r, row_end - 1);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const int j = jw + W * c + 4 * W * u;
          if (ep.gate) load_whole<W, true>(row_of<true>(ep.gate, i / ep.gate_rows, n), j, gv[q & 1][u]);
          if (ep.residual) load_whole<W, OUT_BF16>(row_of<OUT_BF16>(ep.residual, i, ep.ldr), j, rv[q & 1][u]);
        }
      };
      if constexpr (decltype(MORE)::value) load_more(0);
#pragma unroll
      for (int q = 0; q < QB; ++q, y += next) {
        const int i = row0 + 16 * q + r;
        if constexpr (decltype(MORE)::value)
          if (q + 1 < QB) load_more(q + 1);
        if (i >= row_end) break;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          float v[W];
#pragma unroll
          for (int e = 0; e < W; ++e) v[e] = act_value<decltype(A)::value>(acc[W / 4 * u + e / 4][q][e & 3]);
          if constexpr (decltype(MORE)::value) {
            if (ep.gate) {
#pragma unroll
              for (int e = 0; e < W; ++e) v[e] *= gv[q & 1][u][e];
            }
            if (ep.residual) {
#pragma unroll
              for (int e = 0; e < W; ++e) v[e] = rv[q & 1][u][e] + v[e];
            }
          }
          store_whole<W, OUT_BF16>(y + 64 * u, v);
        }
      }
    };
    auto with_more = [&](auto A) {
      if (ep.gate || ep.residual)
        finish(A, std::true_type{});
      else
        finish(A, std::false_type{});
    };
    if (begin >= jw + 64)
      with_more(std::integral_constant<int, SVDQ_ACT_NONE>{});
    else
      with_act(ep.act, with_more);
    return;
  }

  // The other waves: 32 rows at a time through LDS and one loop over the rows, with
  // every column's own case.
  constexpr int LANES = 64 / W;  // lanes of a row
  constexpr int kPitch = 272;    // bytes of a row of 64 sums: rows on different banks
  const int rr = lane / LANES, cc = lane % LANES;
  const int j = jw + W * cc;
#pragma unroll 1
  for (int p = 0; p < (QB + 1) / 2; ++p) {
#pragma unroll
    for (int b = 0; b < (QB + 1) / 2; ++b)
      if (b == p) {  // (accumulators are registers: a branch for each pair of blocks)
#pragma unroll
        for (int h = 0; h < 2 && 2 * b + h < QB; ++h)
#pragma unroll
          for (int f = 0; f < 4; ++f)
            *reinterpret_cast<f32x4*>(part + (16 * h + r) * kPitch + (column_of<OUT_BF16>(0, c, f)) * 4) = acc[f][2 * b + h];
      }
    // other lanes' results: LDS accesses of one wave complete in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int kRows = 64 / LANES, U = QB == 1 || OUT_BF16 ? 2 : 4;  // rows at a time, times U with their loads together
#pragma unroll 1
    for (int k0 = rr; k0 < (QB > 1 ? 32 : 16); k0 += U * kRows) {
      float gv[U][W], rv[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = row0 + 32 * p + k0 + u * kRows;
        if (i < row_end && j < n) {
          if (ep.gate) load_ragged<W, true>(row_of<true>(ep.gate, i / ep.gate_rows, n), j, n, gv[u]);
          if (ep.residual) load_ragged<W, OUT_BF16>(row_of<OUT_BF16>(ep.residual, i, ep.ldr), j, n, rv[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * kRows, i = row0 + 32 * p + k;
        if (i < row_end && j < n) {
          float v[W];
#pragma unroll
          for (int e = 0; e < W; e += 4) {
            const f32x4 t = *reinterpret_cast<const f32x4*>(part + k * kPitch + (W * cc + e) * 4);
#pragma unroll
            for (int x = 0; x < 4; ++x) v[e + x] = t[x];
          }
          with_act(ep.act, [&](auto A) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
              const float t = act_value<decltype(A)::value>(v[e]);
              v[e] = j + e >= ep.act_begin ? t : v[e];
            }
          });
          if (ep.gate) {
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] *= gv[u][e];
          }
          if (ep.residual) {
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = rv[u][e] + v[e];
          }
          store_cols<W, OUT_BF16>(row_of<OUT_BF16>(ep.y, i, ep.ldy), j, n, v);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// One tile: rows i0 .. i0 + TM - 1 (those before row_end), columns j0 .. j0 + TN - 1,
// channel blocks 0 .. G-1 of the operands given.  PARTIAL: the sums alone, to `sums`.
//
// NWM x NWN waves of 16 QB rows x 64 columns each.  Per block of 128 channels the
// records of the tile's rows and columns go from memory into LDS (no registers in
// between), two steps ahead; weights are the first operand of the matrix instruction,
// so that a lane's four results are neighbouring columns of one row.
template <int QB, int NWM, int NWN>
struct TileShape {
  static constexpr int TM = 16 * QB * NWM, TN = 64 * NWN, NW = NWM * NWN;
  static constexpr int kCodes = (TM + TN) * 128;            // bytes of a step's records: rows, then columns
  static constexpr int QS = (QB + 3) / 4 * 4;               // bytes of scales a lane reads
  static constexpr int kScales = 16 * QS * NWM;             // [wave row][16 rows][QS]
  static constexpr int kPart = 32 * 272;                    // finish_rows' part of a wave
  static constexpr int kBuffer = kCodes > NW / 2 * kPart ? kCodes : NW / 2 * kPart;
};
template <int QB, int NWM, int NWN, bool EXACT, bool OUT_BF16, bool GROUPED, bool PARTIAL>
__device__ __forceinline__ void tile(const Fp8Args& a, const uint8_t* qx, const uint8_t* ascale, const uint8_t* qw,
                                     const uint8_t* wscale, const uint16_t* bias, int G, int i0, int j0, int row_end,
                                     uint8_t* s_even, uint8_t* s_odd, uint8_t* s_scale_even, uint8_t* s_scale_odd,
                                     f32x4* sums) {
  typedef TileShape<QB, NWM, NWN> Shape;
  constexpr int TM = Shape::TM, TN = Shape::TN, NW = Shape::NW, QS = Shape::QS;
  constexpr int LX = TM / (8 * NW), LW = TN / (8 * NW);  // 8-record loads a wave and step
  static_assert(LX * 8 * NW == TM && LW * 8 * NW == TN && TM <= 64 * NW, "whole loads");
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / NWN, wn = wave - wm * NWN;
  const int r = lane & 15, c = lane >> 4;
  const int n = a.n, NB = (n + 127) / 128, xr = a.x_rows;

  // What this lane loads: piece (lane & 7) ^ key of records 8 (wave + NW i) + lane / 8.
  // From load to load i the records are 8 NW further, and so are the rows (unless they
  // are gathered) and the columns.
  constexpr uint32_t kNext = 8 * NW * 128;
  const int rec = 8 * wave + (lane >> 3);
  const uint32_t piece = 16u * ((lane & 7) ^ record_key(rec));
  uint32_t xoff[LX];
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < LX; ++i) {
      int s = i0 + rec + 8 * NW * i;
      if (s >= row_end) s = -1;
      if (s >= 0 && a.row_index) s = a.row_index[s];
      xoff[i] = ((unsigned)s < (unsigned)xr ? (uint32_t)s * 128u : 0x7FFFFF80u) + piece;
    }
  } else {
    xoff[0] = (uint32_t)(i0 + rec) * 128u + piece;  // (rows behind the last are past the resource's end)
  }
  // bf16: record 64 w + 16 f + 4 c + v holds column 64 w + 32 (f / 2) + 8 c + 4 (f % 2) + v,
  // so that a lane's results of two blocks f are eight neighbouring columns and four
  // lanes' are 64 bytes of a row (fp32 has those in the records' own order)
  static_assert(NW % 4 == 0, "32 records on are 32 columns on");
  const int rf = rec >> 4 & 3;
  const int col = OUT_BF16 ? (rec & ~63) + 32 * (rf >> 1) + 8 * (rec >> 2 & 3) + 4 * (rf & 1) + (rec & 3) : rec;
  const uint32_t woff = (uint32_t)(j0 + col) * 128u + piece;
  // the row whose scale this thread stages, and its place
  uint32_t soff = 0x7FFFFFFFu;
  if (tid < TM && i0 + tid < row_end) {
    int s = i0 + tid;
    if (GROUPED && a.row_index) s = a.row_index[s];
    if ((unsigned)s < (unsigned)xr) soff = (uint32_t)s;
  }
  const int splace = (tid / (16 * QB)) * 16 * QS + (tid & 15) * QS + (tid >> 4) % QB;

  struct Source {
    __amdgpu_buffer_rsrc_t x, w;
    uint32_t x0, w0;
  };
  auto source = [&](int g) {  // (past the last step zeros, without memory traffic)
    const size_t at = g < G ? (size_t)g : 0;
    Source f{make_rsrc(qx + at * xr * 128, g < G ? (uint32_t)xr * 128u : 0u),
             make_rsrc(qw + at * n * 128, g < G ? (uint32_t)n * 128u : 0u), xoff[0], woff};
    // (a load's offset is formed where it is issued, by one addition, not kept in a register)
    asm("" : "+v"(f.x0), "+v"(f.w0));
    return f;
  };
  // load k of a step's LX + LW
  auto load_codes = [&](const Source& f, uint8_t* to, int k) {
    if (k < LX)
      load_to_lds(f.x, GROUPED ? xoff[k] : f.x0 + k * kNext, to + 1024 * (wave + NW * k));
    else
      load_to_lds(f.w, f.w0 + (k - LX) * kNext, to + TM * 128 + 1024 * (wave + NW * (k - LX)));
  };
  // (past the last step the last one's, unused)
  auto load_sx = [&](int g) -> uint32_t {
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(ascale + (size_t)min(g, G - 1) * xr, (uint32_t)xr);
    return __builtin_amdgcn_raw_buffer_load_b8(rx, soff, 0, 0);
  };
  auto load_sw = [&](int g) -> uint32_t {
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(wscale + (size_t)min(g, G - 1) * NB, (uint32_t)NB);
    return __builtin_amdgcn_raw_buffer_load_b8(rw, (uint32_t)(j0 + 64 * wn) / 128u, 0, 0);
  };
  // this lane's pieces 2 c and 2 c + 1 of record r of 16
  const uint32_t lane_at = r * 128 + 16 * ((2 * c) ^ record_key(r));
  auto read = [&](const uint8_t* records, uint32_t at) -> i32x8 {
    return operand(*reinterpret_cast<const u32x4*>(records + at), *reinterpret_cast<const u32x4*>(records + (at ^ 16)));
  };
  auto read_w = [&](const uint8_t* buf, int f, uint32_t at) {
    return read(buf + TM * 128 + wn * 8192 + f * 2048, at);
  };
  auto read_x = [&](const uint8_t* buf, int q, uint32_t at) { return read(buf + (wm * QB + q) * 2048, at); };

  // the sums start from the bias: the columns of this lane's results of block f
  const int jw = j0 + 64 * wn;  // the wave's first column
  f32x4 acc[4][QB];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const f32x4 t = !PARTIAL && bias ? load4<true>(bias, column_of<OUT_BF16>(jw, c, f), n) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < QB; ++q) acc[f][q] = t;
  }
  constexpr int R = QB / 2;     // blocks of rows in registers at a time
  i32x8 w_even[4], w_odd[4], xv[R];
  uint32_t sx[QS / 4], sw;      // the step's scales: bytes of the rows' four blocks, the columns'
  uint32_t sx_ahead, sw_ahead;  // in flight: the byte this thread stages, two steps ahead; the columns', one ahead

  // A step.  Its columns and its first R blocks of rows are in registers (or on their
  // way), the other blocks follow from `cur`, each into the registers of the block R
  // before it once that one's multiplications are issued.  In the middle, when every
  // wave has all it needs of `cur`, the loads of step g+2 go there, and what has
  // arrived in `next` is read in the same way for step g+1: no multiplication waits
  // for a read issued just before it.
  auto step = [&](int g, uint8_t* cur, const uint8_t* next, uint8_t* s_cur, const uint8_t* s_next, const i32x8(&w)[4],
                  i32x8(&w_next)[4]) {
    uint32_t sw_next = 0, sx_next[QS / 4];
    Source from;
    uint32_t at = lane_at;
    asm("" : "+v"(at));  // (addresses are formed in the step, not kept over all of them)
    constexpr int kEach = (LX + LW) / R;  // loads behind each block of the second half
    static_assert(kEach * R == LX + LW && 4 % R == 0, "");
#pragma unroll
    for (int q = 0; q < QB; ++q) {
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if constexpr (EXACT) {
          const float ss = scale_of((sx[q / 4] >> (8 * (q & 3))) & 255u), sc = scale_of(sw);
#pragma unroll
          for (int h = 0; h < 8; h += 2)
            acc[f][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                decode8((uint32_t)w[f][h], (uint32_t)w[f][h + 1], sc),
                decode8((uint32_t)xv[q % R][h], (uint32_t)xv[q % R][h + 1], ss), acc[f][q], 0, 0, 0);
        } else {
          acc[f][q] = mfma_scaled(w[f], xv[q % R], acc[f][q], sw, sx[q / 4], q & 3);
        }
      }
      // (keeps the multiplications here: nothing else orders them and the barrier)
      asm volatile("" : "+v"(acc[0][q]), "+v"(acc[1][q]), "+v"(acc[2][q]), "+v"(acc[3][q]));
      __builtin_amdgcn_sched_barrier(0);
      if (q < R) {
        xv[q % R] = read_x(cur, q + R, at);
      } else {
        if (q == R) {
          // this wave's loads of step g+1 and its reads of step g
          __builtin_amdgcn_s_waitcnt(wait_for(0, 0));
          __syncthreads();
          sw_next = sw_ahead;
          if (tid < TM) s_cur[splace] = (uint8_t)sx_ahead;
          sx_ahead = load_sx(g + 3);
          sw_ahead = load_sw(g + 2);
          from = source(g + 2);
#pragma unroll
          for (int p = 0; p < QS; p += 4)
            sx_next[p / 4] = *reinterpret_cast<const uint32_t*>(s_next + (wm * 16 + r) * QS + p);
        }
        xv[q % R] = read_x(next, q - R, at);
#pragma unroll
        for (int f = (q - R) * 4 / R; f < (q - R + 1) * 4 / R; ++f) w_next[f] = read_w(next, f, at);
#pragma unroll
        for (int k = (q - R) * kEach; k < (q - R + 1) * kEach; ++k) load_codes(from, cur, k);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    sw = sw_next;
#pragma unroll
    for (int p = 0; p < QS / 4; ++p) sx[p] = sx_next[p];
  };

  {
    const uint32_t first = load_sx(0), second = load_sx(1);
    sw = load_sw(0);
    sw_ahead = load_sw(1);
    sx_ahead = load_sx(2);
    const Source f0 = source(0), f1 = source(1);
#pragma unroll
    for (int k = 0; k < LX + LW; ++k) load_codes(f0, s_even, k);
#pragma unroll
    for (int k = 0; k < LX + LW; ++k) load_codes(f1, s_odd, k);
    if (tid < TM) s_scale_even[splace] = (uint8_t)first, s_scale_odd[splace] = (uint8_t)second;
  }
  __builtin_amdgcn_s_waitcnt(wait_for(LX + LW, 0));  // all but the loads of step 1
  __syncthreads();
#pragma unroll
  for (int q = 0; q < QS; q += 4)
    sx[q / 4] = *reinterpret_cast<const uint32_t*>(s_scale_even + (wm * 16 + r) * QS + q);
#pragma unroll
  for (int f = 0; f < 4; ++f) w_even[f] = read_w(s_even, f, lane_at);
#pragma unroll
  for (int q = 0; q < R; ++q) xv[q] = read_x(s_even, q, lane_at);
  for (int g = 0;; g += 2) {
    step(g, s_even, s_odd, s_scale_even, s_scale_odd, w_even, w_odd);
    if (g + 1 >= G) break;  // (no way from the even step to itself: its reads need not wait for its loads)
    step(g + 1, s_odd, s_even, s_scale_odd, s_scale_even, w_odd, w_even);
    if (g + 2 >= G) break;
  }
  // no load into LDS may be under way when the workgroup's LDS is given away, or used anew
  __builtin_amdgcn_s_waitcnt(wait_for(0, 15));
  if constexpr (PARTIAL) {
    sums += (size_t)wave * QB * 4 * 64 + lane;
#pragma unroll
    for (int q = 0; q < QB; ++q)
#pragma unroll
      for (int f = 0; f < 4; ++f) sums[(q * 4 + f) * 64] = acc[f][q];
  } else {
    __syncthreads();  // (a wave's part of LDS is others' buffer)
    finish_rows<QB, OUT_BF16>(acc, i0 + wm * 16 * QB, row_end, jw, n, a.ep,
                              (wave < NW / 2 ? s_even : s_odd) + wave % (NW / 2) * Shape::kPart);
  }
}

// Tile u of tiles_m x tiles_n: bands of 8 row tiles by the column tiles, so that the
// workgroups of an XCD (which take neighbouring u) share records in its L2.
__device__ __forceinline__ void tile_at(int u, int tiles_m, int tiles_n, int& ti, int& tj) {
  const int band = u / (8 * tiles_n), in = u - band * 8 * tiles_n;
  const int high = min(tiles_m - band * 8, 8);
  tj = in / high;
  ti = band * 8 + in - tj * high;
}

// Tiles of 256 x 256 by the 8-bit instruction (fast sums; the decoded operands of exact
// ones have no registers left), one workgroup a CU, for whole rounds of the CUs; the tiles
// left over are cut into PARTS of 256 x 128 or 128 x 128, so that the last round takes every
// CU for the time of a part.  A step takes 2870 cycles, 2048 of them its multiplications'
// (LDS reads and the barrier the rest); before the first step and behind the last one
// nothing multiplies, 3000 and 4000 cycles without an activation: 8192 x 8192 -> 8192
// 380-400 us (2.75-2.9 PFLOP/s), 4608 x 4608 -> 12288 202 (2.6), with GELU from column
// 4608 on 225-238; 4096 x 1152 -> 4608 29 (1.5), with GELU 35.
template <int PARTS>
__global__ __launch_bounds__(512) void fp8_big_kernel(Fp8Args a, int tiles_m, int tiles_n, int full) {
  typedef TileShape<8, 2, 4> Shape;
  __shared__ __align__(16) uint8_t s_even[Shape::kBuffer];
  __shared__ __align__(16) uint8_t s_odd[Shape::kBuffer];
  __shared__ __align__(16) uint8_t s_scale_even[Shape::kScales];
  __shared__ __align__(16) uint8_t s_scale_odd[Shape::kScales];
  const int d = (int)blockIdx.x;
  int ti, tj;
  if (PARTS == 1 || d < full) {
    tile_at(xcd_range(d, full), tiles_m, tiles_n, ti, tj);
    tile<8, 2, 4, false, true, false, false>(a, a.qx, a.ascale, a.qw, a.wscale, a.bias, a.G, ti * 256, tj * 256, a.b,
                                             s_even, s_odd, s_scale_even, s_scale_odd, nullptr);
    return;
  }
  if constexpr (PARTS > 1) {
    const int u = xcd_range(d - full, (tiles_m * tiles_n - full) * PARTS);
    tile_at(full + u / PARTS, tiles_m, tiles_n, ti, tj);
    const int i0 = ti * 256 + (PARTS == 4 ? 128 * (u >> 1 & 1) : 0), j0 = tj * 256 + 128 * (u & 1);
    if (i0 >= a.b || j0 >= a.n) return;  // (the whole workgroup)
    if constexpr (PARTS == 2)
      tile<4, 4, 2, false, true, false, false>(a, a.qx, a.ascale, a.qw, a.wscale, a.bias, a.G, i0, j0, a.b, s_even,
                                               s_odd, s_scale_even, s_scale_odd, nullptr);
    else
      tile<2, 4, 2, false, true, false, false>(a, a.qx, a.ascale, a.qw, a.wscale, a.bias, a.G, i0, j0, a.b, s_even,
                                               s_odd, s_scale_even, s_scale_odd, nullptr);
  }
}

// The tile of rows sorted by expert that this workgroup takes (grouped.h), with its
// expert's operands; false: none.  An expert's row blocks of one column block are
// neighbours: they share its weights in L2.
struct GroupedTile {
  const uint8_t *qw, *wscale;
  const uint16_t* bias;
  int i0, j0, row_end;
};
template <int TM, int TN>
__device__ __forceinline__ bool grouped_tile(const Fp8Args& a, int tiles_n, GroupedTile& t) {
  const GroupTile g = find_tile<TM>(a.groups.offsets, a.groups.experts, a.b, tiles_n, (int)blockIdx.x,
                                    [](int d, int T) { return xcd_range(d, T); });
  if (!g.live) return false;
  const int tj = g.u / g.blocks;
  const size_t e = (size_t)g.expert;
  t.qw = a.qw + e * a.G * (size_t)a.n * 128;
  t.wscale = a.wscale + e * a.G * ((a.n + 127) / 128);
  t.bias = a.bias ? a.bias + e * a.n : nullptr;
  t.i0 = g.lo + (g.u - tj * g.blocks) * TM;
  t.j0 = tj * TN;
  t.row_end = g.hi;
  return true;
}

// 256 x 256 for experts of many rows (8 experts, 2048 rows each of 4096 -> 4096 252 us,
// 2.2 PFLOP/s).
__global__ __launch_bounds__(512) void fp8_big_grouped_kernel(Fp8Args a, int tiles_n) {
  typedef TileShape<8, 2, 4> Shape;
  __shared__ __align__(16) uint8_t s_even[Shape::kBuffer];
  __shared__ __align__(16) uint8_t s_odd[Shape::kBuffer];
  __shared__ __align__(16) uint8_t s_scale_even[Shape::kScales];
  __shared__ __align__(16) uint8_t s_scale_odd[Shape::kScales];
  GroupedTile t;
  if (!grouped_tile<256, 256>(a, tiles_n, t)) return;  // the whole workgroup
  tile<8, 2, 4, false, true, true, false>(a, a.qx, a.ascale, t.qw, t.wscale, t.bias, a.G, t.i0, t.j0, t.row_end, s_even,
                                          s_odd, s_scale_even, s_scale_odd, nullptr);
}

// Tiles of 128 x 128, two workgroups a CU (of which one ends while the other multiplies):
// every product of many rows with exact sums (the bf16 instruction: 8192 x 8192 -> 8192
// 885 us, 1.24 PFLOP/s, where a library's bf16 product reaches 1.3-1.37; 4608 x 4608 ->
// 12288 with GELU 453; 4096 x 1152 -> 4608 with GELU 55, its 1152 tiles 2.25 rounds of the
// CUs), experts' rows (64 experts, 18006 rows of 2048 -> 1408 135 us, fast sums 101; a
// quarter of the tiles' rows are no expert's: fast sums 73 at even counts), and few tiles,
// which may be split along the channels (PIECES: piece p of tile u takes every block
// from p G / pieces to (p + 1) G / pieces and leaves its sums in slot u pieces + p).
template <bool EXACT, bool OUT_BF16, bool GROUPED, bool PIECES>
__global__ __launch_bounds__(256) void fp8_tile_kernel(Fp8Args a, int tiles_m, int tiles_n, int pieces, f32x4* sums) {
  typedef TileShape<4, 2, 2> Shape;
  __shared__ __align__(16) uint8_t s_even[Shape::kBuffer];
  __shared__ __align__(16) uint8_t s_odd[Shape::kBuffer];
  __shared__ __align__(16) uint8_t s_scale_even[Shape::kScales];
  __shared__ __align__(16) uint8_t s_scale_odd[Shape::kScales];
  const uint8_t *qx = a.qx, *ascale = a.ascale, *qw = a.qw, *wscale = a.wscale;
  const uint16_t* bias = a.bias;
  const int NB = (a.n + 127) / 128;
  int i0, j0, row_end, G = a.G;
  if constexpr (GROUPED) {
    GroupedTile t;
    if (!grouped_tile<128, 128>(a, tiles_n, t)) return;  // the whole workgroup
    qw = t.qw;
    wscale = t.wscale;
    bias = t.bias;
    i0 = t.i0;
    j0 = t.j0;
    row_end = t.row_end;
  } else {
    const int u = xcd_range((int)blockIdx.x, tiles_m * tiles_n * pieces);
    int ti, tj;
    tile_at(u / pieces, tiles_m, tiles_n, ti, tj);
    i0 = ti * 128;
    j0 = tj * 128;
    row_end = a.b;
    if constexpr (PIECES) {
      const int p = u % pieces, g0 = (int)((long long)G * p / pieces);
      G = (int)((long long)G * (p + 1) / pieces) - g0;
      qx += (size_t)g0 * a.x_rows * 128;
      ascale += (size_t)g0 * a.x_rows;
      qw += (size_t)g0 * a.n * 128;
      wscale += (size_t)g0 * NB;
      sums += (size_t)u * (128 * 128 / 4);
    }
  }
  tile<4, 2, 2, EXACT, OUT_BF16, GROUPED, PIECES>(a, qx, ascale, qw, wscale, bias, G, i0, j0, row_end, s_even, s_odd,
                                                  s_scale_even, s_scale_odd, sums);
}

// Tiles of 64 x 128, three workgroups a CU, where those of 128 x 128 leave CUs idle: half
// the multiplications in a step's chain (333 rows, 1000 -> 1500 in fp32: 9.9 us, where
// 36 tiles of 128 x 128 take 13.5).
template <bool EXACT, bool OUT_BF16>
__global__ __launch_bounds__(256) void fp8_small_kernel(Fp8Args a, int tiles_m, int tiles_n) {
  typedef TileShape<2, 2, 2> Shape;
  __shared__ __align__(16) uint8_t s_even[Shape::kBuffer];
  __shared__ __align__(16) uint8_t s_odd[Shape::kBuffer];
  __shared__ __align__(16) uint8_t s_scale_even[Shape::kScales];
  __shared__ __align__(16) uint8_t s_scale_odd[Shape::kScales];
  int ti, tj;
  tile_at(xcd_range((int)blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, ti, tj);
  tile<2, 2, 2, EXACT, OUT_BF16, false, false>(a, a.qx, a.ascale, a.qw, a.wscale, a.bias, a.G, ti * 64, tj * 128, a.b,
                                               s_even, s_odd, s_scale_even, s_scale_odd, nullptr);
}

// The pieces' sums of a tile added in their order, the bias, and the rest.  A workgroup
// takes the blocks q of 16 rows of the tile's four waves.
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void fp8_pieces_kernel(Fp8Args a, int tiles_m, int tiles_n, int pieces,
                                                         const f32x4* __restrict__ sums) {
  __shared__ __align__(16) uint8_t s_part[4][32 * 272];
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int u = (int)blockIdx.x >> 2, q = (int)blockIdx.x & 3;
  int ti, tj;
  tile_at(u, tiles_m, tiles_n, ti, tj);
  const f32x4* from = sums + (size_t)u * pieces * (128 * 128 / 4) + (wave * 16 + q * 4) * 64 + lane;
  const int jw = tj * 128 + 64 * (wave & 1);
  f32x4 acc[4][1];
#pragma unroll
  for (int f = 0; f < 4; ++f) acc[f][0] = from[f * 64];
  for (int p = 1; p < pieces; ++p) {
    from += 128 * 128 / 4;
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f][0] += from[f * 64];
  }
  if (a.bias) {
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f][0] += load4<true>(a.bias, column_of<OUT_BF16>(jw, lane >> 4, f), a.n);
  }
  finish_rows<1, OUT_BF16>(acc, ti * 128 + (wave >> 1) * 64 + 16 * q, a.b, jw, a.n, a.ep, s_part[wave]);
}

}  // namespace

int launch_fp8_tiles(const Fp8Args& a, const Fp8Plan& p, int y_dtype, void* ws, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const bool bf = y_dtype == SVDQ_OUT_BF16;
  if (p.big) {
    const int tm = (a.b + 255) / 256, tn = (a.n + 255) / 256;
    if (a.groups.offsets) return launch_checked(fp8_big_grouped_kernel, p.split.grid, 512, st, a, tn);
    auto go = [&](auto kernel) { return launch_checked(kernel, p.split.grid, 512, st, a, tm, tn, p.full); };
    return p.parts == 1 ? go(fp8_big_kernel<1>) : p.parts == 2 ? go(fp8_big_kernel<2>) : go(fp8_big_kernel<4>);
  }
  const int tm = (a.b + 127) / 128, tn = (a.n + 127) / 128;
  if (p.small) {
    auto go = [&](auto kernel) { return launch_checked(kernel, p.split.grid, 256, st, a, (a.b + 63) / 64, tn); };
    if (p.fast) return go(fp8_small_kernel<false, true>);
    return bf ? go(fp8_small_kernel<true, true>) : go(fp8_small_kernel<true, false>);
  }
  f32x4* sums = reinterpret_cast<f32x4*>(ws);
  auto go = [&](auto kernel) { return launch_checked(kernel, p.split.grid, 256, st, a, tm, tn, p.pieces, sums); };
  // (the kinds of sums and of y that there are)
  auto pick = [&](auto GROUPED, auto PIECES) {
    constexpr bool g = decltype(GROUPED)::value, k = decltype(PIECES)::value;
    if (p.fast) return go(fp8_tile_kernel<false, true, g, k>);
    return bf ? go(fp8_tile_kernel<true, true, g, k>) : go(fp8_tile_kernel<true, false, g, k>);
  };
  if (a.groups.offsets) return pick(std::true_type{}, std::false_type{});
  if (p.pieces == 1) return pick(std::false_type{}, std::false_type{});
  const int status = pick(std::false_type{}, std::true_type{});
  if (status != 0) return status;
  auto join = [&](auto kernel) {
    return launch_checked(kernel, (long long)tm * tn * 4, 256, st, a, tm, tn, p.pieces, (const f32x4*)sums);
  };
  return bf ? join(fp8_pieces_kernel<true>) : join(fp8_pieces_kernel<false>);
}

}  // namespace svdq
