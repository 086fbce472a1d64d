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
// lanes of an operand read, 16 records at the same piece, fall on all 64 banks.
__device__ __forceinline__ int record_key(int r) { return (r >> 1) & 7; }

template <int QB, int NWM, int NWN, bool EXACT, bool OUT_BF16, bool GROUPED>
__global__ __launch_bounds__(64 * NWM * NWN) void fp8_tile_kernel(Fp8Args a, int tiles_m, int tiles_n) {
  constexpr int TM = 16 * QB * NWM, TN = 64 * NWN, NW = NWM * NWN;
  constexpr int LX = TM / (8 * NW), LW = TN / (8 * NW);  // 8-record loads a wave and step
  static_assert(LX * 8 * NW == TM && LW * 8 * NW == TN && TM <= 64 * NW, "whole loads");
  // Two buffers of a step's records (rows, then columns) and of its rows' scales
  // ([wave row][16 rows][QB]); arrays of their own, so that the compiler sees that
  // loads into one are apart from reads of the other.
  __shared__ __align__(16) uint8_t s_even[(TM + TN) * 128];
  __shared__ __align__(16) uint8_t s_odd[(TM + TN) * 128];
  __shared__ __align__(16) uint8_t s_scale_even[TM];
  __shared__ __align__(16) uint8_t s_scale_odd[TM];
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / NWN, wn = wave - wm * NWN;
  const int r = lane & 15, c = lane >> 4;
  const int n = a.n, G = a.G, NB = (n + 127) / 128, xr = a.x_rows;
  const uint8_t* qw = a.qw;
  const uint8_t* wscale = a.wscale;
  const uint16_t* bias = a.bias;
  int i0, j0, row_end;
  if constexpr (GROUPED) {
    const GroupTile g = find_tile<TM>(a.groups.offsets, a.groups.experts, a.b, tiles_n, (int)blockIdx.x,
                                      [](int d, int T) { return xcd_range(d, T); });
    if (!g.live) return;  // the whole workgroup
    const int tj = g.u / g.blocks;
    i0 = g.lo + (g.u - tj * g.blocks) * TM;
    j0 = tj * TN;
    row_end = g.hi;
    const size_t e = (size_t)g.expert;
    qw += e * G * (size_t)n * 128;
    wscale += e * G * NB;
    if (bias) bias += e * n;
  } else {
    // an XCD's workgroups take blocks of 8 row tiles by the column tiles, so that
    // those running together share records in its L2
    const int u = xcd_range((int)blockIdx.x, tiles_m * tiles_n);
    const int band = u / (8 * tiles_n), in = u - band * 8 * tiles_n;
    const int high = min(tiles_m - band * 8, 8), tj = in / high;
    i0 = (band * 8 + in - tj * high) * TM;
    j0 = tj * TN;
    row_end = a.b;
  }

  // what this lane loads: piece (lane & 7) of records 8 (wave + NW i) + lane / 8
  uint32_t xoff[LX], woff[LW];
#pragma unroll
  for (int i = 0; i < LX; ++i) {
    const int rec = 8 * (wave + NW * i) + (lane >> 3);
    int s = i0 + rec < row_end ? i0 + rec : -1;
    if (GROUPED && s >= 0 && a.row_index) s = a.row_index[s];
    xoff[i] = ((unsigned)s < (unsigned)xr ? (uint32_t)s * 128u : 0x7FFFFF80u) + 16u * ((lane & 7) ^ record_key(rec));
  }
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    // record 64 w + 16 f + 4 c + v holds column 64 w + 16 c + 4 f + v: a lane's
    // results of the four blocks f are then 16 neighbouring columns
    const int rec = 8 * (wave + NW * i) + (lane >> 3);
    const int col = j0 + (rec & ~63) + 16 * ((rec >> 2) & 3) + 4 * ((rec >> 4) & 3) + (rec & 3);
    woff[i] = (uint32_t)col * 128u + 16u * ((lane & 7) ^ record_key(rec));
  }
  // the row whose scale this thread stages, and its place
  uint32_t soff = 0x7FFFFFFFu;
  if (tid < TM && i0 + tid < row_end) {
    int s = i0 + tid;
    if (GROUPED && a.row_index) s = a.row_index[s];
    if ((unsigned)s < (unsigned)xr) soff = (uint32_t)s;
  }
  const int splace = (tid / (16 * QB)) * 16 * QB + (tid & 15) * QB + (tid >> 4) % QB;

  auto load_codes = [&](int g, uint8_t* to) {  // (past the last step zeros, without memory traffic)
    const size_t at = g < G ? (size_t)g : 0;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.qx + at * xr * 128, g < G ? (uint32_t)xr * 128u : 0u);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(qw + at * n * 128, g < G ? (uint32_t)n * 128u : 0u);
#pragma unroll
    for (int i = 0; i < LX; ++i) load_to_lds(rx, xoff[i], to + 1024 * (wave + NW * i));
#pragma unroll
    for (int i = 0; i < LW; ++i) load_to_lds(rw, woff[i], to + TM * 128 + 1024 * (wave + NW * i));
  };
  // (past the last step the last one's, unused)
  auto load_sx = [&](int g) -> uint32_t {
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.ascale + (size_t)min(g, G - 1) * xr, (uint32_t)xr);
    return __builtin_amdgcn_raw_buffer_load_b8(rx, soff, 0, 0);
  };
  auto load_sw = [&](int g) -> uint32_t {
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(wscale + (size_t)min(g, G - 1) * NB, (uint32_t)NB);
    return __builtin_amdgcn_raw_buffer_load_b8(rw, (uint32_t)(j0 + 64 * wn) / 128u, 0, 0);
  };
  auto read = [&](const uint8_t* records, int rec) -> i32x8 {
    const uint8_t* p = records + rec * 128;
    const int key = record_key(rec);
    return operand(*reinterpret_cast<const u32x4*>(p + 16 * ((2 * c) ^ key)),
                   *reinterpret_cast<const u32x4*>(p + 16 * ((2 * c + 1) ^ key)));
  };
  auto read_w = [&](const uint8_t* buf, int f) { return read(buf + TM * 128 + wn * 8192, 16 * f + r); };
  auto read_x = [&](const uint8_t* buf, int q) { return read(buf + wm * QB * 2048, 16 * q + r); };

  f32x4 acc[4][QB];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int q = 0; q < QB; ++q) acc[f][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  i32x8 wv[4], xv[QB];
  uint32_t sx[QB / 4], sw;         // the step's scales: bytes of the rows' four blocks, the columns'
  uint32_t sx_ahead, sw_ahead;     // in flight: the byte this thread stages, two steps ahead; the columns', one ahead

  // A step: the operands of step g are in registers (or on their way), step g+1's
  // records in `next` or on their way there, and `cur` is free once every wave has
  // its operands of step g.  Each operand's registers are read again from `next`
  // as soon as its last multiplication has been issued.
  auto step = [&](int g, uint8_t* cur, const uint8_t* next, uint8_t* s_cur, const uint8_t* s_next) {
    auto multiply = [&](int f, int q) {
      if constexpr (EXACT) {
        const float ss = scale_of((sx[q / 4] >> (8 * (q & 3))) & 255u), sc = scale_of(sw);
#pragma unroll
        for (int h = 0; h < 4; ++h)
          acc[f][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              decode8((uint32_t)wv[f][2 * h], (uint32_t)wv[f][2 * h + 1], sc),
              decode8((uint32_t)xv[q][2 * h], (uint32_t)xv[q][2 * h + 1], ss), acc[f][q], 0, 0, 0);
      } else {
        acc[f][q] = mfma_scaled(wv[f], xv[q], acc[f][q], sw, sx[q / 4], q & 3);
      }
    };
#pragma unroll
    for (int f = 0; f < 4; ++f) multiply(f, 0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0): this wave's loads of step g+1 and its reads of step g
    __syncthreads();
    const uint32_t sw_next = sw_ahead;
    if (tid < TM) s_cur[splace] = (uint8_t)sx_ahead;
    sx_ahead = load_sx(g + 3);
    sw_ahead = load_sw(g + 2);
    load_codes(g + 2, cur);
    uint32_t sx_next[QB / 4];
#pragma unroll
    for (int q = 0; q < QB; q += 4)
      sx_next[q / 4] = *reinterpret_cast<const uint32_t*>(s_next + wm * 16 * QB + r * QB + q);
    xv[0] = read_x(next, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 1; q < QB; ++q) {
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        multiply(f, q);
        if (q == QB - 1) {
          __builtin_amdgcn_sched_barrier(0);
          wv[f] = read_w(next, f);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      xv[q] = read_x(next, q);
      __builtin_amdgcn_sched_barrier(0);
    }
    sw = sw_next;
#pragma unroll
    for (int q = 0; q < QB / 4; ++q) sx[q] = sx_next[q];
  };

  load_codes(0, s_even);
  {
    const uint32_t first = load_sx(0), second = load_sx(1);
    sw = load_sw(0);
    sw_ahead = load_sw(1);
    sx_ahead = load_sx(2);
    if (tid < TM) s_scale_even[splace] = (uint8_t)first, s_scale_odd[splace] = (uint8_t)second;
  }
  __builtin_amdgcn_s_waitcnt(0x0070);
  __syncthreads();
  load_codes(1, s_odd);
#pragma unroll
  for (int q = 0; q < QB; q += 4)
    sx[q / 4] = *reinterpret_cast<const uint32_t*>(s_scale_even + wm * 16 * QB + r * QB + q);
#pragma unroll
  for (int f = 0; f < 4; ++f) wv[f] = read_w(s_even, f);
#pragma unroll
  for (int q = 0; q < QB; ++q) xv[q] = read_x(s_even, q);
  for (int g = 0; g < G; g += 2) {
    step(g, s_even, s_odd, s_scale_even, s_scale_odd);
    if (g + 1 < G) step(g + 1, s_odd, s_even, s_scale_odd, s_scale_even);
  }
  // no load into LDS may be under way when the workgroup's LDS is given away
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)

  // rows 16 q + r of the wave, 16 columns from 16 c on
  const int j = j0 + 64 * wn + 16 * c;
  if (j >= n) return;
  constexpr int W = OUT_BF16 ? 8 : 4;
  float bv[16];
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    const f32x4 t = bias ? load4<true>(bias, j + e, n) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < 4; ++v) bv[e + v] = t[v];
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int i = i0 + wm * 16 * QB + 16 * q + r;
    if (i >= row_end) continue;
#pragma unroll
    for (int e0 = 0; e0 < 16; e0 += W) {
      if (j + e0 >= n) break;
      float v[W];
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = acc[(e0 + e) / 4][q][e & 3] + bv[e0 + e];
      with_act(a.ep.act, [&](auto A) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float t = act_value<decltype(A)::value>(v[e]);
          v[e] = j + e0 + e >= a.ep.act_begin ? t : v[e];
        }
      });
      if (a.ep.gate) {
        const uint16_t* row = reinterpret_cast<const uint16_t*>(row_of<true>(a.ep.gate, i / a.ep.gate_rows, n));
        float gv[W];
        load_cols<W, true>(row, j + e0, n, gv);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] *= gv[e];
      }
      if (a.ep.residual) {
        float rv[W];
        load_cols<W, OUT_BF16>(row_of<OUT_BF16>(a.ep.residual, i, a.ep.ldr), j + e0, n, rv);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = rv[e] + v[e];
      }
      store_cols<W, OUT_BF16>(row_of<OUT_BF16>(a.ep.y, i, a.ep.ldy), j + e0, n, v);
    }
  }
}

template <int QB, int NWM, int NWN, bool EXACT, bool OUT_BF16, bool GROUPED>
int launch_tiles_typed(const Fp8Args& a, const Fp8Plan& p, hipStream_t st) {
  constexpr int TM = 16 * QB * NWM, TN = 64 * NWN, threads = 64 * NWM * NWN;
  auto kernel = fp8_tile_kernel<QB, NWM, NWN, EXACT, OUT_BF16, GROUPED>;
  if (!launch_fits(p.split.grid, threads)) return (int)hipErrorInvalidConfiguration;
  const int ok = scratch_free(reinterpret_cast<const void*>(kernel));
  if (ok != 0) return ok;
  hipLaunchKernelGGL(kernel, dim3((unsigned)p.split.grid), dim3(threads), 0, st, a, (a.b + TM - 1) / TM,
                     (a.n + TN - 1) / TN);
  return (int)hipGetLastError();
}

template <int QB, int NWM, int NWN, bool EXACT>
int launch_tiles(const Fp8Args& a, const Fp8Plan& p, hipStream_t st) {
  return a.groups.offsets ? launch_tiles_typed<QB, NWM, NWN, EXACT, !EXACT, true>(a, p, st)
                          : launch_tiles_typed<QB, NWM, NWN, EXACT, !EXACT, false>(a, p, st);
}

}  // namespace

int launch_fp8_tiles(const Fp8Args& a, const Fp8Plan& p, int y_dtype, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const bool exact = y_dtype == SVDQ_OUT_F32;
  if (p.tile_m == 256 && !exact) return launch_tiles<8, 2, 4, false>(a, p, st);
  if (p.tile_m == 128) return exact ? launch_tiles<4, 2, 2, true>(a, p, st) : launch_tiles<4, 2, 2, false>(a, p, st);
  return (int)hipErrorInvalidValue;
}

}  // namespace svdq
