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
  const int splace = (tid / (16 * QB)) * 16 * QB + (tid & 15) * QB + (tid >> 4) % QB;

  struct Source {
    __amdgpu_buffer_rsrc_t x, w;
    uint32_t x0, w0;
  };
  auto source = [&](int g) {  // (past the last step zeros, without memory traffic)
    const size_t at = g < G ? (size_t)g : 0;
    Source f{make_rsrc(a.qx + at * xr * 128, g < G ? (uint32_t)xr * 128u : 0u),
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
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.ascale + (size_t)min(g, G - 1) * xr, (uint32_t)xr);
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
  auto column = [&](int f) { return jw + (OUT_BF16 ? 32 * (f >> 1) + 8 * c + 4 * (f & 1) : 16 * f + 4 * c); };
  f32x4 acc[4][QB];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const f32x4 t = bias ? load4<true>(bias, column(f), n) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < QB; ++q) acc[f][q] = t;
  }
  constexpr int R = QB / 2;     // blocks of rows in registers at a time
  i32x8 w_even[4], w_odd[4], xv[R];
  uint32_t sx[QB / 4], sw;      // the step's scales: bytes of the rows' four blocks, the columns'
  uint32_t sx_ahead, sw_ahead;  // in flight: the byte this thread stages, two steps ahead; the columns', one ahead

  // A step.  Its columns and its first R blocks of rows are in registers (or on their
  // way), the other blocks follow from `cur`, each into the registers of the block R
  // before it once that one's multiplications are issued.  In the middle, when every
  // wave has all it needs of `cur`, the loads of step g+2 go there, and what has
  // arrived in `next` is read in the same way for step g+1: no multiplication waits
  // for a read issued just before it.
  auto step = [&](int g, uint8_t* cur, const uint8_t* next, uint8_t* s_cur, const uint8_t* s_next, const i32x8(&w)[4],
                  i32x8(&w_next)[4]) {
    uint32_t sw_next = 0, sx_next[QB / 4];
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
          for (int p = 0; p < QB; p += 4)
            sx_next[p / 4] = *reinterpret_cast<const uint32_t*>(s_next + wm * 16 * QB + r * QB + p);
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
    for (int p = 0; p < QB / 4; ++p) sx[p] = sx_next[p];
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
  for (int q = 0; q < QB; q += 4)
    sx[q / 4] = *reinterpret_cast<const uint32_t*>(s_scale_even + wm * 16 * QB + r * QB + q);
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

  // The activation, gate and residual, and y's rounding.  A lane holds W neighbouring
  // columns of a row in each of UNITS units; four lanes' are 64 bytes of y.
  constexpr int W = OUT_BF16 ? 8 : 4, UNITS = 16 / W;
  const int row0 = i0 + wm * 16 * QB;
  const int begin = a.ep.act == SVDQ_ACT_NONE ? n : a.ep.act_begin;
  if (j0 + TN <= n && (begin <= j0 || begin >= j0 + TN || (begin - j0) % 64 == 0)) {
    // Whole columns, each wave's all with the activation or all without: straight code,
    // one copy for each case.  (With every case inside one loop over the accumulators
    // the instructions to be fetched, anew for every launch, cost more than the stores:
    // 256 x 128 -> 256, one tile: 7.6 us.)
    auto finish = [&](auto A, auto MORE) {
      uint8_t* y = reinterpret_cast<uint8_t*>(row_of<OUT_BF16>(a.ep.y, row0 + r, a.ep.ldy)) + (jw + W * c) * (OUT_BF16 ? 2 : 4);
      const size_t next = (size_t)16 * a.ep.ldy * (OUT_BF16 ? 2 : 4);
#pragma unroll
      for (int q = 0; q < QB; ++q, y += next) {
        const int i = row0 + 16 * q + r;
        if (i >= row_end) break;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          float v[W];
#pragma unroll
          for (int e = 0; e < W; ++e) v[e] = act_value<decltype(A)::value>(acc[W / 4 * u + e / 4][q][e & 3]);
          if constexpr (decltype(MORE)::value) {
            const int j = jw + W * c + 4 * W * u;
            if (a.ep.gate) {
              float gv[W];
              load_whole<W, true>(row_of<true>(a.ep.gate, i / a.ep.gate_rows, n), j, gv);
#pragma unroll
              for (int e = 0; e < W; ++e) v[e] *= gv[e];
            }
            if (a.ep.residual) {
              float rv[W];
              load_whole<W, OUT_BF16>(row_of<OUT_BF16>(a.ep.residual, i, a.ep.ldr), j, rv);
#pragma unroll
              for (int e = 0; e < W; ++e) v[e] = rv[e] + v[e];
            }
          }
          store_whole<W, OUT_BF16>(y + 64 * u, v);
        }
      }
    };
    auto with_more = [&](auto A) {
      if (a.ep.gate || a.ep.residual)
        finish(A, std::true_type{});
      else
        finish(A, std::false_type{});
    };
    if (begin >= jw + 64)
      with_more(std::integral_constant<int, SVDQ_ACT_NONE>{});
    else
      with_act(a.ep.act, with_more);
    return;
  }

  // The other tiles: 32 rows at a time through the wave's own part of LDS and one loop
  // over the rows, with every column's own case.
  __syncthreads();  // every wave is done with the buffers
  constexpr int LANES = 64 / W;  // lanes of a row
  constexpr int kPitch = 272;    // bytes of a row of 64 sums: rows on different banks
  uint8_t* part = (wave < NW / 2 ? s_even : s_odd) + (wave % (NW / 2)) * 32 * kPitch;
  static_assert(NW / 2 * 32 * kPitch <= (TM + TN) * 128, "the waves' parts fit the buffers");
  const int rr = lane / LANES, cc = lane % LANES;
  const int j = jw + W * cc;
#pragma unroll 1
  for (int p = 0; p < QB / 2; ++p) {
#pragma unroll
    for (int b = 0; b < QB / 2; ++b)
      if (b == p) {  // (accumulators are registers: a branch for each pair of blocks)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int f = 0; f < 4; ++f)
            *reinterpret_cast<f32x4*>(part + (16 * h + r) * kPitch + (column(f) - jw) * 4) = acc[f][2 * b + h];
      }
    // other lanes' results: LDS accesses of one wave complete in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int k = rr; k < 32; k += 64 / LANES) {
      const int i = row0 + 32 * p + k;
      if (i < row_end && j < n) {
        float v[W];
#pragma unroll
        for (int e = 0; e < W; e += 4) {
          const f32x4 t = *reinterpret_cast<const f32x4*>(part + k * kPitch + (W * cc + e) * 4);
#pragma unroll
          for (int x = 0; x < 4; ++x) v[e + x] = t[x];
        }
        with_act(a.ep.act, [&](auto A) {
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float t = act_value<decltype(A)::value>(v[e]);
            v[e] = j + e >= a.ep.act_begin ? t : v[e];
          }
        });
        if (a.ep.gate) {
          float gv[W];
          load_cols<W, true>(row_of<true>(a.ep.gate, i / a.ep.gate_rows, n), j, n, gv);
#pragma unroll
          for (int e = 0; e < W; ++e) v[e] *= gv[e];
        }
        if (a.ep.residual) {
          float rv[W];
          load_cols<W, OUT_BF16>(row_of<OUT_BF16>(a.ep.residual, i, a.ep.ldr), j, n, rv);
#pragma unroll
          for (int e = 0; e < W; ++e) v[e] = rv[e] + v[e];
        }
        store_cols<W, OUT_BF16>(row_of<OUT_BF16>(a.ep.y, i, a.ep.ldy), j, n, v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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
