// INT4 and NVFP4 products with an epilogue for few rows (up to 64, or 16 or 32
// rows of one INT4 expert at a time): the layer's weights bound it.
//
// Y = epilogue(sum_g sx[g,i] sw[g,j] isum[i,j,g] + (bf16(Z) L2)[i,j] + bias[j]),
// with the exact per-group integer sums and the two FMAs per element and group
// of the tiled kernel (gemm_body.h); NVFP4: the sum of the products of the
// dequantized values (exact f16), times the tensor scales, as there.
//
// A wave computes 16 columns of RB blocks of 16 rows.  Of a workgroup's waves,
// nwk split the channel groups of the same columns (wave k takes groups k,
// k + nwk, ...; their sums are added in LDS in wave order) and nwc take
// neighbouring columns.  Nothing is staged in LDS before that: a lane's
// MFMA operand (16 codes of one row or column) is 8 bytes of its packed record,
// so weights and activations go from memory to registers to the MFMA, D groups
// ahead.  Any channel order serves, as both operands unpack alike.
//
// Measured: 64 experts, 128 rows, 2048 -> 1408: 19.0 us (17.4 at the least) for 93
// MB, nearly all weights, 4.9 TB/s (a large copy reaches 5.1).  One row, 4608 ->
// 1152: 5.8 us, and 13 rows, 2048 -> 5001: 6.1 us, which is a launch and one chain of dependent
// loads, not bandwidth.  Against tiles (12288 -> 3000, one layer): 1 to 64 rows
// 10.5-17 us, tiles 20-24 us; for 65 to 128 rows it was faster on some shapes and
// 20-25 % slower on others, so tiles take those.  NVFP4 against split tiles, 8192
// -> 8192: 1 row 12.3 / 28.4 us, 32 rows 17.4 / 29.5, 64 rows 25.4 / 30.1; 4608 ->
// 1152: 9.0 / 14.2, 9.2 / 13.7, 11.0 / 14.2.
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "epilogue.h"
#include "grouped.h"
#include "internal.h"
#include "launch.h"

#pragma clang fp contract(off)

namespace svdq {
namespace {

using namespace dev;

// Groups in flight per wave: 12 bytes of codes and scales a lane, group and row
// block; deeper needs registers that cost resident waves.
constexpr int rows_depth(int rb) { return rb == 1 ? 6 : (rb == 2 ? 4 : 3); }

// FMT: kFmtInt4, or kFmtFp4 (NVFP4: the lane's 8 bytes are one block of 16
// channels, dequantized to f16 and multiplied by two f16 MFMAs; the low-rank
// product is added after the tensor scales txw).
// SWV (INT4): the four scales of a lane's columns are one aligned 8-byte load.
template <int RB, bool OUT_BF16, bool GROUPED, int FMT, bool SWV>
__global__ __launch_bounds__(RB == 4 ? 512 : 1024) void gemm_w4a4_rows_kernel(RowsArgs a, int nwk, int nwc) {
  extern __shared__ __align__(16) uint8_t rows_lds[];
  f32x4* part = reinterpret_cast<f32x4*>(rows_lds);  // [wave][row block][lane]
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ct = wave / nwk, wk = wave - ct * nwk;  // this wave's column block and share of the groups
  const int r = lane & 15, c = lane >> 4;
  const int b = a.b, n = a.n, G = a.G, rank = a.rank;
  const int tiles_n = (n + 16 * nwc - 1) / (16 * nwc);

  const uint8_t* qw = a.qw;
  const uint16_t* wscale = a.wscale;
  const uint16_t* l2 = a.l2;
  const uint16_t* bias = a.bias;
  int i0, j00, row_end;  // first row, the workgroup's first column, end of the rows
  if constexpr (GROUPED) {
    const GroupTile g = find_tile<16 * RB>(a.groups.offsets, a.groups.experts, b, tiles_n, (int)blockIdx.x,
                                           [](int d, int T) { return xcd_range(d, T); });
    if (!g.live) return;  // every wave finds the same tile
    // an expert's row blocks of one column block are neighbours: they share its weights in L2
    const int tj = g.u / g.blocks;
    i0 = g.lo + (g.u - tj * g.blocks) * 16 * RB;
    j00 = tj * 16 * nwc;
    row_end = g.hi;
    const size_t e = (size_t)g.expert;
    qw += e * G * n * 32;
    wscale += e * G * n;
    if (rank > 0) l2 += e * n * rank;
    if (bias) bias += e * n;
  } else {
    i0 = 0;
    j00 = (int)blockIdx.x * 16 * nwc;
    row_end = b;
  }
  const int j0 = j00 + 16 * ct;
  constexpr bool F4 = FMT == kFmtFp4;

  struct Stage {
    uint2 w, a[RB];   // packed codes: this lane's 8 bytes of its column's and rows' records
    uint2 sw;         // fp16 scales of columns 4c .. 4c+3; NVFP4: x, the block scale of the lane's column
    uint32_t sx[RB];  // fp16 scales of the rows; NVFP4: the block scales of the lane's rows
  };
  const int nk = wk < G ? (G - wk + nwk - 1) / nwk : 0;  // groups of this wave
  const uint32_t w_off = (uint32_t)(j0 + r) * 32u + 8u * c;
  const uint32_t s_off = (uint32_t)(j0 + 4 * c) * 2u;
  auto load = [&](int k, Stage& st) {
    const bool live = k < nk;
    const int g = live ? wk + nwk * k : 0;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(qw + (size_t)g * n * 32, live ? (uint32_t)n * 32u : 0u);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.qx + (size_t)g * b * 32, live ? (uint32_t)b * 32u : 0u);
    constexpr int SB = F4 ? 4 : 2;  // bytes of scales a row and group
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(wscale + (size_t)g * n * (SB / 2), live ? (uint32_t)n * SB : 0u);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.ascale + (size_t)g * b * (SB / 2), live ? (uint32_t)b * SB : 0u);
    st.w = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rw, w_off, 0, 0));
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const uint32_t row = (uint32_t)(i0 + 16 * q + r);
      st.a[q] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rx, row * 32u + 8u * c, 0, 0));
      if constexpr (F4)
        st.sx[q] = __builtin_amdgcn_raw_buffer_load_b8(ra, row * 4u + c, 0, 0);
      else
        st.sx[q] = __builtin_amdgcn_raw_buffer_load_b16(ra, row * 2u, 0, 0);
    }
    if constexpr (F4) {
      st.sw.x = __builtin_amdgcn_raw_buffer_load_b8(rs, (uint32_t)(j0 + r) * 4u + c, 0, 0);
    } else if constexpr (SWV) {
      st.sw = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rs, s_off, 0, 0));
    } else {
      uint32_t s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = __builtin_amdgcn_raw_buffer_load_b16(rs, s_off + 2u * e, 0, 0);
      st.sw.x = (s[0] & 0xFFFFu) | (s[1] << 16);
      st.sw.y = (s[2] & 0xFFFFu) | (s[3] << 16);
    }
  };

  f32x4 acc[RB];
#pragma unroll
  for (int q = 0; q < RB; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
  const i32x4 magic = {kMagicBits, kMagicBits, kMagicBits, kMagicBits};
  auto operand = [](const uint2& p) {
    return i32x4{(int)((p.x << 4) & 0xF0F0F0F0u), (int)((p.y << 4) & 0xF0F0F0F0u), (int)(p.x & 0xF0F0F0F0u),
                 (int)(p.y & 0xF0F0F0F0u)};
  };
  auto compute = [&](const Stage& st) {
    if constexpr (F4) {
      auto scale = [](uint32_t byte) { return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(byte, 1.0f, false)[0]; };
      const _Float16 sw = scale(st.sw.x);
      const f16x8 P0 = fp4_operand(st.w.x, sw), P1 = fp4_operand(st.w.y, sw);
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        const _Float16 sx = scale(st.sx[q]);
        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(P0, fp4_operand(st.a[q].x, sx), acc[q], 0, 0, 0);
        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(P1, fp4_operand(st.a[q].y, sx), acc[q], 0, 0, 0);
      }
      return;
    }
    const i32x4 P = operand(st.w);
    float sw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sw[e] = f16_to_f32((uint16_t)((e & 2 ? st.sw.y : st.sw.x) >> (16 * (e & 1))));
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const i32x4 d = __builtin_amdgcn_mfma_i32_16x16x64_i8(P, operand(st.a[q]), magic, 0, 0, 0);
      const float sxq = f16_to_f32((uint16_t)st.sx[q]) * 0.00390625f;
      const float sng = -kMagic * sxq;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[q][e] = __builtin_fmaf(__builtin_fmaf(__int_as_float(d[e]), sxq, sng), sw[e], acc[q][e]);
    }
  };

  // low-rank branch: chunk q of 32 ranks belongs to wave nwk - 1 - q % nwk (the
  // last ones: the first ones fetch the epilogue's operands)
  const bool l2_vec = rank % 8 == 0 && ((uintptr_t)l2 & 15u) == 0, z_vec = rank % 4 == 0 && ((uintptr_t)a.z & 15u) == 0;
  f32x4 up[F4 ? RB : 1];  // NVFP4: the low-rank product apart
  if constexpr (F4)
#pragma unroll
    for (int q = 0; q < RB; ++q) up[q] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto lowrank = [&]() {
    for (int kc = 32 * (nwk - 1 - wk); kc < rank; kc += 32 * nwk) {
      const int t0 = kc + 8 * c;
      u32x4 w = {0u, 0u, 0u, 0u};
      const int j = j0 + r;
      if (j < n) {
        const uint16_t* p = l2 + (size_t)j * rank + t0;
        if (l2_vec) {
          if (t0 < rank) w = ldg16(p);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (t0 + e < rank) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
        }
      }
      const bf16x8 P = __builtin_bit_cast(bf16x8, w);
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        const int i = i0 + 16 * q + r;
        f32x4 z0 = {0.f, 0.f, 0.f, 0.f}, z1 = {0.f, 0.f, 0.f, 0.f};
        if (i < row_end) {
          const float* zr = a.z + (size_t)i * rank + t0;
          if (z_vec) {
            if (t0 < rank) z0 = *reinterpret_cast<const f32x4*>(zr);
            if (t0 + 4 < rank) z1 = *reinterpret_cast<const f32x4*>(zr + 4);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (t0 + e < rank) z0[e] = zr[e];
              if (t0 + 4 + e < rank) z1[e] = zr[4 + e];
            }
          }
        }
        const bf16x8 Q = __builtin_bit_cast(bf16x8, u32x4{pack_bf16x2(z0[0], z0[1]), pack_bf16x2(z0[2], z0[3]),
                                                          pack_bf16x2(z1[0], z1[1]), pack_bf16x2(z1[2], z1[3])});
        f32x4& sum = F4 ? up[F4 ? q : 0] : acc[q];
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(P, Q, sum, 0, 0, 0);
      }
    }
  };

  // A unit is four consecutive columns of a row (a lane's four results).  Unit
  // u of the workgroup: column block u / (64 RB), row block, lane.
  auto unit_at = [&](int u, int& i, int& j) {
    i = i0 + 16 * ((u >> 6) % RB) + (u & 15);
    j = j00 + 16 * (u / (64 * RB)) + 4 * ((u & 63) >> 4);
    return i < row_end && j < n;
  };

  constexpr int D = rows_depth(RB);
  Stage st[D];
#pragma unroll
  for (int u = 0; u < D; ++u) load(u, st[u]);
  // the operands of this thread's first unit's epilogue, while the codes arrive
  int ui, uj;
  const bool mine = tid < nwc * RB * 64 && unit_at(tid, ui, uj);
  EpiLoads el;
  if (mine) el = load_unit<OUT_BF16>(ui, uj, n, bias, a.ep);
  lowrank();
  int k = 0;
  for (; k + D <= nk; k += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      compute(st[u]);
      load(k + u + D, st[u]);
    }
  }
#pragma unroll
  for (int u = 0; u + 1 < D; ++u)
    if (k + u < nk) compute(st[u]);

#pragma unroll
  for (int q = 0; q < RB; ++q) part[(wave * RB + q) * 64 + lane] = F4 ? acc[q] * a.txw + up[F4 ? q : 0] : acc[q];
  __syncthreads();
  auto sum = [&](int u) {
    const int at = u / (64 * RB) * nwk * RB * 64 + u % (64 * RB);
    f32x4 v = part[at];
    for (int w = 1; w < nwk; ++w) v += part[at + w * RB * 64];
    return v;
  };
  if (mine) finish_unit<OUT_BF16>(sum(tid), el, ui, uj, n, a.ep);
  for (int u = tid + (int)blockDim.x; u < nwc * RB * 64; u += (int)blockDim.x)
    if (unit_at(u, ui, uj)) finish_unit<OUT_BF16>(sum(u), load_unit<OUT_BF16>(ui, uj, n, bias, a.ep), ui, uj, n, a.ep);
}

template <int RB, bool OUT_BF16, bool GROUPED, int FMT>
int launch_rows(const RowsArgs& a, hipStream_t st) {
  const RowsSplit split = rows_split(GROUPED ? grouped_row_blocks(a.b, a.groups.experts, 16 * RB) : 1, a.n, a.G, RB);
  const int nwk = split.nwk, nwc = split.nwc;
  const long long grid = split.grid;
  if (!launch_fits(grid, 64 * nwk * nwc)) return (int)hipErrorInvalidConfiguration;
  const size_t lds = (size_t)nwk * nwc * RB * 1024;
  const bool swv = a.n % 4 == 0 && ((uintptr_t)a.wscale & 7u) == 0;
  auto go = [&](auto kernel) {
    const int ok = scratch_free(reinterpret_cast<const void*>(kernel));
    if (ok != 0) return ok;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3((unsigned)(64 * nwk * nwc)), lds, st, a, nwk, nwc);
    return (int)hipGetLastError();
  };
  if constexpr (FMT == kFmtInt4)
    if (!swv) return go(gemm_w4a4_rows_kernel<RB, OUT_BF16, GROUPED, FMT, false>);
  return go(gemm_w4a4_rows_kernel<RB, OUT_BF16, GROUPED, FMT, true>);
}

template <int RB, int FMT>
int launch_rb(const RowsArgs& a, int y_dtype, hipStream_t st) {
  const bool bf = y_dtype == SVDQ_OUT_BF16;
  if constexpr (RB <= 2 && FMT == kFmtInt4)
    if (a.groups.offsets) return bf ? launch_rows<RB, true, true, FMT>(a, st) : launch_rows<RB, false, true, FMT>(a, st);
  return bf ? launch_rows<RB, true, false, FMT>(a, st) : launch_rows<RB, false, false, FMT>(a, st);
}

template <int FMT>
int launch_fmt(const RowsArgs& a, int rb, int y_dtype, hipStream_t st) {
  if (rb == 1) return launch_rb<1, FMT>(a, y_dtype, st);
  if (rb == 2) return launch_rb<2, FMT>(a, y_dtype, st);
  if (rb == 4) return launch_rb<4, FMT>(a, y_dtype, st);
  return (int)hipErrorInvalidValue;
}

}  // namespace

int launch_gemm_rows(const RowsArgs& a, int rb, int y_dtype, int fmt, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  // without groups one workgroup covers every row; experts' row blocks are 16 or 32 rows of INT4
  if (a.groups.offsets ? rb > 2 || fmt != kFmtInt4 : a.b > 16 * rb) return (int)hipErrorInvalidValue;
  return fmt == kFmtFp4 ? launch_fmt<kFmtFp4>(a, rb, y_dtype, st) : launch_fmt<kFmtInt4>(a, rb, y_dtype, st);
}

}  // namespace svdq
