// INT4 product with an epilogue for few rows (up to 64, or up to 64 rows of one
// expert at a time): the layer's weights are read once and bound it.
//
// Y = epilogue(sum_g sx[g,i] sw[g,j] isum[i,j,g] + (bf16(Z) L2)[i,j] + bias[j]),
// with the exact per-group integer sums and the two FMAs per element and group
// of the tiled kernel (gemm_body.h).
//
// A workgroup computes 16 columns of RB blocks of 16 rows; its waves split the
// channel groups (wave w takes groups w, w + NW, ...), and their sums are added
// in LDS in wave order.  Nothing is staged in LDS before that: a lane's
// MFMA operand (16 codes of one row or column) is 8 bytes of its packed record,
// so weights and activations go from memory to registers to the MFMA, D groups
// ahead.  Any channel order serves, as both operands unpack alike.
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

constexpr int rows_depth(int rb) { return rb == 1 ? 6 : (rb == 2 ? 4 : 3); }

// SWV: the four scales of a lane's columns are one aligned 8-byte load.
template <int RB, bool OUT_BF16, bool GROUPED, bool SWV>
__global__ __launch_bounds__(1024) void gemm_w4a4_rows_kernel(RowsArgs a) {
  extern __shared__ __align__(16) uint8_t rows_lds[];
  f32x4* part = reinterpret_cast<f32x4*>(rows_lds);  // [wave][row block][lane]
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nw = (int)(blockDim.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int b = a.b, n = a.n, G = a.G, rank = a.rank;
  const int tiles_n = (n + 15) / 16;

  const uint8_t* qw = a.qw;
  const uint16_t* wscale = a.wscale;
  const uint16_t* l2 = a.l2;
  const uint16_t* bias = a.bias;
  int i0, j0, row_end;
  if constexpr (GROUPED) {
    const GroupTile g = find_tile<16 * RB>(a.groups.offsets, a.groups.experts, b, tiles_n, (int)blockIdx.x,
                                           [](int d, int T) { return xcd_range(d, T); });
    if (!g.live) return;  // every wave finds the same tile
    // an expert's row blocks of one column block are neighbours: they share its weights in L2
    const int tj = g.u / g.blocks;
    i0 = g.lo + (g.u - tj * g.blocks) * 16 * RB;
    j0 = tj * 16;
    row_end = g.hi;
    const size_t e = (size_t)g.expert;
    qw += e * G * n * 32;
    wscale += e * G * n;
    if (rank > 0) l2 += e * n * rank;
    if (bias) bias += e * n;
  } else {
    i0 = 0;
    j0 = (int)blockIdx.x * 16;
    row_end = b;
  }

  struct Stage {
    uint2 w, a[RB];   // packed codes: this lane's 8 bytes of its column's and rows' records
    uint2 sw;         // fp16 scales of columns 4c .. 4c+3
    uint32_t sx[RB];  // fp16 scales of the rows
  };
  const int nk = wave < G ? (G - wave + nw - 1) / nw : 0;  // groups of this wave
  const uint32_t w_off = (uint32_t)(j0 + r) * 32u + 8u * c;
  const uint32_t s_off = (uint32_t)(j0 + 4 * c) * 2u;
  auto load = [&](int k, Stage& st) {
    const bool live = k < nk;
    const int g = live ? wave + nw * k : 0;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(qw + (size_t)g * n * 32, live ? (uint32_t)n * 32u : 0u);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.qx + (size_t)g * b * 32, live ? (uint32_t)b * 32u : 0u);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(wscale + (size_t)g * n, live ? (uint32_t)n * 2u : 0u);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.ascale + (size_t)g * b, live ? (uint32_t)b * 2u : 0u);
    st.w = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rw, w_off, 0, 0));
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const uint32_t row = (uint32_t)(i0 + 16 * q + r);
      st.a[q] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rx, row * 32u + 8u * c, 0, 0));
      st.sx[q] = __builtin_amdgcn_raw_buffer_load_b16(ra, row * 2u, 0, 0);
    }
    if constexpr (SWV) {
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

  // low-rank branch: chunk q of 32 ranks belongs to wave q % NW
  auto lowrank = [&]() {
    for (int kc = 32 * wave; kc < rank; kc += 32 * nw) {
      const int t0 = kc + 8 * c;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      const int j = j0 + r;
      if (j < n) {
        const uint16_t* p = l2 + (size_t)j * rank + t0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (t0 + e < rank) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
      }
      const bf16x8 P = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        const int i = i0 + 16 * q + r;
        float zv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (i < row_end) {
          const float* zr = a.z + (size_t)i * rank + t0;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (t0 + e < rank) zv[e] = zr[e];
        }
        const bf16x8 Q = __builtin_bit_cast(bf16x8, u32x4{pack_bf16x2(zv[0], zv[1]), pack_bf16x2(zv[2], zv[3]),
                                                          pack_bf16x2(zv[4], zv[5]), pack_bf16x2(zv[6], zv[7])});
        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(P, Q, acc[q], 0, 0, 0);
      }
    }
  };

  constexpr int D = rows_depth(RB);
  Stage st[D];
#pragma unroll
  for (int u = 0; u < D; ++u) load(u, st[u]);
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

  // sums of the waves, in wave order, then the epilogue of four columns a thread
#pragma unroll
  for (int q = 0; q < RB; ++q) part[(wave * RB + q) * 64 + lane] = acc[q];
  __syncthreads();
  for (int u = tid; u < RB * 64; u += (int)blockDim.x) {
    f32x4 v = part[u];
    for (int w = 1; w < nw; ++w) v += part[w * RB * 64 + u];
    const int i = i0 + 16 * (u >> 6) + (u & 15), j = j0 + 4 * ((u & 63) >> 4);
    if (i < row_end && j < n) finish_unit<OUT_BF16>(v, i, j, n, bias, a.ep);
  }
}

template <int RB, bool OUT_BF16, bool GROUPED>
int launch_rows(const RowsArgs& a, hipStream_t st) {
  const long long tiles_n = (a.n + 15) / 16;
  const long long grid = GROUPED ? grouped_row_blocks(a.b, a.groups.experts, 16 * RB) * tiles_n : tiles_n;
  if (grid > 0x7FFFFFFF) return (int)hipErrorInvalidValue;
  const int most = RB == 4 ? 8 : 16;
  const int nw = a.G >= 32 ? most : (a.G >= 16 ? 8 : (a.G >= 8 ? 4 : 2));
  const size_t lds = (size_t)nw * RB * 1024;
  const bool swv = a.n % 4 == 0 && ((uintptr_t)a.wscale & 7u) == 0;
  auto go = [&](auto kernel) {
    const int ok = scratch_free(reinterpret_cast<const void*>(kernel));
    if (ok != 0) return ok;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3((unsigned)(64 * nw)), lds, st, a);
    return (int)hipGetLastError();
  };
  return swv ? go(gemm_w4a4_rows_kernel<RB, OUT_BF16, GROUPED, true>)
             : go(gemm_w4a4_rows_kernel<RB, OUT_BF16, GROUPED, false>);
}

template <int RB>
int launch_rb(const RowsArgs& a, int y_dtype, hipStream_t st) {
  const bool bf = y_dtype == SVDQ_OUT_BF16;
  if (a.groups.offsets) return bf ? launch_rows<RB, true, true>(a, st) : launch_rows<RB, false, true>(a, st);
  return bf ? launch_rows<RB, true, false>(a, st) : launch_rows<RB, false, false>(a, st);
}

}  // namespace

int launch_gemm_rows(const RowsArgs& a, int rb, int y_dtype, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  // without groups one workgroup covers every row
  if (!a.groups.offsets && a.b > 16 * rb) return (int)hipErrorInvalidValue;
  if (rb == 1) return launch_rb<1>(a, y_dtype, st);
  if (rb == 2) return launch_rb<2>(a, y_dtype, st);
  if (rb == 4) return launch_rb<4>(a, y_dtype, st);
  return (int)hipErrorInvalidValue;
}

}  // namespace svdq
