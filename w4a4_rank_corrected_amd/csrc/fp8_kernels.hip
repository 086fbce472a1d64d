// The 8-bit floating-point setting: quantization of activations and weights, and
// the product for few rows.
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

// ---------------------------------------------------------------------------
// Activations.  Sixteen lanes hold a block (8 channels a lane): a packed 16-bit
// maximum of the magnitudes' bits (bf16 magnitudes order as integers), four lane
// rotations, the scale's byte from the maximum's exponent and mantissa, and the
// conversion instruction, which divides by the scale and rounds.  A workgroup
// takes 16 rows and up to kFp8ActBlocks blocks of each, loading all of them first.
// Memory bounds it: 8192 x 8192 30.4 us, 6.6 TB/s; 4608 x 4608 13.4 us among other work.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void fp8_act_kernel(const uint16_t* __restrict__ x, int b, int m, int G,
                                                      uint8_t* __restrict__ qx, uint8_t* __restrict__ ascale) {
  const int tid = (int)threadIdx.x, c = tid & 15;
  const int chunks = (G + kFp8ActBlocks - 1) / kFp8ActBlocks;
  const int rb = (int)blockIdx.x / chunks;
  const int g0 = ((int)blockIdx.x - rb * chunks) * kFp8ActBlocks;
  const int row = rb * 16 + (tid >> 4);
  if (row >= b) return;  // (no lane waits for another row's)
  const uint16_t* xr = x + (size_t)row * m;
  u32x4 v[kFp8ActBlocks];
#pragma unroll
  for (int u = 0; u < kFp8ActBlocks; ++u) v[u] = load_bf16x8(xr, (g0 + u) * 128 + 8 * c, m);
#pragma unroll
  for (int u = 0; u < kFp8ActBlocks; ++u) {
    const int g = g0 + u;
    if (g >= G) break;
    const int byte = block_scale_bf16(block_max16(v[u]));
    const uint2 q = encode8(v[u], byte);
    *reinterpret_cast<uint2*>(qx + ((size_t)g * b + row) * 128 + 8 * c) = q;
    if (c == 0) ascale[(size_t)g * b + row] = (uint8_t)stored_scale(byte);
  }
}

// ---------------------------------------------------------------------------
// Weights: a workgroup takes a block of 128 x 128, 64 values a thread in
// registers, finds its largest magnitude, and passes the codes through LDS into
// whole records (W [m][n] is read along the output channels, W^T along the input
// channels).  Done once a layer: 1152 x 6912 in bf16 11 us.
// ---------------------------------------------------------------------------
template <bool BF16, bool TRANS>
__global__ __launch_bounds__(256) void fp8_weight_kernel(const void* __restrict__ w_all, int m, int n, int G, int NB,
                                                         uint8_t* __restrict__ qw, uint8_t* __restrict__ wscale) {
  constexpr int kPitch = 144;  // bytes of a record in LDS: 16-byte reads of neighbouring records on other banks
  __shared__ __align__(16) uint8_t s_code[128 * kPitch];
  __shared__ uint32_t s_max[4];
  const int tid = (int)threadIdx.x, lane = tid & 63;
  long long blk = blockIdx.x;
  const int jb = (int)(blk % NB);
  blk /= NB;
  const int g = (int)(blk % G);
  const size_t e = (size_t)(blk / G);
  const int k0 = g * 128, j0 = jb * 128;
  const uint8_t* w = reinterpret_cast<const uint8_t*>(w_all) + e * (size_t)m * (size_t)n * (BF16 ? 2 : 4);
  // rows of W (or W^T) of the block; thread: columns 4 (tid & 31) .. + 3 of rows tid / 32 + 8 i
  const int rows = TRANS ? n : m, cols = TRANS ? m : n, r0 = TRANS ? j0 : k0, c0 = TRANS ? k0 : j0;
  const int c = 4 * (tid & 31), r = tid >> 5;
  f32x4 v[16];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int rr = r0 + r + 8 * i;
    if (rr < rows) v[i] = load4<BF16>(w + (size_t)rr * cols * (BF16 ? 2 : 4), c0 + c, cols);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) top = max(top, __float_as_uint(v[i][q]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if (lane == 0) s_max[tid >> 6] = top;
  __syncthreads();
  top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  const int byte = block_scale_f32(top);
  const float inv = __uint_as_float((uint32_t)(254 - stored_scale(byte)) << 23);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t q = byte < 0 ? 0x7F7F7F7Fu : encode4(v[i] * inv);
    if constexpr (TRANS) {
      *reinterpret_cast<uint32_t*>(s_code + (r + 8 * i) * kPitch + c) = q;
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) s_code[(c + t) * kPitch + r + 8 * i] = (uint8_t)(q >> (8 * t));
    }
  }
  __syncthreads();
  uint8_t* out = qw + (e * G + g) * (size_t)n * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = tid + 256 * i, j = u >> 3, p = (u & 7) * 16;  // record and 16 bytes of it
    if (j0 + j >= n) continue;
    u32x4 q = *reinterpret_cast<const u32x4*>(s_code + j * kPitch + p);
    // channels behind the last one have code zero in a block of NaN too
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int left = m - (k0 + p + 4 * t);
      if (left < 4) q[t] &= left <= 0 ? 0u : (1u << (8 * left)) - 1u;
    }
    *reinterpret_cast<u32x4*>(out + (size_t)(j0 + j) * 128 + p) = q;
  }
  if (tid == 0) wscale[(e * G + g) * NB + jb] = (uint8_t)stored_scale(byte);
}

// ---------------------------------------------------------------------------
// The product for few rows (or rows of one expert at a time).
//
// A wave computes 16 columns of RB blocks of 16 rows: weights as the first operand,
// so that a lane's four results are neighbouring columns of one row.  Lane l holds
// 32 bytes of the records of column l & 15 and of row l & 15, straight from memory,
// and decodes them, scaled, to bf16: the bf16 matrix instruction adds exact products
// in full fp32 (the 8-bit one does not, see the tiled kernel), and memory bounds the
// kernel either way (8 experts, 4096 -> 1152, a row each 9.3 us, by tiles 18.9; 16 rows,
// 8192 -> 8192 19.3, 3.5 TB/s of weights).  Of a workgroup's waves, nwk split the channel
// blocks of the same columns (wave k takes blocks k, k + nwk, ...; sums added in LDS in
// wave order), nwc take neighbouring columns.
//
// X (one layer, RB 1): a.qx is x itself in bf16, m channels a row, and every workgroup
// quantizes the few blocks there are into LDS while its first weights are on their way:
// one launch instead of two for a row or a few (1 x 1152 -> 6912: 6.4 us, and 2.2 for
// the quantization before it).
// ---------------------------------------------------------------------------
constexpr int fp8_rows_depth(int rb) { return rb == 1 ? 4 : (rb == 2 ? 3 : 2); }

template <int RB, bool OUT_BF16, bool GROUPED, bool X>
__global__ __launch_bounds__(RB == 4 ? 512 : 1024) void fp8_rows_kernel(Fp8Args a, int nwk, int nwc, int m) {
  static_assert(!X || (RB == 1 && !GROUPED), "");
  extern __shared__ __align__(16) uint8_t fp8_rows_lds[];
  f32x4* part = reinterpret_cast<f32x4*>(fp8_rows_lds);  // [wave][row block][lane]
  uint8_t* s_code = fp8_rows_lds + nwk * nwc * RB * 1024;  // X: records [G][b][128], then scales [G][b]
  uint8_t* s_scale = s_code + a.G * a.b * 128;
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ct = wave / nwk, wk = wave - ct * nwk;
  const int r = lane & 15, c = lane >> 4;
  const int n = a.n, G = a.G, NB = (n + 127) / 128, xr = a.x_rows;
  const int tiles_n = (n + 16 * nwc - 1) / (16 * nwc);
  const uint8_t* qw = a.qw;
  const uint8_t* wscale = a.wscale;
  const uint16_t* bias = a.bias;
  int i0, j00, row_end;
  if constexpr (GROUPED) {
    const GroupTile g = find_tile<16 * RB>(a.groups.offsets, a.groups.experts, a.b, tiles_n, (int)blockIdx.x,
                                           [](int d, int T) { return xcd_range(d, T); });
    if (!g.live) return;  // every wave finds the same tile
    const int tj = g.u / g.blocks;
    i0 = g.lo + (g.u - tj * g.blocks) * 16 * RB;
    j00 = tj * 16 * nwc;
    row_end = g.hi;
    const size_t e = (size_t)g.expert;
    qw += e * G * (size_t)n * 128;
    wscale += e * G * NB;
    if (bias) bias += e * n;
  } else {
    const int blocks = (a.b + 16 * RB - 1) / (16 * RB);
    const int u = xcd_range((int)blockIdx.x, blocks * tiles_n), tj = u / blocks;
    i0 = (u - tj * blocks) * 16 * RB;
    j00 = tj * 16 * nwc;
    row_end = a.b;
  }
  const int j0 = j00 + 16 * ct;

  uint32_t src[RB];  // the rows' place in qx, past its end for none
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    const int i = i0 + 16 * q + r;
    int s = i < row_end ? i : -1;
    if (GROUPED && s >= 0 && a.row_index) s = a.row_index[s];
    src[q] = (unsigned)s < (unsigned)xr ? (uint32_t)s : 0x00FFFFFFu;
  }
  struct Stage {
    u32x4 w[2], x[RB][2];
    uint32_t sw, sx[RB];
  };
  const int nk = wk < G ? (G - wk + nwk - 1) / nwk : 0;
  const uint32_t w_off = (uint32_t)(j0 + r) * 128u + 32u * c;
  auto load = [&](int k, Stage& st) {
    const bool live = k < nk;
    const int g = live ? wk + nwk * k : 0;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(qw + (size_t)g * n * 128, live ? (uint32_t)n * 128u : 0u);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.qx + (size_t)g * xr * 128, live ? (uint32_t)xr * 128u : 0u);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(wscale + (size_t)g * NB, live ? (uint32_t)NB : 0u);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.ascale + (size_t)g * xr, live ? (uint32_t)xr : 0u);
    st.w[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, w_off, 0, 0));
    st.w[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, w_off + 16u, 0, 0));
    st.sw = __builtin_amdgcn_raw_buffer_load_b8(rs, (uint32_t)j0 / 128u, 0, 0);
    if constexpr (X) return;
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const uint32_t off = src[q] * 128u + 32u * c;
      st.x[q][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, off, 0, 0));
      st.x[q][1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, off + 16u, 0, 0));
      st.sx[q] = __builtin_amdgcn_raw_buffer_load_b8(ra, src[q], 0, 0);
    }
  };
  f32x4 acc[RB];
#pragma unroll
  for (int q = 0; q < RB; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](int k, Stage& st) {
    if constexpr (X) {
      const int at = (wk + nwk * k) * a.b + r;
      st.x[0][0] = st.x[0][1] = u32x4{0u, 0u, 0u, 0u};
      st.sx[0] = 0;
      if (r < a.b) {
        st.x[0][0] = *reinterpret_cast<const u32x4*>(s_code + at * 128 + 32 * c);
        st.x[0][1] = *reinterpret_cast<const u32x4*>(s_code + at * 128 + 32 * c + 16);
        st.sx[0] = s_scale[at];
      }
    }
#pragma unroll
    for (int q = 0; q < RB; ++q)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const u32x4 &w = st.w[h >> 1], &x = st.x[q][h >> 1];
        const int o = 2 * (h & 1);
        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(w[o], w[o + 1], scale_of(st.sw)),
                                                         decode8(x[o], x[o + 1], scale_of(st.sx[q])), acc[q], 0, 0, 0);
      }
  };

  auto unit_at = [&](int u, int& i, int& j) {
    i = i0 + 16 * ((u >> 6) % RB) + (u & 15);
    j = j00 + 16 * (u / (64 * RB)) + 4 * ((u & 63) >> 4);
    return i < row_end && j < n;
  };
  constexpr int D = fp8_rows_depth(RB);
  Stage st[D];
#pragma unroll
  for (int u = 0; u < D; ++u) load(u, st[u]);
  int ui, uj;
  const bool mine = tid < nwc * RB * 64 && unit_at(tid, ui, uj);
  EpiLoads el;
  if (mine) el = load_unit<OUT_BF16>(ui, uj, n, bias, a.ep);
  if constexpr (X) {
    // sixteen lanes a block, as fp8_act_kernel
    const uint16_t* x = reinterpret_cast<const uint16_t*>(a.qx);
    for (int blk = tid >> 4; blk < a.b * G; blk += (int)blockDim.x >> 4) {
      const int g = blk / a.b, row = blk - g * a.b;
      const u32x4 v = load_bf16x8(x + (size_t)row * m, g * 128 + 8 * (tid & 15), m);
      const int byte = block_scale_bf16(block_max16(v));
      *reinterpret_cast<uint2*>(s_code + blk * 128 + 8 * (tid & 15)) = encode8(v, byte);
      if ((tid & 15) == 0) s_scale[blk] = (uint8_t)stored_scale(byte);
    }
    __syncthreads();
  }
  int k = 0;
  for (; k + D <= nk; k += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      compute(k + u, st[u]);
      load(k + u + D, st[u]);
    }
  }
#pragma unroll
  for (int u = 0; u + 1 < D; ++u)
    if (k + u < nk) compute(k + u, st[u]);

#pragma unroll
  for (int q = 0; q < RB; ++q) part[(wave * RB + q) * 64 + lane] = acc[q];
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

template <int RB, bool OUT_BF16, bool GROUPED, bool X = false>
int launch_fp8_rows_typed(const Fp8Args& a, const RowsSplit& s, hipStream_t st, int m = 0) {
  auto kernel = fp8_rows_kernel<RB, OUT_BF16, GROUPED, X>;
  const int threads = 64 * s.nwk * s.nwc;
  if (!launch_fits(s.grid, threads)) return (int)hipErrorInvalidConfiguration;
  const int ok = scratch_free(reinterpret_cast<const void*>(kernel));
  if (ok != 0) return ok;
  const size_t lds = (size_t)s.nwk * s.nwc * RB * 1024 + (X ? (size_t)a.G * a.b * 129 : 0);
  hipLaunchKernelGGL(kernel, dim3((unsigned)s.grid), dim3((unsigned)threads), lds, st, a, s.nwk, s.nwc, m);
  return (int)hipGetLastError();
}

template <int RB>
int launch_fp8_rows_rb(const Fp8Args& a, const RowsSplit& s, bool bf, hipStream_t st) {
  if (a.groups.offsets)
    return bf ? launch_fp8_rows_typed<RB, true, true>(a, s, st) : launch_fp8_rows_typed<RB, false, true>(a, s, st);
  return bf ? launch_fp8_rows_typed<RB, true, false>(a, s, st) : launch_fp8_rows_typed<RB, false, false>(a, s, st);
}

}  // namespace

int launch_fp8_act(const uint16_t* x, int b, int m, uint8_t* qx, uint8_t* ascale, void* stream) {
  const int G = fp8_blocks(m);
  return launch_checked(fp8_act_kernel, fp8_act_grid(b, m), 256, (hipStream_t)stream, x, b, m, G, qx, ascale);
}

int launch_fp8_weights(const void* w, int dtype, int experts, int m, int n, bool transposed, uint8_t* qw,
                       uint8_t* wscale, void* stream) {
  const int G = fp8_blocks(m), NB = fp8_blocks(n);
  const long long grid = (long long)experts * G * NB;
  auto go = [&](auto kernel) {
    return launch_checked(kernel, grid, 256, (hipStream_t)stream, w, m, n, G, NB, qw, wscale);
  };
  if (dtype == SVDQ_OUT_BF16)
    return transposed ? go(fp8_weight_kernel<true, true>) : go(fp8_weight_kernel<true, false>);
  return transposed ? go(fp8_weight_kernel<false, true>) : go(fp8_weight_kernel<false, false>);
}

int launch_fp8_rows(const Fp8Args& a, const Fp8Plan& plan, int y_dtype, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const bool bf = y_dtype == SVDQ_OUT_BF16;
  if (plan.rb == 1) return launch_fp8_rows_rb<1>(a, plan.split, bf, st);
  if (plan.rb == 2) return launch_fp8_rows_rb<2>(a, plan.split, bf, st);
  if (plan.rb == 4) return launch_fp8_rows_rb<4>(a, plan.split, bf, st);
  return (int)hipErrorInvalidValue;
}

int launch_fp8_rows_x(const Fp8Args& a, const uint16_t* x, int m, const Fp8Plan& plan, int y_dtype, void* stream) {
  if (plan.rb != 1 || a.b > 16 || a.groups.offsets || a.G * a.b > kFp8FusedBlocks) return (int)hipErrorInvalidValue;
  Fp8Args f = a;
  f.qx = reinterpret_cast<const uint8_t*>(x);
  return y_dtype == SVDQ_OUT_BF16 ? launch_fp8_rows_typed<1, true, false, true>(f, plan.split, (hipStream_t)stream, m)
                                  : launch_fp8_rows_typed<1, false, false, true>(f, plan.split, (hipStream_t)stream, m);
}

int launch_fp8_gemm(const Fp8Args& a, const Fp8Plan& plan, int y_dtype, void* ws, void* stream) {
  return plan.rb ? launch_fp8_rows(a, plan, y_dtype, stream) : launch_fp8_tiles(a, plan, y_dtype, ws, stream);
}

}  // namespace svdq
