// Grouped by expert: the activation quantization + low-rank down-projection of
// rows sorted by expert, and the combination of a token's rows afterwards.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "epilogue.h"
#include "grouped.h"
#include "internal.h"
#include "launch.h"
#include "quant.h"

#pragma clang fp contract(off)

namespace svdq {
namespace {

using namespace dev;

// ---------------------------------------------------------------------------
// Row i of expert e: x~ = bf16(fl32(x[row_index[i]] * smooth_inv[e])), its INT4
// codes and scales, z = x~ L1[e] (fp32).  A workgroup of NW waves owns 16 rows of
// one expert (grouped.h) and its waves split the channel groups, so each row's
// Z is complete in the workgroup: the waves' partial sums are added in LDS in
// wave order.  Z is summed over groups in a fixed order.
//
// Four neighbouring lanes hold a row's group (lane 4 r + c: channels 8c .. 8c+7
// and 32+8c .. 32+8c+7), so each 16-byte load of a quad is 64 contiguous bytes;
// an MFMA operand wants lane r + 16 c instead, and x~ and L1 get there by lane
// permutes (ds_bpermute).  Loading in the MFMA's lane order, every quad on four
// rows, kept the address path busy instead: 26.4 against 18.5 us for 18006 rows
// of 2048 channels at rank 16, 43.6 against 26.8 us for 8192 of 4608 at rank 32.
// What bounds it now is the gather: 94 MB of rows and codes in those 18.5 us,
// 5.1 TB/s (a large copy reaches 5.1).  These are of the kernel alone, over and
// over; between the products of a layer's calls, which leave little of x in the
// caches, the first shape takes 21.8 us (4.3 TB/s).
// A row index outside [0, x_rows) reads as a row of zeros.
// Q = kActQuantNone: Z alone, of ranks rank0 .. rank0 + 16 TB - 1 (further ranks
// of layers with more than 64).
// ---------------------------------------------------------------------------
// Waves a SIMD the register budget must allow, by the number of Z blocks.
constexpr int group_waves_per_simd(int tb) { return tb <= 1 ? 6 : (tb <= 3 ? 4 : 3); }
template <int TB, bool SMOOTH, int Q, int NW>
__global__ __launch_bounds__(64 * NW)
__attribute__((amdgpu_waves_per_eu(group_waves_per_simd(TB)))) void grouped_act_kernel(
    const uint16_t* __restrict__ x, int x_rows, const int32_t* __restrict__ row_index, Groups groups, int b, int m,
    int G, const float* __restrict__ inv_all, const uint16_t* __restrict__ l1_all, int rank, int rank0,
    uint8_t* __restrict__ qx, uint16_t* __restrict__ ascale, float* __restrict__ zout) {
  constexpr int NB = TB > 0 ? TB : 1;
  constexpr int D = 2;
  __shared__ __align__(16) float s_inv[NW][64];
  __shared__ __align__(16) float s_z[TB > 0 ? NW * 16 * 16 * TB : 1];
  const int tid = (int)threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane >> 2, c = lane & 3;     // this lane's row and channels
  const int mr = lane & 15, mc = lane >> 4;  // its place in an MFMA operand
  const int pull = 4 * (4 * mr + mc);        // the lane (times 4) that holds its operand
  const GroupTile gt = find_tile<16>(groups.offsets, groups.experts, b, 1, (int)blockIdx.x,
                                     [](int d, int T) { return xcd_range(d, T); });
  if (!gt.live) return;  // the whole workgroup
  const int row0 = gt.lo + gt.u * 16;
  const int row = row0 + r;
  const bool mine = row < gt.hi;
  const float* inv = SMOOTH ? inv_all + (size_t)gt.expert * m : nullptr;
  const uint16_t* l1t = TB > 0 ? l1_all + ((size_t)gt.expert * rank + rank0) * m : nullptr;
  const int ranks = min(rank - rank0, 16 * TB);  // of this launch
  const int src = mine ? (row_index ? row_index[row] : row) : -1;
  const uint32_t l1_bytes = TB > 0 ? (uint32_t)((ranks - 1) * m + 64) * 2u : 0u;
  const int nj = wave < G ? (G - wave + NW - 1) / NW : 0;  // groups of this wave

  struct Stage {
    u32x4 xa, xb;
    u32x4 la[NB], lb[NB];  // L1 rows tb*16 + r, channels 8c.. and 32 + 8c..
    uint32_t iv;           // 1/lambda of channel `lane` of the group
  };
  // the expert's operands and the row's activations are loaded apart: the first
  // groups' L1 and 1/lambda go out before the row index arrives
  auto load_layer = [&](int j, Stage& st) {
    const bool live = j < nj;
    const int g = live ? wave + NW * j : 0;
    if constexpr (TB > 0) {
      const __amdgpu_buffer_rsrc_t rl = make_rsrc(l1t + (size_t)g * 64, live ? l1_bytes : 0u);
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        const int t = tb * 16 + r;
        const uint32_t off = t < ranks ? (uint32_t)(t * m + 8 * c) * 2u : 0x7FFFFFF0u;
        st.la[tb] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rl, off, 0, 0));
        st.lb[tb] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rl, off + 64u, 0, 0));
      }
    }
    if constexpr (SMOOTH) {
      const __amdgpu_buffer_rsrc_t ri = make_rsrc(inv + (size_t)g * 64, live ? 256u : 0u);
      st.iv = __builtin_amdgcn_raw_buffer_load_b32(ri, (uint32_t)lane * 4u, 0, 0);
    }
  };
  f32x4 acc[NB];
#pragma unroll
  for (int t = 0; t < NB; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // rows of another expert (or past the last) drop their stores: offsets past
  // the end of the group's records
  const uint32_t q_off = mine ? (uint32_t)row * 32u + 4u * c : 0x7FFFFFE0u;
  const uint32_t s_off = mine && c == 0 ? (uint32_t)row * 2u : 0x7FFFFFE0u;

  auto process = [&](int j, const Stage& st) {
    const int g = wave + NW * j;
    float v[16];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf16_lo(st.xa[e]);
      v[2 * e + 1] = bf16_hi(st.xa[e]);
      v[8 + 2 * e] = bf16_lo(st.xb[e]);
      v[8 + 2 * e + 1] = bf16_hi(st.xb[e]);
    }
    if constexpr (SMOOTH) {
      // the wave's own slot: LDS accesses of one wave complete in order, so
      // the previous group's reads finish before this write lands
      s_inv[wave][lane] = __uint_as_float(st.iv);
      const float* iv = s_inv[wave];
      const f32x4 i0 = *reinterpret_cast<const f32x4*>(iv + 8 * c);
      const f32x4 i1 = *reinterpret_cast<const f32x4*>(iv + 8 * c + 4);
      const f32x4 i2 = *reinterpret_cast<const f32x4*>(iv + 32 + 8 * c);
      const f32x4 i3 = *reinterpret_cast<const f32x4*>(iv + 36 + 8 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] *= i0[e];
        v[4 + e] *= i1[e];
        v[8 + e] *= i2[e];
        v[12 + e] *= i3[e];
      }
    }
    uint32_t xt[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      xt[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
      v[2 * q] = bf16_lo(xt[q]);
      v[2 * q + 1] = bf16_hi(xt[q]);
    }
    if constexpr (Q == kActQuantInt4) quant_store_int4(v, g, b, q_off, s_off, qx, ascale);
    if constexpr (TB > 0) {
      auto operand = [&](const u32x4& w) {
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = (uint32_t)__builtin_amdgcn_ds_bpermute(pull, (int)w[q]);
        return __builtin_bit_cast(bf16x8, o);
      };
      const bf16x8 a0 = operand(u32x4{xt[0], xt[1], xt[2], xt[3]});
      const bf16x8 a1 = operand(u32x4{xt[4], xt[5], xt[6], xt[7]});
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        acc[tb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, operand(st.la[tb]), acc[tb], 0, 0, 0);
        acc[tb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, operand(st.lb[tb]), acc[tb], 0, 0, 0);
      }
    }
  };

  Stage st[D];
#pragma unroll
  for (int u = 0; u < D; ++u) load_layer(u, st[u]);
  const bool read = src >= 0 && src < x_rows;
  const uint16_t* xr = x + (size_t)(read ? src : 0) * m + 8 * c;
  auto load_x = [&](int j, Stage& st) {
    st.xa = st.xb = u32x4{0u, 0u, 0u, 0u};
    if (read && j < nj) {
      const uint16_t* xg = xr + (size_t)(wave + NW * j) * 64;
      st.xa = ldg16(xg);
      st.xb = ldg16(xg + 32);
    }
  };

#pragma unroll
  for (int u = 0; u < D; ++u) load_x(u, st[u]);
  int j = 0;
  for (; j + D <= nj; j += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      process(j + u, st[u]);
      load_layer(j + u + D, st[u]);
      load_x(j + u + D, st[u]);
    }
  }
#pragma unroll
  for (int u = 0; u + 1 < D; ++u)
    if (j + u < nj) process(j + u, st[u]);

  if constexpr (TB > 0) {
    // partial Z of each wave (MFMA D layout: row 4 mc + v, column 16 tb + mr),
    // then Z[row0 + i][rank0 + t] = sum over waves in order
    constexpr int ZC = 16 * TB;
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int vv = 0; vv < 4; ++vv) s_z[(wave * 16 + 4 * mc + vv) * ZC + tb * 16 + mr] = acc[tb][vv];
    __syncthreads();
    for (int e = tid; e < 16 * ZC; e += 64 * NW) {
      const int i = e / ZC, t = e - i * ZC;
      float zsum = s_z[i * ZC + t];
#pragma unroll
      for (int w = 1; w < NW; ++w) zsum += s_z[(w * 16 + i) * ZC + t];
      if (row0 + i < gt.hi && t < ranks) zout[(size_t)(row0 + i) * rank + rank0 + t] = zsum;
    }
  }
}

// ---------------------------------------------------------------------------
// y[t] = residual[t] + sum_k weight[t][k] rows[index[t][k]], in fp32 in the
// order of k, rounded once.  A thread takes W consecutive columns (16 bytes) of
// a token and issues the loads of up to kCombineBatch rows together, keeping
// them as they lie in memory until they are added (62 registers, so every wave
// slot of a CU is used).  Rows that do not start 16-byte aligned go the same way
// with element-aligned vectors (gfx950 loads and stores them at any address);
// only the last columns of a row are taken one by one.  An index outside [0, R)
// adds nothing.
// Bound by memory: 4096 tokens x 6 rows of 2048 bf16 28.1 us, 4.8 TB/s (36 us
// with the rows widened to fp32 on arrival: 100 registers).
// ---------------------------------------------------------------------------
constexpr int kCombineBatch = 8;
template <bool BF16, bool ALIGNED>
__global__ __launch_bounds__(256) void combine_kernel(const void* __restrict__ rows, int R, int n,
                                                      const int32_t* __restrict__ index,
                                                      const float* __restrict__ weight, int t_count, int k,
                                                      const void* residual, void* y, int units) {
  constexpr int W = BF16 ? 8 : 4;  // columns per thread
  typedef typename std::conditional<BF16, uint16_t, uint32_t>::type Element;
  typedef u32x4 Loose __attribute__((aligned(2)));
  typedef typename std::conditional<ALIGNED, u32x4, Loose>::type Vector;
  const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long t = u / units;
  if (t >= t_count) return;
  const int j = (int)(u - t * units) * W;
  const int cols = min(n - j, W);
  auto get = [&](const void* base, long long row) -> u32x4 {
    const Element* p = reinterpret_cast<const Element*>(base) + (size_t)row * n + j;
    if (ALIGNED || cols == W) return *reinterpret_cast<const Vector*>(p);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e < cols) {
        if constexpr (BF16)
          v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
        else
          v[e] = p[e];
      }
    return v;
  };
  auto value = [](const u32x4& w, int e) -> float {
    if constexpr (BF16) return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    return __uint_as_float(w[e]);
  };
  float sum[W];
#pragma unroll
  for (int e = 0; e < W; ++e) sum[e] = 0.0f;
  u32x4 res = {0u, 0u, 0u, 0u};
  if (residual) res = get(residual, t);
  for (int q0 = 0; q0 < k; q0 += kCombineBatch) {
    u32x4 v[kCombineBatch];
    float w[kCombineBatch];
#pragma unroll
    for (int q = 0; q < kCombineBatch; ++q) {
      w[q] = 0.0f;
      v[q] = u32x4{0u, 0u, 0u, 0u};
      if (q0 + q < k) {
        const int i = index[t * k + q0 + q];
        if (i >= 0 && i < R) {
          w[q] = weight ? weight[t * k + q0 + q] : 1.0f;
          v[q] = get(rows, i);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kCombineBatch; ++q)
#pragma unroll
      for (int e = 0; e < W; ++e) sum[e] = __builtin_fmaf(w[q], value(v[q], e), sum[e]);
  }
  if (residual)
#pragma unroll
    for (int e = 0; e < W; ++e) sum[e] = value(res, e) + sum[e];
  Element* p = reinterpret_cast<Element*>(y) + (size_t)t * n + j;
  u32x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16)
      o[e] = pack_bf16x2(sum[2 * e], sum[2 * e + 1]);
    else
      o[e] = __float_as_uint(sum[e]);
  }
  if (ALIGNED || cols == W) {
    *reinterpret_cast<Vector*>(p) = o;
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e < cols) p[e] = BF16 ? (Element)(o[e >> (BF16 ? 1 : 0)] >> (BF16 ? 16 * (e & 1) : 0)) : (Element)o[e & 3];
  }
}

}  // namespace

int launch_grouped_act(const uint16_t* x, int x_rows, const int32_t* row_index, const int32_t* offsets,
                       const svdq_grouped_layer& L, int b, uint8_t* qx, uint16_t* ascale, float* z, void* stream) {
  const Groups groups{offsets, L.experts};
  const int G = L.m / SVDQ_GROUP;
  const int grid = (int)grouped_row_blocks(b, L.experts, 16);
  // Waves of a row block: four leave room for more row blocks on a CU (30.3 us
  // against 40.3 for 18006 rows of 2048 channels at rank 64, within 4 % of each
  // other at ranks 16 and 32); with fewer row blocks than CUs, eight keep more
  // loads in flight for the same rows.  (Sixteen: 25-40 % slower with many rows,
  // no faster with few.)
  const int nw = grid <= kMaxCUs ? 8 : 4;
  auto go = [&](auto kernel, int rank0) {
    return launch_checked(kernel, grid, 64 * nw, (hipStream_t)stream, x, x_rows, row_index, groups, b, L.m, G,
                          L.smooth_inv, L.l1, L.rank, rank0, qx, ascale, z);
  };
  auto pass = [&](auto TB, auto Q, int rank0) {
    constexpr int tb = decltype(TB)::value, q = decltype(Q)::value;
    auto with_waves = [&](auto NW) {
      constexpr int w = decltype(NW)::value;
      return L.smooth_inv ? go(grouped_act_kernel<tb, true, q, w>, rank0) : go(grouped_act_kernel<tb, false, q, w>, rank0);
    };
    return nw == 8 ? with_waves(std::integral_constant<int, 8>{}) : with_waves(std::integral_constant<int, 4>{});
  };
  // codes and scales with the first 64 ranks, then 64 further ranks a launch
  for (int rank0 = 0; rank0 == 0 || rank0 < L.rank; rank0 += 64) {
    const int tb = (std::min(L.rank - rank0, 64) + 15) / 16;
    auto sized = [&](auto Q) {
      switch (tb) {
        case 1: return pass(std::integral_constant<int, 1>{}, Q, rank0);
        case 2: return pass(std::integral_constant<int, 2>{}, Q, rank0);
        case 3: return pass(std::integral_constant<int, 3>{}, Q, rank0);
        default: return pass(std::integral_constant<int, 4>{}, Q, rank0);
      }
    };
    const std::integral_constant<int, kActQuantInt4> codes;
    const int status = tb == 0 ? pass(std::integral_constant<int, 0>{}, codes, 0)
                       : rank0 == 0 ? sized(codes)
                                    : sized(std::integral_constant<int, kActQuantNone>{});
    if (status != 0) return status;
  }
  return 0;
}

int launch_combine(const void* rows, int R, int n, int dtype, const int32_t* index, const float* weight, int t, int k,
                   const void* residual, void* y, void* stream) {
  const bool bf = dtype == SVDQ_OUT_BF16;
  const int w = bf ? 8 : 4;
  const bool aligned = n % w == 0 && (((uintptr_t)rows | (uintptr_t)residual | (uintptr_t)y) & 15u) == 0;
  const int units = (n + w - 1) / w;
  // A launch of 2^32 threads or more is cut short without an error, so outputs of
  // more 16-byte units (64 GB) are taken some thousand tokens at a time.
  const long long most = (0x100000000LL - 256) / units;
  const size_t row = (size_t)n * (bf ? 2 : 4);
  auto go = [&](auto kernel) {
    for (long long t0 = 0; t0 < t; t0 += most) {
      const int count = (int)std::min<long long>(t - t0, most);
      const uint8_t* res = reinterpret_cast<const uint8_t*>(residual);
      const int status = launch_checked(
          kernel, (int)(((long long)count * units + 255) / 256), 256, (hipStream_t)stream, rows, R, n, index + t0 * k,
          weight ? weight + t0 * k : nullptr, count, k, (const void*)(res ? res + t0 * row : nullptr),
          (void*)(reinterpret_cast<uint8_t*>(y) + t0 * row), units);
      if (status != 0) return status;
    }
    return 0;
  };
  if (bf) return aligned ? go(combine_kernel<true, true>) : go(combine_kernel<true, false>);
  return aligned ? go(combine_kernel<false, true>) : go(combine_kernel<false, false>);
}

}  // namespace svdq
