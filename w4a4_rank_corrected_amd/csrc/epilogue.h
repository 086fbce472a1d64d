// The epilogue of the products with an epilogue (device code): activation,
// gate and residual applied to the fp32 result (bias already added), then one
// rounding to y's type.
//
//   a = act(v) in columns j >= act_begin, v in the others
//   y = residual[i][j] + gate[i / gate_rows][j] * a
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "internal.h"

#pragma clang fp contract(off)

namespace svdq {
namespace dev {

// exp(x) as 2^(x log2 e): one rounding of the argument (an absolute error of
// |x| 2^-24 in x, the relative error of the result) and v_exp_f32.  Results
// below 2^-126 are flushed to zero.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// 1/x to one ulp (v_rcp_f32); 1/inf = 0.
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// GELU in its tanh form, 0.5 v (1 + tanh(u)), u = sqrt(2/pi) (v + 0.044715 v^3),
// as v / (1 + exp(-2 u)): no cancellation where tanh(u) nears -1.  log2 e is in
// the polynomial's constants.
__device__ __forceinline__ float gelu_tanh(float v) {
  constexpr float c = -2.0f * 0.7978845608028654f * 1.44269504088896341f;
  const float x = v * __builtin_fmaf(v * v, c * 0.044715f, c);  // -2 u log2 e
  return v * fast_rcp(1.0f + __builtin_amdgcn_exp2f(x));
}

// GELU with the normal distribution's integral, v Phi(v).  With a = |v|,
// Phi(-a) = 2^q / 2, q = log2(2 Phi(-a)) = a P(a): q is smooth, 0 at 0, and an
// error d of q is one of Phi(-a) d ln 2 in the result, so q's rounding costs
// least where q is large; P's terms of opposite signs are small.  P: degree 9,
// fitted to |error of Phi(-a)| on [0, 5.5] by linear programming (1e-9; a weight
// of at least 2e-4 keeps 5e-6 relative up to a = 5); past it q falls below
// every bound there, to -inf.  In 32 bits, with v_exp_f32 off by an ulp either
// way, Phi is off by at most 9e-8 (the tests sweep every v); a sum of
// alternating terms times exp(-v^2/2) was off by 4e-7.
__device__ __forceinline__ float gelu_erf(float v) {
  constexpr float kPhi[10] = {-1.15110421f,   -0.459222108f,   -0.0524303243f,  0.00691764802f,  3.67327812e-05f,
                              -0.000304470537f, 8.59323773e-05f, -1.30086391e-05f, 1.08956579e-06f, -3.945798e-08f};
  const float a = fabsf(v);
  float p = kPhi[9];
#pragma unroll
  for (int e = 8; e >= 0; --e) p = __builtin_fmaf(p, a, kPhi[e]);
  const float h = 0.5f * __builtin_amdgcn_exp2f(a * p);  // Phi(-|v|)
  return v * (v < 0.0f ? h : 1.0f - h);
}

__device__ __forceinline__ float silu(float v) { return v * fast_rcp(1.0f + fast_exp(-v)); }

// NaN stays NaN
__device__ __forceinline__ float relu(float v) { return v < 0.0f ? 0.0f : v; }

template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if constexpr (ACT == SVDQ_ACT_GELU_TANH) return gelu_tanh(v);
  if constexpr (ACT == SVDQ_ACT_GELU_ERF) return gelu_erf(v);
  if constexpr (ACT == SVDQ_ACT_SILU) return silu(v);
  if constexpr (ACT == SVDQ_ACT_RELU) return relu(v);
  return v;
}

// f(integral_constant<int, ACT>) for the epilogue's activation (a wave-uniform
// choice made once, outside the loops over elements); nothing for none.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == SVDQ_ACT_GELU_TANH)
    f(std::integral_constant<int, SVDQ_ACT_GELU_TANH>{});
  else if (act == SVDQ_ACT_GELU_ERF)
    f(std::integral_constant<int, SVDQ_ACT_GELU_ERF>{});
  else if (act == SVDQ_ACT_SILU)
    f(std::integral_constant<int, SVDQ_ACT_SILU>{});
  else if (act == SVDQ_ACT_RELU)
    f(std::integral_constant<int, SVDQ_ACT_RELU>{});
}

// Vectors at any element's address: gfx950 loads and stores them unaligned, so
// a row need not start 16-byte aligned to be read and written by vectors.
typedef u32x4 u32x4_loose __attribute__((aligned(2)));
typedef uint2 uint2_loose __attribute__((aligned(2)));
typedef f32x4 f32x4_loose __attribute__((aligned(4)));

// Four consecutive columns j .. j+3 of a bf16 or fp32 row as floats; columns
// >= n read as zero.
template <bool BF16>
__device__ __forceinline__ f32x4 load4(const void* row, int j, int n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if constexpr (BF16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + j;
    if (j + 3 < n) {
      const uint2 w = *reinterpret_cast<const uint2_loose*>(p);
      v = f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < n) v[e] = __uint_as_float((uint32_t)p[e] << 16);
    }
  } else {
    const float* p = reinterpret_cast<const float*>(row) + j;
    if (j + 3 < n) {
      v = *reinterpret_cast<const f32x4_loose*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < n) v[e] = p[e];
    }
  }
  return v;
}

template <bool BF16>
__device__ __forceinline__ void store4(void* row, int j, int n, const f32x4& o) {
  if constexpr (BF16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + j;
    if (j + 3 < n) {
      *reinterpret_cast<uint2_loose*>(p) = uint2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < n) p[e] = bf16_bits(o[e]);
    }
  } else {
    float* p = reinterpret_cast<float*>(row) + j;
    if (j + 3 < n) {
      *reinterpret_cast<f32x4_loose*>(p) = o;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < n) p[e] = o[e];
    }
  }
}

// W (4, or 8 of bf16) consecutive columns j .. j+W-1 as floats; columns >= n
// read as zero.
template <int W, bool BF16>
__device__ __forceinline__ void load_cols(const void* row, int j, int n, float (&v)[W]) {
  if constexpr (W == 4) {
    const f32x4 x = load4<BF16>(row, j, n);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x[e];
  } else {
    static_assert(W == 8 && BF16, "eight bf16 columns");
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + j;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (j + 7 < n) {
      w = *reinterpret_cast<const u32x4_loose*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < n) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
  }
}
template <int W, bool BF16>
__device__ __forceinline__ void store_cols(void* row, int j, int n, const float (&v)[W]) {
  if constexpr (W == 4) {
    store4<BF16>(row, j, n, f32x4{v[0], v[1], v[2], v[3]});
  } else {
    static_assert(W == 8 && BF16, "eight bf16 columns");
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + j;
    if (j + 7 < n) {
      *reinterpret_cast<u32x4_loose*>(p) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < n) p[e] = bf16_bits(v[e]);
    }
  }
}

// Row `i` of a matrix of `BF16 ? bf16 : fp32` with row stride ld.
template <bool BF16>
__device__ __forceinline__ const void* row_of(const void* base, int i, int ld) {
  return reinterpret_cast<const uint8_t*>(base) + (size_t)i * (size_t)ld * (BF16 ? 2 : 4);
}
template <bool BF16>
__device__ __forceinline__ void* row_of(void* base, int i, int ld) {
  return reinterpret_cast<uint8_t*>(base) + (size_t)i * (size_t)ld * (BF16 ? 2 : 4);
}

// What the epilogue of four consecutive outputs of row i reads (all zero, and
// the gate one, where there is none).
struct EpiLoads {
  f32x4 bias, gate, residual;
};
template <bool OUT_BF16>
__device__ __forceinline__ EpiLoads load_unit(int i, int j, int n, const uint16_t* bias, const EpiArgs& ep) {
  EpiLoads l{{0.f, 0.f, 0.f, 0.f}, {1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}};
  if (bias) l.bias = load4<true>(bias, j, n);
  if (ep.gate) l.gate = load4<true>(row_of<true>(ep.gate, i / ep.gate_rows, n), j, n);
  if (ep.residual) l.residual = load4<OUT_BF16>(row_of<OUT_BF16>(ep.residual, i, ep.ldr), j, n);
  return l;
}

// The whole epilogue of four consecutive outputs of row i (v without the bias).
template <bool OUT_BF16>
__device__ __forceinline__ void finish_unit(f32x4 v, const EpiLoads& l, int i, int j, int n, const EpiArgs& ep) {
  v += l.bias;
  with_act(ep.act, [&](auto A) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = act_value<decltype(A)::value>(v[e]);
      v[e] = j + e >= ep.act_begin ? a : v[e];
    }
  });
  if (ep.gate) v *= l.gate;
  if (ep.residual) v = l.residual + v;
  store4<OUT_BF16>(row_of<OUT_BF16>(ep.y, i, ep.ldy), j, n, v);
}

}  // namespace dev
}  // namespace svdq
