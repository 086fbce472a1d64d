// Device code of the 8-bit floating-point setting: E4M3 codes with one
// power-of-two scale (E8M0) for each block of 128.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"

namespace svdq {
namespace dev {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 32 codes of a lane.
__device__ __forceinline__ i32x8 operand(const u32x4& lo, const u32x4& hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// acc + A B over 128 channels with the scales' bytes, A's in byte 0 of sa, B's in
// byte `sel` of sb (a constant once inlined): v_mfma_scale_f32_16x16x128_f8f6f4,
// both operands E4M3.  The instruction takes a scale for every 32 channels, lane l
// those of channels 32 (l / 16) .. + 31 of row l % 16; a block of 128 has one, the
// same in all four.  Any order of the channels serves, being the same in both
// operands.  Its sums of eight neighbouring products keep 13 bits below the largest: for
// calls that ask for fast sums only.
__device__ __forceinline__ f32x4 mfma_scaled(const i32x8& a, const i32x8& b, const f32x4& acc, uint32_t sa, uint32_t sb,
                                             int sel) {
  switch (sel) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 0, 0, (int)sa, 0, (int)sb);
    case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 0, 0, (int)sa, 1, (int)sb);
    case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 0, 0, (int)sa, 2, (int)sb);
    default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 0, 0, (int)sa, 3, (int)sb);
  }
}

// Eight codes times their block's scale (a power of two, as a float) in bf16, which
// holds them exactly (four significant bits) inside its range: below 2^-126 to the
// multiples of 2^-133, at 2^128 to infinity.
__device__ __forceinline__ bf16x8 decode8(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// The scale's byte of a block whose largest magnitude has these bits: the least
// exponent e >= -126 with the magnitude at most 448 2^e = 1.75 2^(e+8), plus 127;
// -1 for an infinity or a NaN.
__device__ __forceinline__ int block_scale_f32(uint32_t bits) {
  if (bits >= 0x7F800000u) return -1;
  return max((int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), 1);
}
__device__ __forceinline__ int block_scale_bf16(uint32_t bits) { return block_scale_f32(bits << 16); }
// As stored: 2^0 for a block of NaN.
__device__ __forceinline__ int stored_scale(int byte) { return byte < 0 ? 127 : byte; }

// Four values (already divided by the scale) to codes.
__device__ __forceinline__ uint32_t encode4(const f32x4& v) {
  int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], q, true);
}

// Eight bf16 values to codes.
__device__ __forceinline__ uint2 encode8(const u32x4& v, int byte) {
  if (byte < 0) return uint2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
  const float s = __uint_as_float((uint32_t)byte << 23);
  // (copies: a bit cast of a vector's element takes the vector's first one)
  const uint32_t w0 = v[0], w1 = v[1], w2 = v[2], w3 = v[3];
  uint2 q;
  s16x2 lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2, w0), s, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2, w1), s, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2, w2), s, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2, w3), s, true);
  q.x = __builtin_bit_cast(uint32_t, lo);
  q.y = __builtin_bit_cast(uint32_t, hi);
  return q;
}

// Eight bf16 values of a row from column j on, zeros behind column n - 1.
__device__ __forceinline__ u32x4 load_bf16x8(const uint16_t* __restrict__ row, int j, int n) {
  typedef u32x4 Loose __attribute__((aligned(2)));
  if (j + 8 <= n) return *reinterpret_cast<const Loose*>(row + j);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (j + e < n) v[e >> 1] |= (uint32_t)row[j + e] << (16 * (e & 1));
  return v;
}

// The largest magnitude (its bf16 bits) of a block in sixteen neighbouring lanes,
// eight values each, in every one of them.
__device__ __forceinline__ uint32_t block_max16(const u32x4& v) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  auto mag = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu); };
  u16x2 t = __builtin_elementwise_max(__builtin_elementwise_max(mag(v[0]), mag(v[1])),
                                      __builtin_elementwise_max(mag(v[2]), mag(v[3])));
  uint32_t top = max((uint32_t)t[0], (uint32_t)t[1]);
  // rotations by 8, 4, 2, 1 within rows of 16 lanes (DPP row_ror)
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x128, 0xF, 0xF, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x124, 0xF, 0xF, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x122, 0xF, 0xF, true));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x121, 0xF, 0xF, true));
  return top;
}

}  // namespace dev
}  // namespace svdq
