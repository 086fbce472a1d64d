// The 4-bit quantizers of the activation kernels (device code).
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"
#include "internal.h"

#pragma clang fp contract(off)

namespace svdq {
namespace {

using namespace dev;

// FP8 E4M3 rounding of x >= 0 (nearest, ties to even, saturated at 448): the
// quantum is 2^(e-3) in the binade [2^e, 2^(e+1)) for e >= -6, 2^-9 below.
__device__ __forceinline__ float e4m3_round(float x) {
  if (!(x < 448.0f)) return 448.0f;
  const int e = max((int)((__float_as_uint(x) >> 23) & 0xFF) - 127, -6);
  const float down = __uint_as_float((uint32_t)(127 - (e - 3)) << 23);  // 2^-(e-3), exact
  const float up = __uint_as_float((uint32_t)(127 + (e - 3)) << 23);    // 2^(e-3)
  return fminf(__builtin_rintf(x * down) * up, 448.0f);
}

// Bit pattern of a non-negative E4M3 value.
__device__ __forceinline__ uint32_t e4m3_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  const int e = (int)((u >> 23) & 0xFF) - 127;
  if (v == 0.0f) return 0u;
  if (e >= -6) return ((uint32_t)(e + 7) << 3) | ((u >> 20) & 7u);
  return (uint32_t)(v * 512.0f);  // subnormal: v = m 2^-9, m = 1..7 (exact)
}

// Quantizes one row-group piece of the smoothed tile and stores its codes and
// scale (INT4 or NVFP4; nothing for kActQuantNone).  v: this lane's 16
// smoothed bf16 values (channels 8c..8c+7 and 32+8c..32+8c+7 of group g of
// row `row`), in the lane layout of the act-quant kernels: lanes l, l ^ 16,
// l ^ 32, l ^ 48 hold the same row.  q_off / s_off: this lane's byte offsets
// of its code words and of the row's scale in the group's records.
template <int Q>
__device__ __forceinline__ void quant_store(const float (&v)[16], int g, int b, int row, int c, uint32_t q_off,
                                            uint32_t s_off, uint8_t* __restrict__ qx,
                                            uint16_t* __restrict__ ascale, float tx) {
  if constexpr (Q == kActQuantFp4) {
    // NVFP4: blocks of 16 channels; this lane holds half of block c >> 1
    // (v[0..7]) and half of block 2 + (c >> 1) (v[8..15]), lane l ^ 16 the
    // other halves.  sb = E4M3(fl32(amax / 6) / t), S = sb t (t a power of
    // two), codes E2M1_RNE_sat(fl32(v / S)) with the quotient's sign.
    float am[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 16; ++e) am[e >> 3] = fmaxf(am[e >> 3], fabsf(v[e]));
    uint32_t w[2];
    uint32_t sbits[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float a = fmaxf(am[h], __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(am[h]), 0x401F)));
      const float u = a / 6.0f;                    // IEEE division (correctly rounded)
      const float sb = e4m3_round(u * (1.0f / tx));  // 1/t and the product are exact
      sbits[h] = e4m3_bits(sb);
      const float S = sb * tx;                      // exact
      const float rc = S > 0.0f ? 1.0f / S : 0.0f;
      const float S8 = 8.0f * S;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float vv = v[8 * h + e];
        const float pq = vv * rc;
        const float rem = __builtin_fmaf(-pq, S, vv);
        const float q1 = __builtin_fmaf(rem, rc, pq);
        y[e] = S > 0.0f ? __builtin_copysignf(fabsf(vv) <= S8 ? q1 : 8.0f, vv) : 0.0f;
      }
      // two codes per byte, the even channel in the low nibble (RNE on the
      // E2M1 grid, saturating: the hardware conversion at unit scale)
      uint32_t word = 0u;
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, y[0], y[1], 1.0f, 0);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, y[2], y[3], 1.0f, 1);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, y[4], y[5], 1.0f, 2);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, y[6], y[7], 1.0f, 3);
      w[h] = word;
    }
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(qx + (size_t)g * b * 32, (uint32_t)b * 32u);
    __builtin_amdgcn_raw_buffer_store_b32(w[0], rq, q_off, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(w[1], rq, q_off + 16u, 0, 0);
    // block scales: record [m/64][b][4] bytes, byte j = block j; the lanes
    // with even c store blocks c/2 and 2 + c/2 (odd c: an offset past the
    // end, dropped)
    uint8_t* sc8 = reinterpret_cast<uint8_t*>(ascale);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(sc8 + (size_t)g * b * 4, (uint32_t)b * 4u);
    const uint32_t s8_off = (c & 1) == 0 ? (uint32_t)row * 4u + (uint32_t)(c >> 1) : 0x7FFFFFF0u;
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)sbits[0], rs, s8_off, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)sbits[1], rs, s8_off + 2u, 0, 0);
  }
  if constexpr (Q == kActQuantInt4) {
    float am = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) am = fmaxf(am, fabsf(v[e]));
    am = max4_rows(am);
    float s32 = am / 7.0f;                 // IEEE division (correctly rounded)
    s32 = fminf(s32, 65504.0f);            // saturate instead of rounding to inf
    const _Float16 s16 = (_Float16)s32;    // round to nearest even
    const float sf = (float)s16;
    const float rc = sf > 0.0f ? 1.0f / sf : 0.0f;
    // rb[e]: the bits of q + 1.5 * 2^23, whose low byte is the code in two's
    // complement (the addition rounds to the nearest integer, ties to even)
    uint32_t rb[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float pq = v[e] * rc;
      const float rem = __builtin_fmaf(-pq, sf, v[e]);
      const float q1 = __builtin_fmaf(rem, rc, pq);
      const float q = __builtin_amdgcn_fmed3f(q1, -7.0f, 7.0f);
      rb[e] = __float_as_uint(q + kMagic);
    }
    // Nibble e of a word (bits 4e..4e+3) is code e: byte permutes gather the
    // even codes' and the odd codes' low bytes into two words, then one
    // bitfield insert takes the low nibbles of the first and the shifted low
    // nibbles of the second.
    auto pack8 = [](const uint32_t* c8) {
      const uint32_t e01 = __builtin_amdgcn_perm(c8[2], c8[0], 0x0c0c0400u);  // bytes: c0, c2, 0, 0
      const uint32_t e23 = __builtin_amdgcn_perm(c8[6], c8[4], 0x04000c0cu);  // bytes: 0, 0, c4, c6
      const uint32_t o01 = __builtin_amdgcn_perm(c8[3], c8[1], 0x0c0c0400u);
      const uint32_t o23 = __builtin_amdgcn_perm(c8[7], c8[5], 0x04000c0cu);
      return ((e01 | e23) & 0x0F0F0F0Fu) | (((o01 | o23) << 4) & 0xF0F0F0F0u);
    };
    const uint32_t w0 = pack8(rb), w1 = pack8(rb + 8);
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(qx + (size_t)g * b * 32, (uint32_t)b * 32u);
    __builtin_amdgcn_raw_buffer_store_b32(w0, rq, q_off, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(w1, rq, q_off + 16u, 0, 0);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(ascale + (size_t)g * b, (uint32_t)b * 2u);
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, s16), rs, s_off, 0, 0);
  }
}

// The INT4 quantizer of quant_store with fewer instructions per element (three
// instead of five, and no IEEE division): the same codes and scales for all
// finite values.  A row's four lanes are neighbours here (lane 4 r + c).
//   scale: fl32(am / 7) as p = am r7, fma(fma(-p, 7, am), r7, p) with r7 =
//     fl32(1/7): the same fp16 for every bf16 am (enumerated in the tests).
//   codes: round_half_even(fl32(v / s)) needs v / s only near a tie k + 1/2.  A
//     bf16 v (8 significant bits) and an fp16 s (11) have v / s = k + 1/2 exactly
//     or at least 2^-12 away from it, for |v / s| in 1/4 .. 8 (a nonzero
//     2 v - (2k+1) s is a multiple of the finer of s's last bit and twice v's: s's
//     is s 2^-11 or more, twice v's v 2^-7 or more, and the distance is that over
//     2 s).  With rc = 1/s to an ulp, v rc is off by at most 2^-20, so fma(v, rc,
//     384), which rounds to multiples of 2^-15, lands on the tie exactly where there
//     is one and on its own side of it elsewhere; the clamp and the rounding addition
//     then give the definition's code (384 is even, so ties keep their parity).
__device__ __forceinline__ void quant_store_int4(const float (&v)[16], int g, int b, uint32_t q_off, uint32_t s_off,
                                                 uint8_t* __restrict__ qx, uint16_t* __restrict__ ascale) {
  float am = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) am = fmaxf(am, fabsf(v[e]));
  // the row's other three lanes: quad_perm [1,0,3,2], then [2,3,0,1]
  am = fmaxf(am, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(am), 0xB1, 0xF, 0xF, false)));
  am = fmaxf(am, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(am), 0x4E, 0xF, 0xF, false)));
  constexpr float r7 = 1.0f / 7.0f, kSnap = 384.0f;
  const float p7 = am * r7;
  const float s32 = fminf(__builtin_fmaf(__builtin_fmaf(-p7, 7.0f, am), r7, p7), 65504.0f);
  const _Float16 s16 = (_Float16)s32;
  const float sf = (float)s16;
  const float rc = sf > 0.0f ? __builtin_amdgcn_rcpf(sf) : 0.0f;
  uint32_t rb[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float q = __builtin_amdgcn_fmed3f(__builtin_fmaf(v[e], rc, kSnap), kSnap - 7.0f, kSnap + 7.0f);
    rb[e] = __float_as_uint(q + (kMagic - kSnap));
  }
  auto pack8 = [](const uint32_t* c8) {  // as in quant_store
    const uint32_t e01 = __builtin_amdgcn_perm(c8[2], c8[0], 0x0c0c0400u);
    const uint32_t e23 = __builtin_amdgcn_perm(c8[6], c8[4], 0x04000c0cu);
    const uint32_t o01 = __builtin_amdgcn_perm(c8[3], c8[1], 0x0c0c0400u);
    const uint32_t o23 = __builtin_amdgcn_perm(c8[7], c8[5], 0x04000c0cu);
    return ((e01 | e23) & 0x0F0F0F0Fu) | (((o01 | o23) << 4) & 0xF0F0F0F0u);
  };
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(qx + (size_t)g * b * 32, (uint32_t)b * 32u);
  __builtin_amdgcn_raw_buffer_store_b32(pack8(rb), rq, q_off, 0, 0);
  __builtin_amdgcn_raw_buffer_store_b32(pack8(rb + 8), rq, q_off + 16u, 0, 0);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(ascale + (size_t)g * b, (uint32_t)b * 2u);
  __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, s16), rs, s_off, 0, 0);
}

}  // namespace
}  // namespace svdq
