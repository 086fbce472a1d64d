/* Exhaustive host check of the grouped activation kernel's INT4 quantizer.
 *
 * Definition: s = fp16(fl32(A / 7)) saturated, code = clamp(round_half_even(
 * fl32(v / s)), -7, 7), 0 when s = 0.  The kernel evaluates
 *     p = fl32(A r7); s32 = fma(fma(-p, 7, A), r7, p)        (r7 = fl32(1/7))
 *     code bits = bits(fl32(med3(fma(v, rc, 384), 377, 391) + (1.5*2^23 - 384))) & 0xF
 * with rc = 1/s to one ulp (v_rcp_f32): the correctly rounded reciprocal and
 * both of its neighbours are tried.  Every pair the kernel can meet is
 * enumerated: every positive finite bf16 group maximum A and every bf16 v with
 * |v| <= A, both signs.  Prints "scales pairs mismatches ties".
 *
 * Usage: quant_snap_exhaustive <table.bin> [coarse]
 *   table.bin: 32768 uint16, s(A) bits for every bf16 A, then 32768 float32,
 *              fl32(A / 7) saturated; coarse: a snap of 1.5 * 2^21 instead of
 *              384, whose grid (2^-2) swallows near-ties (a planted mistake). */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static float from_bits(uint32_t u) {
  float f;
  memcpy(&f, &u, 4);
  return f;
}
static uint32_t to_bits(float f) {
  uint32_t u;
  memcpy(&u, &f, 4);
  return u;
}
static float half_to_float(uint32_t h) {
  const uint32_t e = (h >> 10) & 0x1F, m = h & 0x3FF;
  return e == 0 ? ldexpf((float)m, -24) : ldexpf((float)(m | 0x400), (int)e - 25);
}
/* fp16 bits of a non-negative float below 65520, to nearest even */
static uint32_t float_to_half(float f) {
  if (f == 0.0f) return 0;
  int e;
  frexpf(f, &e);                                  /* f = x 2^e, x in [1/2, 1) */
  const int q = e - 11 < -24 ? -24 : e - 11;      /* exponent of the last place */
  const double n = nearbyint(ldexp((double)f, -q));
  const float r = (float)ldexp(n, q);
  if (r == 0.0f) return 0;
  frexpf(r, &e);
  if (e <= -14) return (uint32_t)ldexp((double)r, 24);
  return ((uint32_t)(e + 14) << 10) | ((uint32_t)ldexp((double)r, 11 - e) & 0x3FF);
}

int main(int argc, char** argv) {
  static uint16_t tab[32768];
  static float quo[32768];
  FILE* fp = argc > 1 ? fopen(argv[1], "rb") : NULL;
  if (!fp || fread(tab, 2, 32768, fp) != 32768 || fread(quo, 4, 32768, fp) != 32768) return 2;
  fclose(fp);
  const float snap = argc > 2 && strcmp(argv[2], "coarse") == 0 ? 3145728.0f : 384.0f;
  const float r7 = 1.0f / 7.0f, magic = 12582912.0f;
  long long scales = 0, pairs = 0, bad = 0, ties = 0;
#pragma omp parallel for schedule(dynamic, 64) reduction(+ : scales, pairs, bad, ties)
  for (uint32_t a = 1; a < 0x7F80u; ++a) {
    const float A = from_bits(a << 16);
    const float p = A * r7;
    float s32 = fmaf(fmaf(-p, 7.0f, A), r7, p);
    if (!(s32 < 65504.0f)) s32 = 65504.0f;
    ++scales;
    if (float_to_half(s32) != tab[a] || float_to_half(quo[a]) != tab[a]) {
      ++bad;
      continue;
    }
    const float s = half_to_float(tab[a]);
    if (s == 0.0f) continue;                      /* rc = 0: v1 = snap, code 0 */
    const float rc0 = 1.0f / s;
    const float rcs[3] = {rc0, nextafterf(rc0, INFINITY), nextafterf(rc0, 0.0f)};
    for (uint32_t b = 0; b <= a; ++b) {
      const float v = from_bits(b << 16);
      const float q = v / s, half = q - floorf(q);
      ties += q < 8.0f && half == 0.5f;
      float d = nearbyintf(q);
      if (d > 7.0f) d = 7.0f;
      const int want = (int)d;
      for (int k = 0; k < 3; ++k)
        for (int sign = 0; sign < 2; ++sign) {
          float t = fmaf(sign ? -v : v, rcs[k], snap);
          t = t < snap - 7.0f ? snap - 7.0f : (t > snap + 7.0f ? snap + 7.0f : t);
          const uint32_t code = to_bits(t + (magic - snap)) & 0xFu;
          bad += code != ((uint32_t)(sign ? -want : want) & 0xFu);
        }
      pairs += 6;
    }
  }
  printf("%lld %lld %lld %lld\n", scales, pairs, bad, ties);
  return bad ? 1 : 0;
}
