/* Host sweep of the epilogue's GELU_ERF: the 32-bit steps of gelu_erf
 * (csrc/epilogue.h), with 2^q correctly rounded and off by an ulp either way,
 * against Phi in 64 bits.
 *     a = |v|; p = Horner(c[9] .. c[0]; a); h = 2^(a p) / 2; Phi = v < 0 ? h : 1 - h
 * Every `step`-th float from 2^-31 up to the largest finite one, both signs.
 * Results of 2^q below 2^-126 count as zero.  Prints "values worst_error
 * at_value"; worst_error is the absolute error of Phi.
 *
 * Usage: gelu_erf_sweep step c0 c1 ... c9 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static float neighbour(float x, int k) {
  uint32_t u;
  if (!(x > 0.0f)) return x;
  memcpy(&u, &x, 4);
  u += (uint32_t)k;
  memcpy(&x, &u, 4);
  return x;
}

int main(int argc, char** argv) {
  if (argc != 12) return 2;
  const uint32_t step = (uint32_t)atoi(argv[1]);
  float c[10];
  for (int i = 0; i < 10; ++i) c[i] = strtof(argv[2 + i], NULL);
  double worst = -1.0, at = 0.0;
  long count = 0;
#pragma omp parallel for schedule(dynamic, 65536) reduction(+ : count)
  for (uint32_t u = 0x30000000u; u < 0x7F800000u; u += step) {
    float a;
    memcpy(&a, &u, 4);
    float p = c[9];
    for (int i = 8; i >= 0; --i) p = fmaf(p, a, c[i]);
    float e = (float)exp2((double)(a * p));
    if (!(e >= 1.17549435e-38f)) e = e != e ? e : 0.0f;
    const double lower = 0.5 * erfc((double)a * 0.70710678118654752440); /* Phi(-a) */
    const double upper = 0.5 * erfc((double)a * -0.70710678118654752440);
    for (int k = -1; k <= 1; ++k) {
      const float h = 0.5f * neighbour(e, k);
      const double d0 = fabs((double)h - lower), d1 = fabs((double)(1.0f - h) - upper);
      const double d = d0 > d1 || d0 != d0 ? d0 : d1;
      if (!(d <= worst)) {
#pragma omp critical
        if (!(d <= worst)) worst = d, at = a;
      }
    }
    ++count;
  }
  printf("%ld %.6g %.9g\n", count, worst, at);
  return 0;
}
