// The kernel that a product in 8-bit floating point takes, for tests that say which
// one they are about: plan.cpp built for the host with this entry point.
#include "internal.h"

// out: row blocks of the row kernel (0: tiles), tiles of 256 x 256, tiles of 64 x 128,
// parts of the last round, pieces along the channels, workspace in 64 KB.
extern "C" void fp8_plan_query(int b, int n, int m, int experts, int y_dtype, int* out) {
  const svdq::Fp8Plan p = svdq::fp8_plan(b, n, m, experts, y_dtype);
  out[0] = p.rb;
  out[1] = p.big;
  out[2] = p.small;
  out[3] = p.parts;
  out[4] = p.pieces;
  out[5] = (int)(p.ws_bytes >> 16);
}
