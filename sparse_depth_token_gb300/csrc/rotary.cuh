// The rotation angles of rotary positions, shared by the cache append and the standalone
// operator.
#pragma once

#include <stdint.h>

namespace xmod {

// (cos, sin) of pos * f turns: the nearest quarter turn and a remainder r of at most pi/4,
// by the series of sine (to r^9 / 9!, off by 2e-9) and cosine (to r^8 / 8!, off by 3e-8).
__device__ __forceinline__ float2 rotation(uint64_t f, int pos) {
  const uint32_t turn = (uint32_t)((f * (uint64_t)(int64_t)pos) >> 32);
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float r = (float)(int32_t)(turn - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float r2 = r * r;
  float s = fmaf(r2, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(s, r2, 8.3333333e-3f);
  s = fmaf(s, r2, -1.6666667e-1f);
  s = fmaf(s * r2, r, r);
  float c = fmaf(r2, 2.4801587e-5f, -1.3888889e-3f);
  c = fmaf(c, r2, 4.1666667e-2f);
  c = fmaf(c, r2, -0.5f);
  c = fmaf(c, r2, 1.0f);
  float2 cs = quarter & 1 ? make_float2(s, c) : make_float2(c, s);
  // quarters 1 and 2 have a negative cosine, 2 and 3 a negative sine
  if ((quarter + 1) & 2) cs.x = -cs.x;
  if (quarter & 2) cs.y = -cs.y;
  return cs;
}

}  // namespace xmod
