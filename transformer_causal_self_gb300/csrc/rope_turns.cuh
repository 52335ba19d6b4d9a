// The RoPE angle of any position below 2^24, in quarter turns.
#pragma once

#include "common.cuh"

namespace csattn {

// cos and sin of pos * theta for 0 <= pos < 2^24 and theta <= 1, given turns = theta * 2 / pi as
// hi + lo.  Counted in quarter turns, the angle's whole part is an integer that comes off without
// an error: pos * hi is taken exactly (a product and its remainder by an FMA), whole parts are
// at most 2^24, and what is left is within half a quarter turn.  Then the Taylor sums of sine and
// cosine on [-pi/4, pi/4], truncated below 2^-27.  Off by less than 2^-22.
// (On the host, too, where it is tested against long doubles.)
__host__ __device__ __forceinline__ void turn_cos_sin(int pos, float hi, float lo, float& c,
                                                      float& s) {
  const float p = static_cast<float>(pos);
  const float a = p * hi;
  const float rest = fmaf(p, lo, fmaf(p, hi, -a));
  // (past 2^22 quarter turns the product's remainder is half a turn or more itself)
  const float whole = rintf(a), more = rintf((a - whole) + rest);
  const float r = (((a - whole) - more) + rest) * 1.57079632679489662f;
  const float z = r * r;
  float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sn = fmaf(sn, z, 1.f / 120.f);
  sn = fmaf(sn, z, -1.f / 6.f);
  sn = fmaf(sn * z, r, r);
  float cs = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  cs = fmaf(cs, z, -1.f / 720.f);
  cs = fmaf(cs, z, 1.f / 24.f);
  cs = fmaf(cs, z, -0.5f);
  cs = fmaf(cs, z, 1.f);
  const int q = static_cast<int>(whole) + static_cast<int>(more);
  s = (q & 1) ? cs : sn;
  c = (q & 1) ? sn : cs;
  if (q & 2) s = -s;
  if ((q + 1) & 2) c = -c;
}

}  // namespace csattn
