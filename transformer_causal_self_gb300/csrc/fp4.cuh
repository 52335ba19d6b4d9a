// The 4-bit KV cache: e2m1 values with one scale byte for every 16 channels.
//
// A block x of 16 channels is stored as x4_i = e2m1(x_i / s), two to a byte (the even channel in
// the low four bits), and the byte of s: the upper bits of an f16 without its sign, 5 of exponent
// and 3 of mantissa, so that s is that byte shifted left by 7 and read as f16.
//   s = the nearest such number to a / 6, a the block's largest magnitude (6 is e2m1's), ties to
//       even, at most 10240 = 1.25 * 2^13; x4_i the nearest e2m1 to x_i / s, ties to even, at most
//       6 in magnitude; a block whose s is 0 (a at most 6 * 2^-18) holds zeros.
// e2m1 has one bit of mantissa, so a scale that were a power of two would lose up to a factor of two
// of its few values; three bits bring a / s within 7 % of 6 (but for a below 6 * 2^-14, where s
// is subnormal, and above 61440).  x4 * s has 6 significant bits, at least 2^-18 and at most 61440
// in magnitude: an f16 and a bf16 number, subnormals of s included, so that reading is exact, and so
// are the operands of the attention, which never see a scale apart from its values.
// e2m1 has neither infinities nor NaN: a block with either is stored as zeros with the byte 255,
// which is a NaN, and reads as 16 NaN.
//
// Both roundings are decided exactly in fp32: a border between two codes times s, or between two
// scales times 6, has 8 significant bits or fewer, and a bf16 number has 8, so a quotient is
// either on a border or at least 2^-10 (relative to it 2^-8) away from it; the products with the
// rounded reciprocals are off by 2^-22, and a rounding to 11 bits (or, of the smallest scales, to
// steps of 2^-12 of the border's) puts those on a border back there.
#pragma once

#include "fp8.cuh"

namespace csattn {

constexpr uint32_t kFp4Top = 226;  // the byte of 10240
constexpr uint32_t kFp4Nan = 255;

// scale byte of a block whose largest magnitude has the bf16 bits `top` (0x7f80 and above: an
// infinity or NaN is in it)
__device__ __forceinline__ uint32_t fp4_scale_code(uint32_t top) {
  const float t = fminf(__uint_as_float(top << 16) * (1.f / 6.f), 10240.f);
  // (below 2^-14 in steps of 2^-17, by way of steps of 2^-29; both by adding what has that step)
  const float y = (t * 131072.f + 2048.f) - 2048.f + 12582912.f;
  const uint32_t small = __float_as_uint(y) & 15u;
  const uint32_t h = __half_as_ushort(__float2half_rn(t));
  const uint32_t code = min((h + 63u + ((h >> 7) & 1u)) >> 7, kFp4Top);
  return top >= 0x7f80u ? kFp4Nan : (t < 6.103515625e-5f ? small : code);
}

// s of a byte
__device__ __forceinline__ float fp4_scale(uint32_t code) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(code << 7)));
}

// eight bf16 times inv to e2m1 (to nearest even, at most 6 in magnitude), by way of f16
__device__ __forceinline__ uint32_t pack_e2m1x8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4], r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = pack_f16x2(bf16lo_to_f32(w[i]) * inv, bf16hi_to_f32(w[i]) * inv);
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 a, %1;\n\tcvt.rn.satfinite.e2m1x2.f16x2 b, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 c, %3;\n\tcvt.rn.satfinite.e2m1x2.f16x2 d, %4;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return r;
}

// 1 / s within 2^-23 of it, s a scale that is not 0
__device__ __forceinline__ float fp4_inverse(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// byte I of a word, two e2m1, to f16x2: exact
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  static_assert(I >= 0 && I < 4, "byte of a word");
  uint32_t r;
  if constexpr (I == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (I == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (I == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace csattn
