// The 8-bit KV cache: e4m3 values with one power-of-two scale per row and KV head.
//
// A row x of d channels is stored as x8_i = e4m3(x_i * 2^-e) and the byte e + 127, so
// that x_i ~ x8_i * 2^e.  A power of two costs a floating-point format no precision
// (only where its subnormals begin), the scale takes one byte, and x8 * 2^e has 4
// significant bits at exponents bf16 holds, so reading a row back to bf16 is exact.
//   values:       e is the least integer with a <= 448 * 2^e, a the largest |x_i|
//   rotated keys: the least with sqrt(2) * a <= 448 * 2^e, a the largest |channel|
//                 before the rotation: a rotation of a channel pair lengthens neither
//                 channel beyond sqrt(2) * a, so the scale does not depend on the
//                 position (nor on the sine's last bits), and no value saturates.
// e is kept in [-124, 120]: 2^-124 * 2^-9 = 2^-133 is bf16's smallest value; with e = 120,
// values stop at 240, because 256 * 2^120 = 2^128 is past bf16's largest.
// e4m3 has no infinities: an infinity or NaN is stored as NaN and has no part in a.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace csattn {

constexpr int kScaleMin = 3;    // code of e = -124
constexpr int kScaleMax = 247;  // code of e = 120

// Scale code of a row whose largest finite magnitude has the bf16 bits `top`.
// With top = (1 + M/128) * 2^(E-127), a <= 448 * 2^e means e >= E - 135, one more when
// 1 + M/128 exceeds 448/256 = 1.75 (M > 96), or 1.75/sqrt(2) = 1.2374 (M > 30).
__device__ __forceinline__ int scale_code(uint32_t top, bool rotated) {
  const int c = static_cast<int>(top >> 7) - 8 + ((top & 0x7fu) > (rotated ? 30u : 96u) ? 1 : 0);
  return min(max(c, kScaleMin), kScaleMax);
}

// the larger magnitude, half by half (signs are left over; a NaN makes the half NaN)
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// largest magnitude bits of 16 bf16; 0x7f80 and above: an infinity or NaN is among them
__device__ __forceinline__ uint32_t absmax16(const uint4& a, const uint4& b) {
  const uint32_t x = absmax_bf16x2(absmax_bf16x2(a.x, a.y), absmax_bf16x2(a.z, a.w));
  const uint32_t y = absmax_bf16x2(absmax_bf16x2(b.x, b.y), absmax_bf16x2(b.z, b.w));
  const uint32_t m = absmax_bf16x2(x, y) & 0x7fff7fffu;
  return max(m & 0xffffu, m >> 16);
}
__device__ __forceinline__ uint32_t fold2(uint32_t acc) {
  return max(acc & 0xffffu, acc >> 16);
}
// the same over the finite values alone
__device__ __forceinline__ uint32_t finite_absmax8(const uint4& w, uint32_t acc) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t m = v[i] & 0x7fff7fffu;
    if ((m & 0x7f80u) == 0x7f80u) m &= 0xffff0000u;
    if ((m & 0x7f800000u) == 0x7f800000u) m &= 0xffffu;
    acc = __vmaxu2(acc, m);
  }
  return acc;
}

// max over the G (a power of two) neighbouring lanes that share a row
template <int G>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Largest magnitude bits of a row held as 16 channels in each of G lanes; *bad tells
// whether the row holds an infinity or NaN (then the finite values alone count).
template <int G>
__device__ __forceinline__ uint32_t row_absmax(const uint4& a, const uint4& b, bool* bad) {
  uint32_t top = row_max<G>(absmax16(a, b));
  *bad = top >= 0x7f80u;
  // every lane takes part in the shuffles of the second pass
  if (__any_sync(0xffffffffu, *bad)) {
    const uint32_t fin = row_max<G>(fold2(finite_absmax8(b, finite_absmax8(a, 0u))));
    if (*bad) top = fin;
  }
  return top;
}

// What a value of a row that is out of the ordinary becomes: `bad` (an infinity or NaN is in
// it), or code kScaleMax.
__device__ __forceinline__ float odd_value(float x, bool bad, int code) {
  if (bad && !(fabsf(x) < INFINITY)) return __int_as_float(0x7fffffff);
  return code == kScaleMax ? fminf(fmaxf(x, -240.f), 240.f) : x;
}

// The bf16 of a row times 2^-(code - 127): a power of two, so exact (what falls below bf16's
// normal numbers is far below e4m3's least).
__device__ __forceinline__ uint4 scale_row(const uint4& w, int code) {
  const uint32_t s = static_cast<uint32_t>(254 - code) << 7, ss = s | (s << 16);
  uint4 r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(w.x), "r"(ss));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(w.y), "r"(ss));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.z) : "r"(w.z), "r"(ss));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.w) : "r"(w.w), "r"(ss));
  return r;
}

// four e4m3 (round to nearest even) of a scaled row's values, at most 448 by the choice of code
__device__ __forceinline__ uint32_t pack_e4m3x4(float y0, float y1, float y2, float y3, int code,
                                                bool bad) {
  if (bad || code == kScaleMax) {
    y0 = odd_value(y0, bad, code);
    y1 = odd_value(y1, bad, code);
    y2 = odd_value(y2, bad, code);
    y3 = odd_value(y3, bad, code);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y2, y3), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// two e4m3 (the low 16 bits) to f16x2: exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t four) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(four));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// zero the bytes of four e4m3 that are NaN
__device__ __forceinline__ uint32_t finite_e4m3x4(uint32_t w) {
  const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // 0x7f + 1
  return w & ~(nan | (nan - (nan >> 7)));
}

// Where the rows of a cache are: contiguous [B, Hkv, Lmax, ...] (block_table == nullptr)
// or pages [num_pages, Hkv, page_size, ...].
struct CacheRows {
  const int32_t* block_table;
  int Hkv, Lmax;  // Lmax: rows a sequence has room for
  int page_size, num_pages, max_pages;
  // index (in rows) of row r of KV head g of sequence b, or -1 for a page outside the pool
  __device__ __forceinline__ long long at(int b, int g, int r) const {
    if (block_table == nullptr) return (static_cast<long long>(b) * Hkv + g) * Lmax + r;
    return in_page(b, g, r, page(b, r));
  }
  // the same in two steps: the page (of a paged cache), and the row in it
  __device__ __forceinline__ int page(int b, int r) const {
    return block_table[static_cast<size_t>(b) * max_pages + r / page_size];
  }
  __device__ __forceinline__ long long in_page(int b, int g, int r, int page) const {
    if (block_table == nullptr) return (static_cast<long long>(b) * Hkv + g) * Lmax + r;
    if (page < 0 || page >= num_pages) return -1;
    return (static_cast<long long>(page) * Hkv + g) * page_size + r % page_size;
  }
};

// cos and sin of pos * theta, theta = hi + lo, 0 <= pos * theta < 2^16: the product as two floats
// (exact but for lo's), the nearest multiple of pi/2 taken off it in three parts (a Cody-Waite
// reduction; the parts are twice those of pi/4 in sinf of S. L. Moshier's Cephes library, whose
// eightfold common.cuh takes for 2 pi), then the Taylor sums on [-pi/4, pi/4] (truncated below
// 2^-27).  Off by less than 2^-23, a quarter of what __sincosf is: a key is rounded to e4m3 once,
// and every error before decides more ties.
// (On the host, too, where it is tested against long doubles.)
__host__ __device__ __forceinline__ void angle_cos_sin(int pos, float th_hi, float th_lo, float& c,
                                                       float& s) {
  const float p = static_cast<float>(pos);
  const float a_hi = p * th_hi;
  const float a_lo = fmaf(p, th_lo, fmaf(p, th_hi, -a_hi));
  const float k = rintf(a_hi * 0.63661977f);  // 2 / pi
  float r = fmaf(-k, 1.5703125f, a_hi);       // pi/2 = 201/128 + 2029/2^22 + 7.549789954e-8
  r = fmaf(-k, 4.837512969970703125e-4f, r);
  r = fmaf(-k, 7.549789954e-8f, r) + a_lo;
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
  const int q = static_cast<int>(k);
  s = (q & 1) ? cs : sn;
  c = (q & 1) ? sn : cs;
  if (q & 2) s = -s;
  if ((q + 1) & 2) c = -c;
}

// RoPE of 16 channels held as two pieces of eight (see rope_piece): y[0..7] and y[8..15]
// are the turned channels of the first and the second piece.  layout 1 (split-half): pairs
// (u_i, w_i), angle i; layout 2 (adjacent): piece one holds pairs 0..3, piece two 4..7.
__device__ __forceinline__ void rope16(const uint4& a, const uint4& b, int layout,
                                       const float (&cs)[8], const float (&sn)[8],
                                       float (&y)[16]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float u0 = bf16lo_to_f32(wa[i]), u1 = bf16hi_to_f32(wa[i]);
    const float w0 = bf16lo_to_f32(wb[i]), w1 = bf16hi_to_f32(wb[i]);
    if (layout == 1) {
      y[2 * i] = fmaf(u0, cs[2 * i], -w0 * sn[2 * i]);
      y[2 * i + 1] = fmaf(u1, cs[2 * i + 1], -w1 * sn[2 * i + 1]);
      y[8 + 2 * i] = fmaf(u0, sn[2 * i], w0 * cs[2 * i]);
      y[8 + 2 * i + 1] = fmaf(u1, sn[2 * i + 1], w1 * cs[2 * i + 1]);
    } else if (layout == 2) {
      y[2 * i] = fmaf(u0, cs[i], -u1 * sn[i]);
      y[2 * i + 1] = fmaf(u0, sn[i], u1 * cs[i]);
      y[8 + 2 * i] = fmaf(w0, cs[4 + i], -w1 * sn[4 + i]);
      y[8 + 2 * i + 1] = fmaf(w0, sn[4 + i], w1 * cs[4 + i]);
    } else {
      y[2 * i] = u0;
      y[2 * i + 1] = u1;
      y[8 + 2 * i] = w0;
      y[8 + 2 * i + 1] = w1;
    }
  }
}

// First channels of the two pieces of thread c of a row: halves of the row (each load and
// store of a row's lanes is contiguous), or with adjacent pairs 16 channels in a row, so
// that the thread's angles are 8c..8c+7 in both layouts.
__device__ __forceinline__ void rope_piece(int layout, int half, int c, int* e0, int* e1) {
  *e0 = layout == 2 ? 16 * c : 8 * c;
  *e1 = layout == 2 ? 16 * c + 8 : half + 8 * c;
}

// A query row for the products with an e4m3 cache: 16 channels of it (bf16) in each of G lanes
// are rotated (rope != 0) in fp32 and rounded once, to f16, scaled by a power of two that puts
// the largest channel before the rotation in [2^14, 2^15).  Returns what the scores are
// multiplied by.  All lanes of the warp call it.
template <int G>
__device__ __forceinline__ float query_to_f16(uint4& lo, uint4& hi, int rope,
                                              const float (&cs)[8], const float (&sn)[8]) {
  bool bad;
  const uint32_t top = row_absmax<G>(lo, hi, &bad);
  const int E = min(max(static_cast<int>(top >> 7), 15), 254);  // (scales stay normal numbers)
  const float f = __uint_as_float(static_cast<uint32_t>(268 - E) << 23);
  float y[16];
  rope16(lo, hi, rope, cs, sn, y);
  lo = make_uint4(pack_f16x2(y[0] * f, y[1] * f), pack_f16x2(y[2] * f, y[3] * f),
                  pack_f16x2(y[4] * f, y[5] * f), pack_f16x2(y[6] * f, y[7] * f));
  hi = make_uint4(pack_f16x2(y[8] * f, y[9] * f), pack_f16x2(y[10] * f, y[11] * f),
                  pack_f16x2(y[12] * f, y[13] * f), pack_f16x2(y[14] * f, y[15] * f));
  return __uint_as_float(static_cast<uint32_t>(E - 14) << 23);
}

}  // namespace csattn
