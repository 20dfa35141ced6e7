// A rotary pair in integers, off by less than 2^-48 of the pair's larger element: what decides between two 4-bit codes where fp32 leaves it
// open.  (In fp64, whose units are few here, one such pair held a launch up by 14 us.)
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

namespace clo {

// What an element of a pair that fp32 rotated to x, y may be off by, with what the quotient by a group's scale and the ends of the interval round; one:
// the magnitude is 1.  Of the pair's length r = sqrt(x^2 + y^2): sine and cosine are off by 7.5e-8 of |p| + |q| <= sqrt(2) r (p, q: the unrotated pair
// times the magnitude), the product of q and the sine rounds by 2^-24 of r at most, and so do the two products with the magnitude together.  Of the
// element: the sum, the quotient and the interval's end round by 2^-24 each.  1.66e-7 r (2.26e-7 r) and 1.79e-7 of the larger element a, with
// r <= a + b / 2 for the smaller one b.
__host__ __device__ inline float rotation_error(float x, float y, bool one) {
  const float a = fmaxf(fabsf(x), fabsf(y)), b = fminf(fabsf(x), fabsf(y));
  return fmaf(a, one ? 3.46e-7f : 4.06e-7f, b * (one ? 0.83e-7f : 1.13e-7f));
}

// The elements whose 4-bit codes differ between the two ends of an interval, a bit per nibble (bit 4 k).  Zeros of either sign are one value; where
// the ends have both, the code becomes that of a positive zero.
__host__ __device__ inline uint32_t codes_differ(uint32_t* low, uint32_t high) {
  const uint32_t d = *low ^ high, any = *low | high;
  const uint32_t held = (any | any >> 1 | any >> 2) & 0x11111111u;  // not zero at both ends
  *low &= ~((d & ~(held << 3)) & 0x88888888u);
  return (d | d >> 1 | d >> 2 | d >> 3) & held;
}

// The upper half of a 128-bit product.
__host__ __device__ inline int64_t mul_high(int64_t a, int64_t b) {
#ifdef __CUDA_ARCH__
  return __mul64hi(a, b);
#else
  return (int64_t)(((__int128)a * b) >> 64);
#endif
}

// Sine and cosine of an angle in turns * 2^64, as multiples of 2^-62.  The angle's quarter goes by symmetry; the rest, at most an eighth of a
// turn, by Taylor's series: x^16 / 16! is below 2^-49 there.
__host__ __device__ inline void sin_cos_exact(uint64_t angle, int64_t* sine, int64_t* cosine) {
  constexpr double kOne = 4611686018427387904.0;  // 2^62
  const uint64_t quarter = (angle + (uint64_t(1) << 61)) >> 62;
  const int64_t rest = (int64_t)(angle - (quarter << 62));
  const int64_t x = mul_high(rest, 7244019458077122842ll) << 2;  // 2 pi 2^60
  const int64_t z = mul_high(x, x) << 3;                         // x^2 as a multiple of 2^-63
  // 1 / n!, alternating
  constexpr int64_t kSin[8] = {(int64_t)kOne, (int64_t)(-kOne / 6), (int64_t)(kOne / 120), (int64_t)(-kOne / 5040), (int64_t)(kOne / 362880),
                               (int64_t)(-kOne / 39916800), (int64_t)(kOne / 6227020800.0), (int64_t)(-kOne / 1307674368000.0)};
  constexpr int64_t kCos[8] = {(int64_t)kOne, (int64_t)(-kOne / 2), (int64_t)(kOne / 24), (int64_t)(-kOne / 720), (int64_t)(kOne / 40320),
                               (int64_t)(-kOne / 3628800), (int64_t)(kOne / 479001600.0), (int64_t)(-kOne / 87178291200.0)};
  int64_t s = kSin[7], c = kCos[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) {
    s = kSin[i] + (mul_high(s, z) << 1);
    c = kCos[i] + (mul_high(c, z) << 1);
  }
  s = mul_high(s, x) << 2;
  const int64_t cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
  *cosine = (quarter + 1) & 2 ? -cs : cs;
  *sine = quarter & 2 ? -sn : sn;
}

// v * 2^exponent as fp32, rounded to the odd one of the two nearest numbers: it lies on the same side of every border between codes as v, as
// borders have fewer bits.
__host__ __device__ inline float odd_float(int64_t v, int exponent) {
  const uint64_t m = v < 0 ? (uint64_t)-v : (uint64_t)v;
  if (m == 0) return 0.f;
#ifdef __CUDA_ARCH__
  const int zeros = __clzll((long long)m);
#else
  const int zeros = __builtin_clzll(m);
#endif
  const uint64_t top = m << zeros;
  const uint32_t bits = (uint32_t)(top >> 40) | ((top << 24) != 0 ? 1u : 0u);
  const float f = scalbnf((float)bits, exponent + 40 - zeros);
  return v < 0 ? -f : f;
}

// The elements p, q (bf16) of a pair, rotated by angle (turns * 2^64) and multiplied by magnitude.  Infinities and NaN: NaN.
__host__ __device__ inline void rotate_exact(uint16_t p, uint16_t q, uint64_t angle, float magnitude, float* rotated_p, float* rotated_q) {
  int64_t s, c;
  sin_cos_exact(angle, &s, &c);
  // mantissas of 8 bits, of 24 for the magnitude; exponents of their units
  const int fp = p >> 7 & 0xff, fq = q >> 7 & 0xff;
  if (fp == 0xff || fq == 0xff) {
    *rotated_p = *rotated_q = NAN;
    return;
  }
  const int64_t mp = (int64_t)((p & 0x7f) | (fp ? 0x80 : 0)) * (p & 0x8000 ? -1 : 1), mq = (int64_t)((q & 0x7f) | (fq ? 0x80 : 0)) * (q & 0x8000 ? -1 : 1);
  const int ep = (fp ? fp : 1) - 134, eq = (fq ? fq : 1) - 134, e = ep > eq ? ep : eq;
  const int dp = e - ep < 62 ? e - ep : 62, dq = e - eq < 62 ? e - eq : 62;
  s >>= 8;
  c >>= 8;
  const int64_t a = ((mp * c) >> dp) - ((mq * s) >> dq), b = ((mq * c) >> dq) + ((mp * s) >> dp);
  uint32_t g;
  memcpy(&g, &magnitude, 4);
  const int fg = g >> 23 & 0xff;
  const int64_t mg = (int64_t)((g & 0x7fffff) | (fg ? 0x800000 : 0)) << 39;
  const bool one = magnitude == 1.f;
  const int up = one ? 0 : 64 - 39 + (fg ? fg : 1) - 150;
  *rotated_p = odd_float(one ? a : mul_high(a, mg), e - 54 + up);
  *rotated_q = odd_float(one ? b : mul_high(b, mg), e - 54 + up);
}

}  // namespace clo
