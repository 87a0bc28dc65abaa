// The 4-bit cache's rows.  A row of d channels (one token of one kv head) is cut into groups of 32
// consecutive channels, each with a bf16 scale s = bf16(max|x| / 7) and codes c = the integer
// nearest to x / s (ties to even) within +-7, held as c + 8 in 4 bits: byte i of the row is channel
// 2 i in its low half and 2 i + 1 in its high half.  A scale of 8 significant bits times a code is
// exact in fp32 and, within its range, in fp16.
#pragma once

#include <cstdint>

namespace sl8 {

constexpr int kGroup4 = 32;  // channels that share a scale

// bf16(max|x| / 7) as fp32; an infinity stays one.  Maxima drop a NaN, but that of NaNs alone is one, whose bits
// the rounding below would wrap to those of -0: it counts as 0.  The division by a product and a correction by its
// exact remainder (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990), which for 7 gives the quotient's fp32 rounding for every significand; where the remainder may underflow
// or the product is infinite, by division.
__device__ __forceinline__ float group_scale(float amax) {
  amax = fmaxf(amax, 0.0f);
  constexpr float kSeventh = 1.0f / 7.0f;
  const float q = amax * kSeventh;
  float d = fmaf(fmaf(-7.0f, q, amax), kSeventh, q);
  if (!(amax > 1e-25f && amax < INFINITY)) d = __fdiv_rn(amax, 7.0f);
  const uint32_t u = __float_as_uint(d);  // not negative
  return __uint_as_float((u + 0x7fffu + ((u >> 16) & 1u)) & 0xffff0000u);
}

__device__ __forceinline__ float max3(float a, float b, float c) {  // of magnitudes; drops NaN
  asm("max.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(fabsf(b)), "f"(fabsf(c)));
  return a;
}

// The kN nibbles c + 8 of x / s, the first lowest.  k = round(x * (1 / s)) is off by one at most,
// next to a border, and x - k s is exact in one fma (k s has 11 bits, and x and k s are within a
// factor of two of each other for k != 0): where it is below s / 2 in magnitude, k is the nearest
// integer to x / s; the others are moved by what it says.
template <int kN>
__device__ __forceinline__ uint32_t nibbles(const float (&x0)[kN], float s) {
  constexpr float kRound = 12582912.0f + 8.0f;  // 1.5 * 2^23 + 8: k + 8 in the low bits of the sum
  constexpr uint32_t kBits = 0x4b400000u;       // ... and 1.5 * 2^23 above them
  float x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = x0[i];
  const bool tiny = s < 1e-30f;  // 1 / s may pass fp32: the same quotient from both times 2^96
  if (tiny) {
    s *= 7.922816251426434e28f;
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] *= 7.922816251426434e28f;
  }
  if (s == 0.0f || s == INFINITY) return 0x88888888u >> (32 - 4 * kN);
  const float r = __frcp_rn(s), h = 0.5f * s;
  uint32_t w[kN];
  float off = 0.0f;  // the largest remainder; NaN if there is one
#pragma unroll
  for (int i = 0; i < kN; i += 2) {
    const float z0 = fmaf(x[i], r, kRound), z1 = fmaf(x[i + 1], r, kRound);
    const float e0 = fmaf(kRound - z0, s, x[i]), e1 = fmaf(kRound - z1, s, x[i + 1]);
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(off) : "f"(fabsf(e0)), "f"(fabsf(e1)));
    w[i] = __float_as_uint(z0);
    w[i + 1] = __float_as_uint(z1);
  }
  if (!(off < h) || tiny) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float k = __uint_as_float(w[i]) - kRound;
      const float e = fmaf(-k, s, x[i]);
      int c = static_cast<int>(k);
      if (fabsf(e) > h || (fabsf(e) == h && (c & 1))) c += e > 0.0f ? 1 : -1;
      c = max(-7, min(7, c));  // a scale below 2^-126 can be far below max|x| / 7
      w[i] = kBits + (isnan(x[i]) ? 8u : static_cast<uint32_t>(c + 8));
    }
  }
  // sum of (w - kBits) 16^i: what the bits above the nibbles add, mod 2^32, is the same for all
  uint32_t p = w[kN - 1], extra = kBits;
#pragma unroll
  for (int i = kN - 2; i >= 0; --i) {
    p = p * 16u + w[i];
    extra = extra * 16u + kBits;
  }
  return p - extra;
}

// a b + c of two bf16 numbers and an fp32 one, one rounding; at the rate of fp32's own.  kA, kB: the half
// of the word that a number is in.
template <int kA, int kB>
__device__ __forceinline__ float fma_mixed(uint32_t a, uint32_t b, float c) {
  const uint16_t x = static_cast<uint16_t>(kA ? a >> 16 : a), y = static_cast<uint16_t>(kB ? b >> 16 : b);
  float d;
  asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(x), "h"(y), "f"(c));
  return d;
}

}  // namespace sl8
