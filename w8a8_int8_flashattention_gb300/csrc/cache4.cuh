// The 4-bit cache's rows.  A row of d channels (one token of one kv head) is cut into groups of 32
// consecutive channels, each with a bf16 scale s = bf16(max|x| / 7) and codes c = the integer
// nearest to x / s (ties to even) within +-7, held as c + 8 in 4 bits: byte i of the row is channel
// 2 i in its low half and 2 i + 1 in its high half.  A scale of 8 significant bits times a code is
// exact in fp32 and, within its range, in fp16.
#pragma once

#include <cstdint>

namespace sl8 {

constexpr int kGroup4 = 32;  // channels that share a scale

// bf16(max|x| / 7) as fp32; a NaN never gets here (maxima drop it), an infinity stays one.
__device__ __forceinline__ float group_scale(float amax) {
  const uint32_t u = __float_as_uint(__fdiv_rn(amax, 7.0f));  // not negative
  return __uint_as_float((u + 0x7fffu + ((u >> 16) & 1u)) & 0xffff0000u);
}

// The four nibbles c + 8 of x / s, the first lowest.  k = round(x * (1 / s)) is off by one at most,
// next to a border, and x - k s is exact in one fma (k s has 11 bits, and x and k s are within a
// factor of two of each other for k != 0): where it is below s / 2 in magnitude, k is the nearest
// integer to x / s; the others are moved by what it says.
__device__ __forceinline__ uint32_t nibbles4(const float (&x0)[4], float s) {
  constexpr float kRound = 12582912.0f + 8.0f;  // 1.5 * 2^23 + 8: k + 8 in the low bits of the sum
  float x[4] = {x0[0], x0[1], x0[2], x0[3]};
  const bool tiny = s < 1e-30f;  // 1 / s may pass fp32: the same quotient from both times 2^96
  if (tiny) {
    s *= 7.922816251426434e28f;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= 7.922816251426434e28f;
  }
  if (s == 0.0f || s == INFINITY) return 0x8888u;
  const float r = __frcp_rn(s), h = 0.5f * s;
  uint32_t w[4];
  bool sure = !tiny;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float z = fmaf(x[i], r, kRound);
    sure = sure && fabsf(fmaf(kRound - z, s, x[i])) < h;
    w[i] = __float_as_uint(z);
  }
  if (!sure) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float k = __uint_as_float(w[i]) - kRound;
      const float e = fmaf(-k, s, x[i]);
      int c = static_cast<int>(k);
      if (fabsf(e) > h || (fabsf(e) == h && (c & 1))) c += e > 0.0f ? 1 : -1;
      c = max(-7, min(7, c));  // a scale below 2^-126 can be far below max|x| / 7
      w[i] = isnan(x[i]) ? 8u : static_cast<uint32_t>(c + 8);
    }
  }
  return (w[0] & 15u) | ((w[1] & 15u) << 4) | ((w[2] & 15u) << 8) | ((w[3] & 15u) << 12);
}

}  // namespace sl8
