// Device helpers that the decode kernels share: reductions over the lanes of a query
// column, exact widening of int8 codes, warp-level MMAs and the query row quantiser.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sl8_internal.h"

namespace sl8 {

constexpr float kLazy = 8.0f;  // log2 headroom of the lazy max
constexpr int kLazyLists = 5;  // the same over page lists, where the V scales have the rest (scale_limit)

__device__ __forceinline__ float bf16_bits(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ float f16_bits(uint32_t b) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
}
__device__ __forceinline__ float warp_max_f(float a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}
// max / sum over the 8 lanes of one thread-in-group column (lanes t, t+4, ..., t+28)
__device__ __forceinline__ float col_max(float a) {
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
  return fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
}
__device__ __forceinline__ float col_sum(float a) {
  a += __shfl_xor_sync(0xffffffffu, a, 4);
  a += __shfl_xor_sync(0xffffffffu, a, 8);
  return a + __shfl_xor_sync(0xffffffffu, a, 16);
}
// A sum that a NaN logit has made NaN belongs to no maximum where all of a warp's logits were
// NaN (maxima drop it): with the reference 0 instead of -inf, which says that there was no
// token, the merges keep it.
__device__ __forceinline__ float keep_nan(float m, float l) { return isnan(l) && m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns, DeviceStatus* st,
                                          int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns, st, site));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^n as a float for -126 <= n <= 127, 0 below.
__device__ __forceinline__ float pow2i(int n) {
  return n < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// P' of one token and two query columns as fp16 pairs, rounded, and what the rounding left:
// (p s_v) 2^-E in this order, two at a time (s_v 2^-E alone may pass fp32 where p is 0).
__device__ __forceinline__ void weights_f16x2(float pa, float pb, float v, float inv_a, float inv_b, uint32_t& hi,
                                              uint32_t& lo) {
  asm("{\n\t.reg .b64 p, f;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 f, {%2, %2};\n\tmul.rn.f32x2 p, p, f;\n\t"
      "mov.b64 f, {%3, %4};\n\tmul.rn.f32x2 p, p, f;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(pa), "+f"(pb)
      : "f"(v), "f"(inv_a), "f"(inv_b));
  const __half2 h = __floats2half2_rn(pa, pb);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = f16x2_of(pa - f.x, pb - f.y);
}
// 1 / x of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float pow2_inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }
// The slow step of the online softmax over page lists, for one query column of a unit: logits xA
// and xB (log2 units) of the lane's two tokens, whose V scales are vA and vB.  P' = p s_v 2^-E
// goes to the MMAs in fp16, and E has to follow the weights p s_v, not the scales alone: a
// token of no weight and a huge scale would push all other P' below fp16's normal range.  So 2^E
// is about the largest weight, the unit's or what the earlier ones' has become under the new
// maximum, and at most twice it: P' is off by 2^-11 of itself or by 2^-24 of that weight.  The
// unit's comes from x plus s_v's exponent, whose maximum needs no wait for x's (where |x| passes
// 2^20, from s_v alone).  Returns what the O' so far is multiplied with.
__device__ __forceinline__ float grow_column(float xA, float xB, float vA, float vB, float& m, float& th, float& l,
                                             float& inv) {  // inv = 2^-E
  auto bounded = [](float x) { return fminf(fmaxf(x, -1048576.0f), 1048576.0f); };
  auto with_scale = [&](float x, float v) {  // v < 2^(its exponent field - 126)
    return bounded(x) + static_cast<float>(static_cast<int>((__float_as_uint(v) >> 23) & 0xffu) - 126);
  };
  const float mx = col_max(fmaxf(xA, xB)), my = col_max(fmaxf(with_scale(xA, vA), with_scale(xB, vB)));
  float shift = 0.0f;
  if (mx > th) {
    shift = m - mx;
    l *= ex2(shift);
    m = mx;
    th = mx + static_cast<float>(kLazyLists);
  }
  const int before = 127 - static_cast<int>(__float_as_uint(inv) >> 23);
  const int now = __float2int_ru(my - bounded(m)) - 1;  // the weight is in [2^(now - 1), 2^(now + 1))
  const int E = max(-126, min(126, max(now, before + __float2int_rd(fmaxf(shift, -252.0f)))));
  inv = pow2i(-E);
  return ex2(shift + static_cast<float>(before - E));  // at most 2
}
// The V scale up to which no column needs the slow step: with p <= 2^5 and s_v <= 2^10 2^E for the
// least E of the columns, P' stays below 2^15.  A list whose heaviest token has small values (an
// attention sink) keeps E low, and rows above the limit take the slow step every time: with 2^8
// and 2^7, 600 lists of 4,096 tokens at d = 64 whose heaviest rows had a 200th of the others'
// scales took 60.3 us; 55.2 so, as any other lists.
__device__ __forceinline__ float scale_limit(float inv_a, float inv_b) {
  float inv = fmaxf(inv_a, inv_b);
  inv = fmaxf(inv, __shfl_xor_sync(0xffffffffu, inv, 1));
  inv = fmaxf(inv, __shfl_xor_sync(0xffffffffu, inv, 2));
  return pow2i(min(127, 127 - static_cast<int>(__float_as_uint(inv) >> 23) + 15 - kLazyLists));
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// Two int8 codes, already offset by 128 (byte ^ 0x80), picked from ub by sel (0x4140:
// bytes 0 and 1; 0x4342: bytes 2 and 3) and widened exactly to an fp16 pair: each byte
// u becomes the mantissa of 1024 + u, and subtracting 1152 leaves u - 128.
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t ub, uint32_t sel) {
  const uint32_t h = prmt(ub, 0x64646464u, sel);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Exact int8 products summed in int32: 16 rows x 32 bytes of A, 8 columns of B.
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 fp16 matrix held one register per lane (lane l: row l / 4,
// columns 2 (l % 4) and 2 (l % 4) + 1), into the same layout.
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Quantise one q row of D values (f16/bf16/f32) held by a warp, D / 32 per lane.
template <int D>
__device__ __forceinline__ float quant_row_warp(const float (&v)[D / 32], int8_t (&code)[D / 32]) {
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) amax = fmaxf(amax, fabsf(v[e]));
  amax = warp_max_f(amax);
  const float sc = __fdiv_rn(amax, 127.0f);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    int c = 0;
    if (sc != 0.0f) {
      c = __float2int_rn(__fdiv_rn(v[e], sc));
      c = c > 127 ? 127 : (c < -127 ? -127 : c);
    }
    code[e] = static_cast<int8_t>(c);
  }
  return sc;
}

// The same quantiser without a division per value.  x * (1 / s) is within 2^-16 of the fp32
// quotient x / s (|x / s| <= 127; one rounding each in 1 / s and the quotient, the product
// is exact in the fma), so wherever it lies more than 1e-4 from a rounding border, both
// round to the same code; the few values nearer than that, rows whose scale has no fp32
// reciprocal and values that are not finite take the division.
struct RowScale {
  float s, r;  // the scale; what to multiply with, or 0 where the division is always taken
};
__device__ __forceinline__ RowScale row_scale(float amax) {
  const float s = __fdiv_rn(amax, 127.0f);
  // a row of zeros needs none: its codes are 0 whatever they are multiplied with
  return {s, s == 0.0f ? 1.0f : s > 1e-30f && s < 1e30f ? __frcp_rn(s) : 0.0f};
}
// Codes of four values, one per byte.
__device__ __forceinline__ uint32_t quant4(const float (&x)[4], const RowScale& q) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it leaves the nearest integer in the low bits
  uint32_t w[4];
  bool sure = q.r != 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float z = fmaf(x[i], q.r, kRound);
    sure = sure && fabsf(fmaf(x[i], q.r, kRound - z)) < 0.4999f;
    w[i] = __float_as_uint(z);
  }
  if (!sure) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = q.s == 0.0f ? 0u : static_cast<uint32_t>(max(-127, min(127, __float2int_rn(__fdiv_rn(x[i], q.s)))));
  }
  return prmt(prmt(w[0], w[1], 0x0040), prmt(w[2], w[3], 0x0040), 0x5410);
}

__device__ __forceinline__ float load_q_elem(const void* base, sl8_dtype dt, int64_t idx) {
  return dt == SL8_BF16 ? bf16_bits(static_cast<const uint16_t*>(base)[idx])
       : dt == SL8_F16 ? f16_bits(static_cast<const uint16_t*>(base)[idx])
                       : static_cast<const float*>(base)[idx];
}
// kN runs of four consecutive elements, the runs `step` elements apart, each from a multiple
// of four.  The type is looked at once, around all loads, so that they are in flight
// together.
template <int kN>
__device__ __forceinline__ void load_runs(const void* base, sl8_dtype dt, int64_t idx, int step, float (&x)[kN][4]) {
  if (dt == SL8_F32) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + idx + i * step);
      x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
    }
    return;
  }
  uint2 v[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + idx + i * step);
  if (dt == SL8_BF16) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      x[i][0] = bf16_bits(v[i].x & 0xffffu), x[i][1] = bf16_bits(v[i].x >> 16);
      x[i][2] = bf16_bits(v[i].y & 0xffffu), x[i][3] = bf16_bits(v[i].y >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      x[i][0] = f16_bits(v[i].x & 0xffffu), x[i][1] = f16_bits(v[i].x >> 16);
      x[i][2] = f16_bits(v[i].y & 0xffffu), x[i][3] = f16_bits(v[i].y >> 16);
    }
  }
}
__device__ __forceinline__ void store_out(void* out, sl8_dtype dt, int64_t idx, float v) {
  if (dt == SL8_F32) static_cast<float*>(out)[idx] = v;
  else if (dt == SL8_BF16) static_cast<__nv_bfloat16*>(out)[idx] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[idx] = __float2half_rn(v);
}

}  // namespace sl8
