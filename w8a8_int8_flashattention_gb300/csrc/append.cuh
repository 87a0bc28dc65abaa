// Rotary positions fused with the quantised append to the paged cache, for the int8 pages
// (paged.cu) and the 4-bit ones (cache4.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "cache4.cuh"
#include "decode_unit.cuh"
#include "sl8_internal.h"

namespace sl8 {

namespace {

struct AppendArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements from token to token
  int32_t T, Hq, Hkv;
  const int32_t* positions;  // [axes][T]
  int32_t axes, rot;
  const float* inv_freq;     // [rot / 2]
  void* q_out;
  const int32_t* slot_map;   // [T]
  void *k_pages, *v_pages;
  void *k_scale, *v_scale;
  const float* k_mean;       // [Hkv][D], nullable (4 bits)
  int32_t num_pages, page;
  int32_t iters;             // row groups of a token that one warp handles
  int32_t parts;             // warps per token
  uint8_t axis[128];         // axis of each rotary pair
};

// Four values as they lie in memory, and widened to fp32.
template <typename T>
struct Raw4 {
  uint2 v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void widen(float (&x)[4]) const;
};
template <>
struct Raw4<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void widen(float (&x)[4]) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
};
template <>
__device__ __forceinline__ void Raw4<__half>::widen(float (&x)[4]) const {
  x[0] = f16_bits(v.x & 0xffffu), x[1] = f16_bits(v.x >> 16);
  x[2] = f16_bits(v.y & 0xffffu), x[3] = f16_bits(v.y >> 16);
}
template <>
__device__ __forceinline__ void Raw4<__nv_bfloat16>::widen(float (&x)[4]) const {
  x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4]);
template <>
__device__ __forceinline__ void store4<float>(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
template <>
__device__ __forceinline__ void store4<__half>(__half* p, const float (&x)[4]) {
  const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Angles as fixed-point turns.  turns_of(f) is f / (2 pi) mod 1 in units of 2^-64: the
// 24-bit mantissa of f times 2^64 / (2 pi), shifted by f's exponent.  Times an int32 position,
// mod 2^64, the top 32 bits are the turns of the position's angle at any position, where a
// product in fp32 would lose 0.06 rad at position 2^20; whole turns drop out by themselves.
// What g drops of f / (2 pi), less than 2^-63 turns (for f above 1, f times that), is at most
// 2^-32 turns at position 2^31, and 2^-22 (1.5e-6 rad) at f = 1,000.
__device__ __forceinline__ uint64_t turns_of(float f) {
  constexpr uint64_t kInv2Pi = 0x28be60db9391054aull;  // 2^64 / (2 pi)
  const uint32_t u = __float_as_uint(f);
  const int e = static_cast<int>((u >> 23) & 0xffu) - 127;  // |f| = m 2^(e - 23)
  const uint64_t m = e == -127 ? 0u : ((u & 0x7fffffu) | 0x800000u);
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int sh = 23 - e;  // right shift of the 128-bit product
  uint64_t g = 0;
  if (sh <= 0) g = sh > -64 ? lo << -sh : 0;
  else if (sh < 64) g = (hi << (64 - sh)) | (lo >> sh);
  else if (sh < 128) g = hi >> (sh - 64);
  return (u >> 31) ? 0 - g : g;
}
// Cosine and sine of the angle of `pos`: sincospif takes half turns.
__device__ __forceinline__ void turn(int32_t pos, uint64_t g, float& c, float& s) {
  const uint64_t w = static_cast<uint64_t>(static_cast<int64_t>(pos)) * g;
  sincospif(static_cast<float>(static_cast<int32_t>(w >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
}

// Rotate q and k, quantise k and v.  A row (one head of one token) is held by D / 8 lanes,
// two groups of four values each: lane l of the row holds rotary pairs 4 l .. 4 l + 3 as
// (4 l, rot / 2 + 4 l) halves, or the eight adjacent values 8 l .. 8 l + 7 when pairs are
// adjacent, and the lanes past the rotated part hold eight plain values.  So a lane needs
// the same four angles for every head: it computes them once per token and keeps them in
// registers, and no lane exchanges values but the row maximum.  A warp takes 256 / D rows of
// one kind (q, k or v) at a time, a "group", and has kBatch groups of loads in flight.
// HBM-bound: q, k and v are read once, q is written once and k, v as codes; 16,384 tokens of
// 16 + 2 x 8 heads at d = 256 take 85 us, 5.5 TB/s, 0.81 of the measured copy rate (with
// four groups in flight 89, five 98: the registers cost more warps than they add loads).
// One wave of 4,099 tokens (16 + 2 x 2 heads, d = 128) takes 11 us, and 11.8 with eight warps a
// CTA instead of four, whose slots are free only once all of them end.
//
// kBits = 8: int8 codes, one fp32 scale a row.  kBits = 4: a bf16 scale for each group of 32
// channels.  A lane's eight values in a row are a quarter of one; the runs of four that a lane has when
// pairs are halves lie in two, whose other runs any lane of the row may hold, so the maxima are
// shuffled to the order of the channels and the scales back.  The same 16,384 tokens take 86 us (108
// with a division for each scale, two scales a lane and each value's border tested by itself); the 4,099
// 11.0, and 13.9 with more than 72 registers, which would be more than one wave of warps.
template <typename T, int D, bool kAdjacent, int kBits>
__global__ void __launch_bounds__(128, kBits == 4 ? 7 : 0) rope_append_kernel(const AppendArgs a, DeviceStatus* st) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = sizeof(T) == 4 ? 2 : 3;
  const int lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * 4 + (threadIdx.x >> 5);
  const uint32_t tok = a.parts == 1 ? w : w / static_cast<uint32_t>(a.parts);
  if (tok >= static_cast<uint32_t>(a.T)) return;
  const int part = static_cast<int>(w - tok * a.parts);
  const int l = lane % kLanes, sub = lane / kLanes;
  const bool turned = 8 * l < a.rot;
  const int ea = !kAdjacent && turned ? 4 * l : 8 * l;
  const int eb = !kAdjacent && turned ? a.rot / 2 + 4 * l : 8 * l + 4;
  // groups: gq of q rows, then gk of k rows, then gk of v rows; this warp's are [g0, g1)
  const int gq = (a.Hq + kRows - 1) / kRows, gk = (a.Hkv + kRows - 1) / kRows;
  const int g0 = part * a.iters, g1 = min(gq + 2 * gk, g0 + a.iters);
  const int32_t slot = a.slot_map[tok];
  float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto rotate = [&](float (&x)[4], float (&y)[4]) {
    if (!turned) return;
    if constexpr (kAdjacent) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
        x[2 * j] = fmaf(x0, c[j], -(x1 * s[j]));
        x[2 * j + 1] = fmaf(x1, c[j], x0 * s[j]);
        y[2 * j] = fmaf(y0, c[j + 2], -(y1 * s[j + 2]));
        y[2 * j + 1] = fmaf(y1, c[j + 2], y0 * s[j + 2]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x0 = x[j], y0 = y[j];
        x[j] = fmaf(x0, c[j], -(y0 * s[j]));
        y[j] = fmaf(y0, c[j], x0 * s[j]);
      }
    }
  };
  // Groups [from, to) of one kind, whose rows start at src: kBatch groups are on their way
  // while one is worked on.  The last head stands in for lanes past it, which store nothing.
  auto stream = [&](const T* src, int from, int to, int heads, int ea, int eb, auto first, auto work) {
    Raw4<T> ra[kBatch], rb[kBatch];
    auto fetch = [&](int g, Raw4<T>& x, Raw4<T>& y) {
      const T* p = src + min(g * kRows + sub, heads - 1) * D;
      x.load(p + ea);
      y.load(p + eb);
    };
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (from + i < to) fetch(from + i, ra[i], rb[i]);
    first();
    for (int g = from; g < to; g += kBatch) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (g + i >= to) break;
        float x[4], y[4];
        ra[i].widen(x);
        rb[i].widen(y);
        if (g + i + kBatch < to) fetch(g + i + kBatch, ra[i], rb[i]);
        work((g + i) * kRows + sub, x, y);
      }
    }
  };
  bool angles = false;
  auto make_angles = [&] {  // once, behind the first rows' loads
    if (angles || !turned) return;
    angles = true;
    float f[4];
    int32_t pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a.inv_freq[4 * l + i];
      pos[i] = a.positions[static_cast<int64_t>(a.axis[4 * l + i]) * a.T + tok];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(pos[i], turns_of(f[i]), c[i], s[i]);
  };
  if (g0 < gq) {
    T* const out = static_cast<T*>(a.q_out) + tok * a.q_out_stride;
    stream(static_cast<const T*>(a.q) + tok * a.q_stride, g0, min(g1, gq), a.Hq, ea, eb, make_angles,
           [&](int h, float (&x)[4], float (&y)[4]) {
             rotate(x, y);
             if (h < a.Hq) {
               store4<T>(out + h * D + ea, x);
               store4<T>(out + h * D + eb, y);
             }
           });
  }
  if (g1 <= gq || slot < 0) return;
  const uint32_t pg = static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page);
  if (pg >= static_cast<uint32_t>(a.num_pages)) {
    if (lane == 0 && g1 == gq + 2 * gk) record_status(st, kStatusBadArg, 810);
    return;
  }
  // the slot's row in the first head of its page
  const int64_t row0 = static_cast<int64_t>(pg) * a.Hkv * a.page + (static_cast<uint32_t>(slot) - pg * a.page);
  auto store_codes = [&](void* pages, void* scales, int h, int qa, int qb, const float (&x)[4], const float (&y)[4]) {
    const int64_t row = row0 + static_cast<int64_t>(h) * a.page;
    if constexpr (kBits == 8) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(x[j]), fabsf(y[j])));
      if constexpr (kLanes == 32) {  // magnitudes order as their bits do
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
      } else {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
      const RowScale rs = row_scale(m);
      const uint32_t ca = quant4(x, rs), cb = quant4(y, rs);
      if (h < a.Hkv) {
        *reinterpret_cast<uint32_t*>(static_cast<int8_t*>(pages) + row * D + qa) = ca;
        *reinterpret_cast<uint32_t*>(static_cast<int8_t*>(pages) + row * D + qb) = cb;
        if (l == 0) static_cast<float*>(scales)[row] = rs.s;
      }
    } else {
      // runs that are not neighbours: lanes 4 i .. 4 i + 3 get the scale of group i, then each run its group's
      float ma = max3(fabsf(x[0]), x[1], x[2]), mb = max3(fabsf(y[0]), y[1], y[2]);
      ma = fmaxf(ma, fabsf(x[3])), mb = fmaxf(mb, fabsf(y[3]));
      const int r = a.rot / 8;  // lanes that turn; runs 0 .. r - 1 are their first, r .. 2 r - 1 their second
      const int u = 2 * l, s0 = u < r ? u : u < 2 * r ? u - r : l, s1 = u + 1 < r ? u + 1 : u + 1 < 2 * r ? u + 1 - r : l;
      const float a0 = __shfl_sync(0xffffffffu, ma, s0, kLanes), b0 = __shfl_sync(0xffffffffu, mb, s0, kLanes);
      const float a1 = __shfl_sync(0xffffffffu, ma, s1, kLanes), b1 = __shfl_sync(0xffffffffu, mb, s1, kLanes);
      ma = u < r ? a0 : u < 2 * r ? b0 : ma;
      mb = u + 1 < r ? a1 : u + 1 < 2 * r ? b1 : mb;
      float m = fmaxf(ma, mb);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const float s = group_scale(m);
      const float sa = __shfl_sync(0xffffffffu, s, qa / 32 * 4, kLanes), sb = __shfl_sync(0xffffffffu, s, qb / 32 * 4, kLanes);
      const uint32_t ca = nibbles<4>(x, sa), cb = nibbles<4>(y, sb);
      if (h < a.Hkv) {
        uint8_t* const p = static_cast<uint8_t*>(pages) + row * (D / 2);
        *reinterpret_cast<uint16_t*>(p + qa / 2) = static_cast<uint16_t>(ca);
        *reinterpret_cast<uint16_t*>(p + qb / 2) = static_cast<uint16_t>(cb);
        if (l % 4 == 0) static_cast<uint16_t*>(scales)[row * (D / 32) + l / 4] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
      }
    }
  };
  // 4 bits, a lane's eight values in a row: four lanes a group
  [[maybe_unused]] auto store_eight = [&](void* pages, void* scales, int h, const float (&x)[4], const float (&y)[4]) {
    const int64_t row = row0 + static_cast<int64_t>(h) * a.page;
    float m = max3(max3(max3(fabsf(x[0]), x[1], x[2]), x[3], y[0]), y[1], y[2]);
    m = fmaxf(m, fabsf(y[3]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float s = group_scale(m);
    const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    const uint32_t c = nibbles<8>(z, s);
    if (h < a.Hkv) {
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(pages) + row * (D / 2) + 4 * l) = c;
      if (l % 4 == 0) static_cast<uint16_t*>(scales)[row * (D / 32) + l / 4] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
    }
  };
  const int ka = max(g0 - gq, 0), kb = min(g1 - gq, gk);
  if (ka < kb)
    stream(static_cast<const T*>(a.k) + tok * a.k_stride, ka, kb, a.Hkv, ea, eb, make_angles,
           [&](int h, float (&x)[4], float (&y)[4]) {
             rotate(x, y);
             if constexpr (kBits == 4) {
               if (a.k_mean) {
                 const float* mean = a.k_mean + min(h, a.Hkv - 1) * D;
                 const float4 u = *reinterpret_cast<const float4*>(mean + ea), w = *reinterpret_cast<const float4*>(mean + eb);
                 x[0] -= u.x, x[1] -= u.y, x[2] -= u.z, x[3] -= u.w;
                 y[0] -= w.x, y[1] -= w.y, y[2] -= w.z, y[3] -= w.w;
               }
             }
             if constexpr (kBits == 4 && kAdjacent) store_eight(a.k_pages, a.k_scale, h, x, y);
             else store_codes(a.k_pages, a.k_scale, h, ea, eb, x, y);
           });
  const int va = max(g0 - gq - gk, 0), vb = g1 - gq - gk;
  if (va < vb)
    stream(static_cast<const T*>(a.v) + tok * a.v_stride, va, vb, a.Hkv, kBits == 4 ? 8 * l : ea, kBits == 4 ? 8 * l + 4 : eb,
           [] {}, [&](int h, float (&x)[4], float (&y)[4]) {
             if constexpr (kBits == 4) store_eight(a.v_pages, a.v_scale, h, x, y);
             else store_codes(a.v_pages, a.v_scale, h, ea, eb, x, y);
           });
}

template <typename T, int D, int kBits>
cudaError_t launch_append_td(const AppendArgs& a, bool adjacent, unsigned grid, cudaStream_t s) {
  if (adjacent) rope_append_kernel<T, D, true, kBits><<<grid, 128, 0, s>>>(a, device_status_ptr());
  else rope_append_kernel<T, D, false, kBits><<<grid, 128, 0, s>>>(a, device_status_ptr());
  return cudaGetLastError();
}
template <typename T, int kBits>
cudaError_t launch_append_t(const AppendArgs& a, int32_t d, bool adjacent, unsigned grid, cudaStream_t s) {
  switch (d) {
    case 32: return launch_append_td<T, 32, kBits>(a, adjacent, grid, s);
    case 64: return launch_append_td<T, 64, kBits>(a, adjacent, grid, s);
    case 128: return launch_append_td<T, 128, kBits>(a, adjacent, grid, s);
    case 256: return launch_append_td<T, 256, kBits>(a, adjacent, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int kBits>
cudaError_t launch_append(const RopeAppendArgs& r, cudaStream_t s) {
  AppendArgs a{};
  a.q = r.q;
  a.k = r.k;
  a.v = r.v;
  a.q_stride = r.q_stride;
  a.k_stride = r.k_stride;
  a.v_stride = r.v_stride;
  a.q_out_stride = r.q_out_stride;
  a.T = r.T;
  a.Hq = r.Hq;
  a.Hkv = r.Hkv;
  a.positions = r.positions;
  a.axes = r.axes;
  a.rot = r.rot_dim;
  a.inv_freq = r.inv_freq;
  a.q_out = r.q_out;
  a.slot_map = r.slot_map;
  a.k_pages = r.k_pages;
  a.v_pages = r.v_pages;
  a.k_scale = r.k_scale;
  a.v_scale = r.v_scale;
  a.k_mean = r.k_mean;
  a.num_pages = r.num_pages;
  a.page = r.page_size;
  if (r.pair_axis)
    for (int i = 0; i < r.rot_dim / 2; ++i) a.axis[i] = r.pair_axis[i];
  // one warp per token once that fills the device (about 32 warps an SM); below, a token's
  // rows are cut into parts, whose warps each compute the angles again
  const int32_t rows_at_once = 256 / r.d;
  const int32_t groups = (r.Hq + rows_at_once - 1) / rows_at_once + 2 * ((r.Hkv + rows_at_once - 1) / rows_at_once);
  const int64_t fill = 32ll * num_sms();
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(groups, fill / r.T));
  a.iters = static_cast<int32_t>((groups + parts - 1) / parts);
  a.parts = (groups + a.iters - 1) / a.iters;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(r.T) * a.parts + 3) / 4);
  switch (r.dtype) {
    case SL8_F16: return launch_append_t<__half, kBits>(a, r.d, r.adjacent, grid, s);
    case SL8_BF16: return launch_append_t<__nv_bfloat16, kBits>(a, r.d, r.adjacent, grid, s);
    case SL8_F32: return launch_append_t<float, kBits>(a, r.d, r.adjacent, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

}  // namespace sl8
