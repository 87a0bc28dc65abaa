// The paged 4-bit cache (rows as in cache4.cuh): the rotary append that fills it, and reading it
// back as dense keys and values, for sm_103a.
//
// The "SuperL8" READMEs (github.com/jajmangold/superl8) name 4-bit values in the paged cache
// ("Engine" table, k8v3; "Attention kernels" table, attn_decode's int4 V variant) without a
// layout; the one here is a reading.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "append.cuh"
#include "cache4.cuh"
#include "sl8_internal.h"

namespace sl8 {

namespace {

// Tokens of one (sequence, kv head) per CTA: a thread takes eight channels of kReadRows rows, 16 bytes a store.
constexpr int kReadRows = 4;
constexpr int read_tokens(int d) { return kReadRows * 256 / (d / 8); }

// (x & mask) | bits, the mask an immediate: as one operation.
__device__ __forceinline__ uint32_t lop3_and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
  return r;
}
// Eight values as one store, or two of fp32.
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) { return f16x2_of(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()), pack2(x[4], x[5], T()), pack2(x[6], x[7], T()));
}

// Codes of a word's eight nibbles, exact, as bf16: word i holds those of nibbles i and i + 4, the low bits of 128 + nibble.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&c)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t n = lop3_and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(c[i]) : "r"(n), "r"(0x3f803f80u), "r"(0xc308c308u));  // less 136
  }
}

// out = code * s (+ the mean that the append took off), one rounding to fp32 and one to the output's type.  Bound by HBM,
// 0.56 bytes in and 2 (4) out a value, and by issue next to it: all of a thread's loads are on their way at once (pages,
// then codes and scales, keys and values alike; 131,072 tokens of 8 heads at d = 128 137 us one row after another, 110 so),
// codes become bf16 numbers two at a time and meet their scales in mixed-precision fmas (107, and a packed batch of 8
// prefixes of 1,024 to 8,192 tokens 40.4 -> 38.9), and pages and rows are found from the row before (106, 0.95 of the copy
// rate; the batch 38.3, 0.74).  The sequences take turns in the grid: the CTAs of ragged ones that have no token come
// between others.
template <typename T, int D>
__global__ void __launch_bounds__(256) read4_kernel(const Read4Args a, DeviceStatus* st) {
  constexpr int kLanes = D / 8, kRows = 256 / kLanes, kTok = read_tokens(D);
  const uint32_t u = blockIdx.x / static_cast<uint32_t>(a.Hkv), h = blockIdx.x - u * a.Hkv;
  const uint32_t chunk = u / static_cast<uint32_t>(a.B), b = u - chunk * a.B;
  const int first = static_cast<int>(chunk) * kTok;
  const int l = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int32_t cap = a.max_blocks * a.page;
  int64_t L = a.seqlens[b], room = min(cap, a.N), at = static_cast<int64_t>(b) * a.Hkv * a.N;
  bool bad = L < 0;
  if (a.cu_seqlens) {
    at = a.cu_seqlens[b];
    const int64_t end = min(static_cast<int64_t>(a.cu_seqlens[b + 1]), a.total);
    if (at < 0) bad = true, at = 0, room = 0;
    room = min(room, end - at);
  }
  if (L > room) bad = true, L = room;
  if (bad && first == 0 && h == 0 && threadIdx.x == 0) record_status(st, kStatusBadArg, 860);
  const int n = static_cast<int>(min(L, static_cast<int64_t>(first) + kTok));
  if (first >= n) return;
  int32_t pg[kReadRows], off[kReadRows];
  const int32_t* const table = a.table + static_cast<int64_t>(b) * a.max_blocks;
  const int mine = first + sub;
  int blk = min(mine, n - 1) / a.page, in = min(mine, n - 1) - blk * a.page;
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {  // rows past the last one repeat another and store nothing
    if (i > 0 && mine + i * kRows < n) {
      in += kRows;
      if (in >= a.page) {
        const int k = in / a.page;
        blk += k;
        in -= k * a.page;
      }
    }
    pg[i] = table[blk];
    off[i] = in;
  }
  uint32_t w[2][kReadRows];
  uint16_t s[2][kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (pg[i] < 0 || pg[i] >= a.num_pages) {
      record_status(st, kStatusBadArg, 861);
      pg[i] = 0;
    }
    const int64_t row = (static_cast<int64_t>(pg[i]) * a.Hkv + h) * a.page + off[i];
    if (a.k_out) {
      w[0][i] = *reinterpret_cast<const uint32_t*>(a.k_pages + row * (D / 2) + 4 * l);
      s[0][i] = a.k_scale[row * (D / 32) + l / 4];
    }
    if (a.v_out) {
      w[1][i] = *reinterpret_cast<const uint32_t*>(a.v_pages + row * (D / 2) + 4 * l);
      s[1][i] = a.v_scale[row * (D / 32) + l / 4];
    }
  }
  float mean[8] = {};
  if (a.k_mean) {
    const float4* m = reinterpret_cast<const float4*>(a.k_mean + h * D + 8 * l);
    const float4 x = m[0], y = m[1];
    mean[0] = x.x, mean[1] = x.y, mean[2] = x.z, mean[3] = x.w;
    mean[4] = y.x, mean[5] = y.y, mean[6] = y.z, mean[7] = y.w;
  }
  const int64_t step = static_cast<int64_t>(kRows) * D * (a.cu_seqlens ? a.Hkv : 1);
  const int64_t dst = (a.cu_seqlens ? (at + mine) * a.Hkv + h : at + static_cast<int64_t>(h) * a.N + mine) * D + 8 * l;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    T* const out = static_cast<T*>(kv ? a.v_out : a.k_out) + dst;
    if (!(kv ? a.v_out : a.k_out)) continue;
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      if (mine + i * kRows >= n) break;
      const uint32_t f = s[kv][i];
      uint32_t c[4];
      codes8(w[kv][i], c);
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = fma_mixed<0, 0>(c[e], f, kv == 0 ? mean[e] : 0.0f);
        x[e + 4] = fma_mixed<1, 0>(c[e], f, kv == 0 ? mean[e + 4] : 0.0f);
      }
      store8(out + i * step, x);
    }
  }
}

template <typename T>
cudaError_t launch_read_t(const Read4Args& a, int32_t d, unsigned grid, cudaStream_t s) {
  switch (d) {
    case 32: read4_kernel<T, 32><<<grid, 256, 0, s>>>(a, device_status_ptr()); break;
    case 64: read4_kernel<T, 64><<<grid, 256, 0, s>>>(a, device_status_ptr()); break;
    case 128: read4_kernel<T, 128><<<grid, 256, 0, s>>>(a, device_status_ptr()); break;
    case 256: read4_kernel<T, 256><<<grid, 256, 0, s>>>(a, device_status_ptr()); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append_int4(const RopeAppendArgs& r, cudaStream_t s) {
  TraceScope tr("rope_append_int4", s);
  return launch_append<4>(r, s);
}

cudaError_t launch_paged_read_int4(const Read4Args& a, int32_t d, cudaStream_t s) {
  TraceScope tr("paged_read_int4", s);
  const int64_t chunks = (static_cast<int64_t>(a.N) + read_tokens(d) - 1) / read_tokens(d);
  const unsigned grid = static_cast<unsigned>(chunks * a.B * a.Hkv);
  switch (a.out_dtype) {
    case SL8_F16: return launch_read_t<__half>(a, d, grid, s);
    case SL8_BF16: return launch_read_t<__nv_bfloat16>(a, d, grid, s);
    case SL8_F32: return launch_read_t<float>(a, d, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sl8
