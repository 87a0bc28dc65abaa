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

constexpr int kReadTok = 64;  // tokens of one (sequence, kv head) per CTA

// Eight values as one store, or two of fp32.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
  store4<T>(p, a);
  store4<T>(p + 4, b);
}

// out = code * s (+ the mean that the append took off), one rounding.
template <typename T, int D>
__global__ void __launch_bounds__(256) read4_kernel(const Read4Args a, DeviceStatus* st) {
  constexpr int kLanes = D / 8, kRows = 256 / kLanes;  // eight channels a thread
  const uint32_t u = blockIdx.x / static_cast<uint32_t>(a.Hkv), h = blockIdx.x - u * a.Hkv;
  const uint32_t chunks = (static_cast<uint32_t>(a.N) + kReadTok - 1) / kReadTok;
  const uint32_t b = u / chunks;
  const int first = static_cast<int>(u - b * chunks) * kReadTok;
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
  const int n = static_cast<int>(min(L, static_cast<int64_t>(first) + kReadTok));
  float mean[8] = {};
  if (a.k_mean) {
    const float4* m = reinterpret_cast<const float4*>(a.k_mean + h * D + 8 * l);
    const float4 x = m[0], y = m[1];
    mean[0] = x.x, mean[1] = x.y, mean[2] = x.z, mean[3] = x.w;
    mean[4] = y.x, mean[5] = y.y, mean[6] = y.z, mean[7] = y.w;
  }
  for (int t = first + sub; t < n; t += kRows) {
    int32_t pg = a.table[static_cast<int64_t>(b) * a.max_blocks + t / a.page];
    if (pg < 0 || pg >= a.num_pages) {
      record_status(st, kStatusBadArg, 861);
      pg = 0;
    }
    const int64_t row = (static_cast<int64_t>(pg) * a.Hkv + h) * a.page + t % a.page;
    const int64_t dst = (a.cu_seqlens ? (at + t) * a.Hkv + h : at + static_cast<int64_t>(h) * a.N + t) * D + 8 * l;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      T* const out = static_cast<T*>(kv ? a.v_out : a.k_out);
      if (!out) continue;
      const uint32_t w = *reinterpret_cast<const uint32_t*>((kv ? a.v_pages : a.k_pages) + row * (D / 2) + 4 * l);
      const float s = __uint_as_float(static_cast<uint32_t>((kv ? a.v_scale : a.k_scale)[row * (D / 32) + l / 4]) << 16);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = static_cast<float>(static_cast<int>((w >> (4 * i)) & 15u) - 8);
        x[i] = kv == 0 ? fmaf(c, s, mean[i]) : c * s;
      }
      store8<T>(out + dst, x);
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
  const int64_t chunks = (static_cast<int64_t>(a.N) + kReadTok - 1) / kReadTok;
  const unsigned grid = static_cast<unsigned>(chunks * a.B * a.Hkv);
  switch (a.out_dtype) {
    case SL8_F16: return launch_read_t<__half>(a, d, grid, s);
    case SL8_BF16: return launch_read_t<__nv_bfloat16>(a, d, grid, s);
    case SL8_F32: return launch_read_t<float>(a, d, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sl8
