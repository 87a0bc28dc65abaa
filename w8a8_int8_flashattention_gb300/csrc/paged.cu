// The paged int8 cache's bookkeeping and writes, for sm_103a: the page plan of a serving
// step (block tables, slot map and free list from request lengths), rotary positions
// fused with the int8 append, and the per-page key bounds that the page selection scores.
//
// The "SuperL8" README (github.com/jajmangold/superl8) lists the paged int8 KV cache
// ("Engine" table, "Paged KV cache" row) and the kernels that read it; the writes, their
// layouts and formulas are readings, stated with each kernel.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sl8_internal.h"

namespace cg = cooperative_groups;

namespace sl8 {

namespace {

// ---------------------------------------------------------------- page plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;

// Exclusive prefix over the block of a pair of 64-bit counts; totals in ta, tb.
__device__ __forceinline__ void block_prefix2(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb, int64_t* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += xa;
      ib += xb;
    }
  }
  if (lane == 31) {
    sm[warp] = ia;
    sm[32 + warp] = ib;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t wa = sm[lane], wb = sm[32 + lane];
    const int64_t a0 = wa, b0 = wb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t xa = __shfl_up_sync(0xffffffffu, wa, o), xb = __shfl_up_sync(0xffffffffu, wb, o);
      if (lane >= o) {
        wa += xa;
        wb += xb;
      }
    }
    sm[lane] = wa - a0;
    sm[32 + lane] = wb - b0;
    if (lane == 31) {
      sm[64] = wa;
      sm[65] = wb;
    }
  }
  __syncthreads();
  const int64_t ea = sm[warp] + ia - a, eb = sm[32 + warp] + ib - b;
  ta = sm[64];
  tb = sm[65];
  __syncthreads();
  a = ea;
  b = eb;
}

// Largest i in [0, n) with p[i] <= x (p nondecreasing, p[0] <= x).
__device__ __forceinline__ int find_owner(const int64_t* p, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct PlanArgs {
  const int32_t* ctx;
  const int32_t* add;
  const int32_t* release;  // nullable
  int32_t B, page, max_blocks;
  int32_t* table;
  int32_t* free_pages;
  int32_t free_cap;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t max_tokens;
  int32_t *seqlens, *granted, *cu_new, *slot_map, *token_pos;
};

struct PlanSmem {
  int64_t cu[kPlanThreads + 1];    // tokens before each request of the block of requests
  int64_t need[kPlanThreads + 1];  // pages (pushed or taken) before each
  int32_t ctx[kPlanThreads];       // length that stays (0 for a released slot)
  int32_t ok[kPlanThreads];
  int64_t scan[66];
};

// One cluster plans the step, in two passes over blocks of kPlanThreads requests; every CTA
// scans each block's counts itself and then takes its share of the block's pages and
// tokens, found by binary search in the scanned prefixes.  Pass 1 pushes the pages of the
// released slots; pass 2 grants requests in order, writes the new table entries and maps
// the tokens.  A token's page is read from the table for a block the request had before
// and straight from the free list for a new one, so no CTA waits for another's table
// writes.  The cluster barriers order pass 1's pushes and table reads before pass 2, and
// each block's length reads before the writes that may alias them (in-place lengths).
// Latency-bound: the bytes are 8 per token and 8 per moved page.
__global__ void __launch_bounds__(kPlanThreads, 1) paged_assign_kernel(const PlanArgs a, DeviceStatus* st) {
  __shared__ PlanSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x), tid = threadIdx.x;
  const int first = rank * kPlanThreads + tid, step = ranks * kPlanThreads;
  const int64_t cap = static_cast<int64_t>(a.max_blocks) * a.page;
  int64_t have = *a.free_count;
  if (have < 0 || have > a.free_cap) {
    if (first == 0) record_status(st, kStatusBadArg, 800);
    have = have < 0 ? 0 : a.free_cap;
  }
  if (a.release) {
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
      const int n = min(kPlanThreads, a.B - b0);
      int64_t pages = 0, zero = 0, total, unused;
      if (tid < n && a.release[b0 + tid] != 0) {
        const int32_t c = a.ctx[b0 + tid];
        if (c < 0 || c > cap) {
          if (rank == 0) record_status(st, kStatusBadArg, 801);
        } else {
          pages = (static_cast<int64_t>(c) + a.page - 1) / a.page;
        }
      }
      block_prefix2(pages, zero, total, unused, sm.scan);
      sm.need[tid] = pages;
      __syncthreads();
      for (int64_t e = first; e < total; e += step) {
        const int i = find_owner(sm.need, n, e);
        const int64_t dst = have + e;
        if (dst < a.free_cap) a.free_pages[dst] = a.table[static_cast<int64_t>(b0 + i) * a.max_blocks + (e - sm.need[i])];
      }
      have += total;
      if (have > a.free_cap) {
        if (first == 0) record_status(st, kStatusBadArg, 802);
        have = a.free_cap;
      }
      __syncthreads();
    }
  }
  if (ranks > 1) cluster.sync();
  else __syncthreads();
  int64_t cu0 = 0, need0 = 0, taken = 0;  // sums over the blocks of requests before this one
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int n = min(kPlanThreads, a.B - b0);
    const int b = b0 + tid;
    int32_t c = 0;
    int64_t tokens = 0, own = 0;
    bool valid = false;
    if (tid < n) {
      c = a.release && a.release[b] != 0 ? 0 : a.ctx[b];
      const int32_t add = a.add[b];
      valid = c >= 0 && c <= cap && add >= 0;
      if (!valid && rank == 0) record_status(st, kStatusBadArg, 803);
      c = c < 0 ? 0 : (c > cap ? static_cast<int32_t>(cap) : c);
      if (valid) tokens = add;
    }
    int64_t cu = tokens, zero = 0, cu_total, unused;
    block_prefix2(cu, zero, cu_total, unused, sm.scan);
    // a request that cannot fit (its table row, the step's tokens) asks for no page
    bool ok = valid && c + tokens <= cap && cu0 + cu + tokens <= a.max_tokens;
    const int32_t held = (c + a.page - 1) / a.page;
    if (ok) own = (c + tokens + a.page - 1) / a.page - held;
    int64_t before = own, need_total;
    zero = 0;
    block_prefix2(before, zero, need_total, unused, sm.scan);
    ok = ok && (own == 0 || need0 + before + own <= have);
    sm.cu[tid] = cu0 + cu;
    sm.need[tid] = need0 + before;
    sm.ctx[tid] = c;
    sm.ok[tid] = ok;
    const int64_t mine = ok ? own : 0;
    int64_t got = mine, got_total;
    zero = 0;
    block_prefix2(got, zero, got_total, unused, sm.scan);
    if (tid == 0) {
      sm.cu[n] = cu0 + cu_total;
      sm.need[n] = need0 + need_total;
    }
    // every CTA has read this block's lengths: the outputs may be the same buffers
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    if (rank == 0 && tid < n) {
      a.seqlens[b] = c + (ok ? static_cast<int32_t>(tokens) : 0);
      a.granted[b] = ok ? static_cast<int32_t>(tokens) : 0;
      const int64_t at = cu0 + cu;
      a.cu_new[b] = static_cast<int32_t>(at < 0x7fffffff ? at : 0x7fffffff);
    }
    // granted requests that need pages are a prefix of those that do, so their pages are
    // the got_total entries below have - need0
    for (int64_t e = first; e < got_total; e += step) {
      const int i = find_owner(sm.need, n, need0 + e);
      const int64_t blk = (sm.ctx[i] + a.page - 1) / a.page + (need0 + e - sm.need[i]);
      a.table[static_cast<int64_t>(b0 + i) * a.max_blocks + blk] = a.free_pages[have - 1 - (need0 + e)];
    }
    const int64_t t1 = min(cu0 + cu_total, static_cast<int64_t>(a.max_tokens));
    for (int64_t t = cu0 + first; t < t1; t += step) {
      const int i = find_owner(sm.cu, n, t);
      const int32_t pos = static_cast<int32_t>(min(sm.ctx[i] + (t - sm.cu[i]), static_cast<int64_t>(0x7fffffff)));
      int32_t slot = -1;
      if (sm.ok[i]) {
        const int32_t blk = pos / a.page, nb = (sm.ctx[i] + a.page - 1) / a.page;
        const int32_t pg = blk < nb ? a.table[static_cast<int64_t>(b0 + i) * a.max_blocks + blk]
                                    : a.free_pages[have - 1 - (sm.need[i] + blk - nb)];
        slot = pg * a.page + (pos - blk * a.page);
      }
      a.slot_map[t] = slot;
      if (a.token_pos) a.token_pos[t] = pos;
    }
    cu0 += cu_total;
    need0 += need_total;
    taken += got_total;
    __syncthreads();
  }
  // padding past the last token
  for (int64_t t = min(cu0, static_cast<int64_t>(a.max_tokens)) + first; t < a.max_tokens; t += step) {
    a.slot_map[t] = -1;
    if (a.token_pos) a.token_pos[t] = 0;
  }
  // every CTA has read free_count (before the barriers above): it may be free_count_out
  if (first == 0) {
    a.cu_new[a.B] = static_cast<int32_t>(cu0 < 0x7fffffff ? cu0 : 0x7fffffff);
    *a.free_count_out = static_cast<int32_t>(have - taken);
  }
}

// ---------------------------------------------------------------- rotary append
struct AppendArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements from token to token
  int32_t T, Hq, Hkv;
  const int32_t* positions;  // [axes][T]
  int32_t axes, rot;
  const float* inv_freq;     // [rot / 2]
  void* q_out;
  const int32_t* slot_map;   // [T]
  int8_t *k_pages, *v_pages;
  float *k_scale, *v_scale;
  int32_t num_pages, page;
  int32_t iters;             // row groups of a token that one warp handles
  int32_t parts;             // warps per token
  uint8_t axis[128];         // axis of each rotary pair
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
template <>
__device__ __forceinline__ void load4<__half>(const __half* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
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
// 24-bit mantissa of f times 2^64 / (2 pi), shifted by f's exponent (frequencies below
// 2^-41 count as 0).  Times an int32 position, mod 2^64, the top 32 bits are the turns of
// the position's angle to 2^-32 at any position, where a product in fp32 would lose
// 0.06 rad at position 2^20; whole turns drop out by themselves.
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
// registers, and no lane exchanges values but the row maximum.  HBM-bound: q, k and v are
// read once, q is written once and k, v as codes.
template <typename T, int D, bool kAdjacent>
__global__ void __launch_bounds__(256) rope_append_kernel(const AppendArgs a, DeviceStatus* st) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t tok = w / a.parts;
  if (tok >= a.T) return;
  const int part = static_cast<int>(w - tok * a.parts);
  const int l = lane % kLanes, sub = lane / kLanes;
  const bool turned = 8 * l < a.rot;
  const int ea = !kAdjacent && turned ? 4 * l : 8 * l;
  const int eb = !kAdjacent && turned ? a.rot / 2 + 4 * l : 8 * l + 4;
  float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int rows = a.Hq + 2 * a.Hkv;
  const int r_begin = part * a.iters * kRows, r_end = min(rows, r_begin + a.iters * kRows);
  if (turned && r_begin < a.Hq + a.Hkv) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = 4 * l + i;
      turn(a.positions[static_cast<int64_t>(a.axis[p]) * a.T + tok], turns_of(a.inv_freq[p]), c[i], s[i]);
    }
  }
  const int32_t slot = a.slot_map[tok];
  bool keep = slot >= 0;
  int64_t row0 = 0;  // the slot's row in the first head of its page
  if (keep) {
    const int32_t pg = slot / a.page;
    if (pg >= a.num_pages) {
      if (lane == 0 && part == 0) record_status(st, kStatusBadArg, 810);
      keep = false;
    } else {
      row0 = static_cast<int64_t>(pg) * a.Hkv * a.page + slot % a.page;
    }
  }
  for (int r0 = r_begin; r0 < r_end; r0 += kRows) {
    const int r = r0 + sub;
    const bool live = r < r_end;
    const bool is_q = r < a.Hq, is_k = !is_q && r < a.Hq + a.Hkv;
    const int h = is_q ? r : (is_k ? r - a.Hq : r - a.Hq - a.Hkv);
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live && (is_q || keep)) {
      const T* src = static_cast<const T*>(is_q ? a.q : (is_k ? a.k : a.v)) +
                     tok * (is_q ? a.q_stride : (is_k ? a.k_stride : a.v_stride)) + static_cast<int64_t>(h) * D;
      load4<T>(src + ea, x);
      load4<T>(src + eb, y);
    }
    if (turned && (is_q || is_k)) {
      if constexpr (kAdjacent) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
          x[2 * i] = fmaf(x0, c[i], -(x1 * s[i]));
          x[2 * i + 1] = fmaf(x1, c[i], x0 * s[i]);
          y[2 * i] = fmaf(y0, c[i + 2], -(y1 * s[i + 2]));
          y[2 * i + 1] = fmaf(y1, c[i + 2], y0 * s[i + 2]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = x[i], y0 = y[i];
          x[i] = fmaf(x0, c[i], -(y0 * s[i]));
          y[i] = fmaf(y0, c[i], x0 * s[i]);
        }
      }
    }
    if (live && is_q) {
      T* dst = static_cast<T*>(a.q_out) + tok * a.q_out_stride + static_cast<int64_t>(h) * D;
      store4<T>(dst + ea, x);
      store4<T>(dst + eb, y);
    }
    if (r0 + kRows <= a.Hq || !keep) continue;  // uniform: the warp's rows are all q rows, or nothing is stored
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(x[i]), fabsf(y[i])));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float sc = __fdiv_rn(m, 127.0f);
    if (!live || is_q) continue;
    uint32_t ca = 0, cb = 0;
    if (sc != 0.0f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = max(-127, min(127, __float2int_rn(__fdiv_rn(x[i], sc))));
        const int q = max(-127, min(127, __float2int_rn(__fdiv_rn(y[i], sc))));
        ca |= static_cast<uint32_t>(p & 0xff) << (8 * i);
        cb |= static_cast<uint32_t>(q & 0xff) << (8 * i);
      }
    }
    const int64_t row = row0 + static_cast<int64_t>(h) * a.page;
    int8_t* dst = (is_k ? a.k_pages : a.v_pages) + row * D;
    *reinterpret_cast<uint32_t*>(dst + ea) = ca;
    *reinterpret_cast<uint32_t*>(dst + eb) = cb;
    if (l == 0) (is_k ? a.k_scale : a.v_scale)[row] = sc;
  }
}

// ---------------------------------------------------------------- page bounds
struct BoundsArgs {
  const int8_t* k_pages;
  const float* k_scale;
  int32_t num_pages, page;
  const int32_t* table;
  int32_t max_blocks;
  const int32_t* seqlens;
  const int32_t* add;  // nullable: every block
  int32_t max_new, per_seq, B, Hkv;
  int8_t* bounds;
  float* scale;
};

// Per-channel bounds of a page's keys.  With S the largest row scale among the page's
// valid rows, row t's keys are code * (s_t / S) in steps of S; the bounds are the floor
// of the least and the ceiling of the largest, so lo S <= k <= hi S holds for every key
// (up to the rounding of s_t / S and of the product).  A warp per (page, kv head): D / 16
// lanes hold a row, 16 channels each, and the rows run over the remaining lanes.
// HBM-bound on the codes, which the append has just left in L2.
template <int D>
__global__ void __launch_bounds__(256) page_bounds_kernel(const BoundsArgs a, DeviceStatus* st) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int h = static_cast<int>(w % a.Hkv);
  const int64_t u = w / a.Hkv;
  const int b = static_cast<int>(u / a.per_seq), i = static_cast<int>(u - static_cast<int64_t>(b) * a.per_seq);
  if (b >= a.B) return;
  const int64_t cap = static_cast<int64_t>(a.max_blocks) * a.page;
  int64_t L = a.seqlens[b];
  bool bad = L < 0 || L > cap;
  L = L < 0 ? 0 : (L > cap ? cap : L);
  int64_t add = L;
  if (a.add) {
    add = a.add[b];
    bad = bad || add < 0 || add > L || add > a.max_new;
    add = add < 0 ? 0 : (add > L ? L : add);
    if (add > a.max_new) add = a.max_new;
  }
  if (bad && i == 0 && h == 0 && lane == 0) record_status(st, kStatusBadArg, 820);
  const int64_t blk = (L - add) / a.page + i;
  if (add == 0 || blk * a.page >= L) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(a.page), L - blk * a.page));
  int32_t pg = a.table[static_cast<int64_t>(b) * a.max_blocks + blk];
  if (pg < 0 || pg >= a.num_pages) {
    if (lane == 0) record_status(st, kStatusBadArg, 821);
    return;
  }
  const int64_t ph = static_cast<int64_t>(pg) * a.Hkv + h;
  const int8_t* codes = a.k_pages + ph * a.page * D;
  const float* ks = a.k_scale + ph * a.page;
  float S = 0.0f;
  for (int t = lane; t < n; t += 32) S = fmaxf(S, ks[t]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) S = fmaxf(S, __shfl_xor_sync(0xffffffffu, S, o));
  const int l = lane % kLanes;
  float lo[16], hi[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    lo[e] = INFINITY;
    hi[e] = -INFINITY;
  }
#pragma unroll 2
  for (int t = lane / kLanes; t < n; t += kRows) {
    const uint4 v = *reinterpret_cast<const uint4*>(codes + static_cast<int64_t>(t) * D + 16 * l);
    const float f = S == 0.0f ? 0.0f : __fdiv_rn(ks[t], S);
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float y = static_cast<float>(static_cast<int8_t>(x[e / 4] >> (8 * (e % 4)))) * f;
      lo[e] = fminf(lo[e], y);
      hi[e] = fmaxf(hi[e], y);
    }
  }
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
      hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
    }
  }
  if (lane < kLanes) {
    uint32_t a4[4] = {0, 0, 0, 0}, b4[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      a4[e / 4] |= static_cast<uint32_t>(static_cast<int>(floorf(lo[e])) & 0xff) << (8 * (e % 4));
      b4[e / 4] |= static_cast<uint32_t>(static_cast<int>(ceilf(hi[e])) & 0xff) << (8 * (e % 4));
    }
    int8_t* dst = a.bounds + ph * 2 * D + 16 * l;
    *reinterpret_cast<uint4*>(dst) = make_uint4(a4[0], a4[1], a4[2], a4[3]);
    *reinterpret_cast<uint4*>(dst + D) = make_uint4(b4[0], b4[1], b4[2], b4[3]);
    if (lane == 0) a.scale[ph] = S;
  }
}

template <typename T, int D>
cudaError_t launch_append_td(const AppendArgs& a, bool adjacent, unsigned grid, cudaStream_t s) {
  if (adjacent) rope_append_kernel<T, D, true><<<grid, 256, 0, s>>>(a, device_status_ptr());
  else rope_append_kernel<T, D, false><<<grid, 256, 0, s>>>(a, device_status_ptr());
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_append_t(const AppendArgs& a, int32_t d, bool adjacent, unsigned grid, cudaStream_t s) {
  switch (d) {
    case 32: return launch_append_td<T, 32>(a, adjacent, grid, s);
    case 64: return launch_append_td<T, 64>(a, adjacent, grid, s);
    case 128: return launch_append_td<T, 128>(a, adjacent, grid, s);
    case 256: return launch_append_td<T, 256>(a, adjacent, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_paged_assign(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* release, int32_t B,
                                int32_t page_size, int32_t max_blocks, int32_t* block_table, int32_t* free_pages,
                                int32_t free_capacity, const int32_t* free_count, int32_t* free_count_out,
                                int32_t max_tokens, int32_t* seqlens, int32_t* granted, int32_t* cu_new,
                                int32_t* slot_map, int32_t* token_pos, cudaStream_t s) {
  TraceScope tr("paged_assign", s);
  const PlanArgs a{ctx_lens, new_lens, release, B, page_size, max_blocks, block_table, free_pages, free_capacity,
                   free_count, free_count_out, max_tokens, seqlens, granted, cu_new, slot_map, token_pos};
  // one CTA where its threads cover the step's tokens a few times over: a cluster only
  // adds its barriers there
  const unsigned ranks = static_cast<int64_t>(max_tokens) + B <= 4 * kPlanThreads ? 1 : kPlanCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_assign_kernel, a, device_status_ptr());
}

cudaError_t launch_rope_append(const RopeAppendArgs& r, cudaStream_t s) {
  TraceScope tr("rope_append", s);
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
  a.num_pages = r.num_pages;
  a.page = r.page_size;
  if (r.pair_axis)
    for (int i = 0; i < r.rot_dim / 2; ++i) a.axis[i] = r.pair_axis[i];
  // one warp per token once that fills the device (about 32 warps an SM); below, a token's
  // rows are cut into parts, whose warps each compute the angles again
  const int32_t rows_at_once = 256 / r.d;
  const int32_t groups = (r.Hq + 2 * r.Hkv + rows_at_once - 1) / rows_at_once;
  const int64_t fill = 32ll * num_sms();
  int64_t iters = (static_cast<int64_t>(r.T) * groups + fill - 1) / fill;
  if (iters > groups) iters = groups;
  a.iters = static_cast<int32_t>(iters);
  a.parts = static_cast<int32_t>((groups + iters - 1) / iters);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(r.T) * a.parts + 7) / 8);
  switch (r.dtype) {
    case SL8_F16: return launch_append_t<__half>(a, r.d, r.adjacent, grid, s);
    case SL8_BF16: return launch_append_t<__nv_bfloat16>(a, r.d, r.adjacent, grid, s);
    case SL8_F32: return launch_append_t<float>(a, r.d, r.adjacent, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_page_bounds(const int8_t* k_pages, const float* k_scale_pages, int32_t num_pages, int32_t page_size,
                               const int32_t* block_table, int32_t max_blocks, const int32_t* seqlens,
                               const int32_t* new_lens, int32_t max_new, int32_t B, int32_t Hkv, int32_t d,
                               int8_t* bounds, float* bound_scale, cudaStream_t s) {
  TraceScope tr("page_bounds", s);
  // blocks that max_new tokens can touch: one more than they fill
  int64_t per_seq = new_lens ? (static_cast<int64_t>(max_new) + page_size - 2) / page_size + 1 : max_blocks;
  if (per_seq > max_blocks) per_seq = max_blocks;
  const BoundsArgs a{k_pages, k_scale_pages, num_pages, page_size, block_table, max_blocks, seqlens, new_lens, max_new,
                     static_cast<int32_t>(per_seq), B, Hkv, bounds, bound_scale};
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(B) * per_seq * Hkv + 7) / 8);
  switch (d) {
    case 32: page_bounds_kernel<32><<<grid, 256, 0, s>>>(a, device_status_ptr()); break;
    case 64: page_bounds_kernel<64><<<grid, 256, 0, s>>>(a, device_status_ptr()); break;
    case 128: page_bounds_kernel<128><<<grid, 256, 0, s>>>(a, device_status_ptr()); break;
    case 256: page_bounds_kernel<256><<<grid, 256, 0, s>>>(a, device_status_ptr()); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace sl8
