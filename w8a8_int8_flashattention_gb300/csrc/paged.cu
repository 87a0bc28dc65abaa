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

#include <algorithm>
#include <cstdint>

#include "decode_unit.cuh"
#include "sl8_internal.h"

namespace cg = cooperative_groups;

namespace sl8 {

namespace {

// ---------------------------------------------------------------- page plan
constexpr int kPlanCluster = 8;
constexpr int kMapRequests = 2048;  // requests whose token counts the mapping kernel holds in shared memory

// Exclusive prefix of a 64-bit count over the block; its sum in total.
template <int kT>
__device__ __forceinline__ int64_t block_prefix(int64_t x, int64_t& total, int64_t* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  // every warp scans the warp sums for itself
  constexpr int kW = kT / 32;
  int64_t w = sm[lane % kW];
#pragma unroll
  for (int o = 1; o < kW; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, kW - 1);
  const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return (warp > 0 ? before : 0) + incl - x;
}

// Largest i in [0, n) with p[i] <= x (p nondecreasing, p[0] <= x).
template <typename P>
__device__ __forceinline__ int find_owner(const P* p, int n, P x) {
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
  bool vec;  // slot_map and token_pos take 16-byte stores
  bool map;  // the plan maps the tokens too
  uint32_t num_ids;  // page ids whose slots all stay below 2^31
};

// Slots and positions of the tokens [t0, t1) of a step's packed order, which belong to n
// requests with cu[i] tokens before the i-th (counted from `base`): four tokens a search,
// from a multiple of four.  length(i, p) says how many tokens request i had before the step
// and whether it was granted; row(i) is its table row, with the new pages already entered.
// The tokens of a page whose slots do not fit an int32 get none.
template <typename P, typename Length, typename Row>
__device__ __forceinline__ void map_tokens(const PlanArgs& a, int64_t base, int64_t t0, int64_t t1, uint32_t first,
                                           uint32_t step, const P* cu, int n, Length length, Row row, DeviceStatus* st) {
  const uint32_t page = static_cast<uint32_t>(a.page);
  for (int64_t t4 = (t0 & ~int64_t(3)) + 4 * static_cast<int64_t>(first); t4 < t1; t4 += 4 * static_cast<int64_t>(step)) {
    int32_t slot[4], pos[4];
    int i = find_owner(cu, n, static_cast<P>((t4 > t0 ? t4 : t0) - base));
    uint32_t blk = 0, off = 0, p = 0;
    int32_t pg = -1;
    bool fresh = true, ok = false;  // fresh: the first token of the quad or of a request
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      slot[j] = pos[j] = -1;
      const int64_t t = t4 + j;
      if (t < t0 || t >= t1) continue;
      const P rel = static_cast<P>(t - base);
      while (i + 1 < n && cu[i + 1] <= rel) {
        ++i;
        fresh = true;
      }
      if (fresh) {
        int32_t had;
        ok = length(i, had);
        p = static_cast<uint32_t>(had) + static_cast<uint32_t>(rel - cu[i]);
        blk = p / page;
        off = p - blk * page;
      }
      pos[j] = static_cast<int32_t>(min(p, 0x7fffffffu));
      if (ok) {
        if (fresh || off == page) {
          if (!fresh) {
            ++blk;
            off = 0;
          }
          pg = row(i)[blk];
          if (static_cast<uint32_t>(pg) >= a.num_ids) {
            record_status(st, kStatusBadArg, 804);
            pg = -1;
          }
        }
        if (pg >= 0) slot[j] = pg * a.page + static_cast<int32_t>(off);
      }
      ++p;
      ++off;
      fresh = false;
    }
    if (a.vec && t4 >= t0 && t4 + 4 <= t1) {
      *reinterpret_cast<int4*>(a.slot_map + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.token_pos) *reinterpret_cast<int4*>(a.token_pos + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t4 + j;
        if (t < t0 || t >= t1) continue;
        a.slot_map[t] = slot[j];
        if (a.token_pos) a.token_pos[t] = pos[j];
      }
    }
  }
}
// Padding past the last token.
__device__ __forceinline__ void map_padding(const PlanArgs& a, int64_t t0, uint32_t first, uint32_t step) {
  for (int64_t t = t0 + first; t < a.max_tokens; t += step) {
    a.slot_map[t] = -1;
    if (a.token_pos) a.token_pos[t] = 0;
  }
}

// *to(e) = from(e) for e = first, first + step, .. below count, four on their way at once.
template <typename From, typename To>
__device__ __forceinline__ void move_pages(uint32_t count, uint32_t first, uint32_t step, From from, To to) {
  for (uint32_t e0 = first; e0 < count; e0 += 4 * step) {
    int32_t page[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e0 + j * step < count) page[j] = from(e0 + j * step);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e0 + j * step < count) *to(e0 + j * step) = page[j];
  }
}

template <int kT>
struct PlanSmem {
  // of each request of the block of requests, counted from the block's first (at most 2^31 - 1)
  uint32_t cu[kT + 1];    // tokens before it
  uint32_t need[kT + 1];  // pages (pushed or asked for) before it
  int32_t ctx[kT];        // length that stays (0 for a released slot)
  int32_t ok[kT];
  int64_t scan[32];
  uint32_t got;           // pages granted
};
__device__ __forceinline__ uint32_t clamp31(int64_t x) { return static_cast<uint32_t>(x < 0x7fffffff ? x : 0x7fffffff); }

// One cluster plans the step, in two passes over blocks of kT requests; every CTA scans each
// block's counts itself and then takes its share of the block's pages, found by binary
// search in the scanned prefixes.  Pass 1 pushes the pages of the released slots; pass 2
// grants requests in order, writes the new table entries and maps the tokens (a.map; else
// map_tokens_kernel does).  The cluster barriers order pass 1's pushes and table reads
// before pass 2, each block's length reads before the writes that may alias them (in-place
// lengths), and the table writes before the mapping that reads them.  Bound by the latency
// of its barriers and dependent loads: 12.0 us with the mapping for 256 requests, 254,000
// tokens and some 29,000 moved pages, whose bytes take 0.3.
template <int kT>
__global__ void __launch_bounds__(kT, 1) paged_assign_kernel(const PlanArgs a, DeviceStatus* st) {
  __shared__ PlanSmem<kT> sm;
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t ranks = gridDim.x, rank = blockIdx.x, tid = threadIdx.x;
  const uint32_t first = rank * kT + tid, step = ranks * kT;
  auto sync = [&] {
    if (ranks > 1) cluster.sync();
    else __syncthreads();
  };
  const int32_t cap = a.max_blocks * a.page;  // below 2^31
  const uint32_t page = static_cast<uint32_t>(a.page);
  // the first block's lengths come in with the count, for both passes
  int32_t rel0 = 0, ctx0 = 0, add0 = 0;
  if (tid < static_cast<uint32_t>(min(kT, a.B))) {
    rel0 = a.release ? a.release[tid] : 0;
    ctx0 = a.ctx[tid];
    add0 = a.add[tid];
  }
  int64_t have = *a.free_count;
  if (have < 0 || have > a.free_cap) {
    if (first == 0) record_status(st, kStatusBadArg, 800);
    have = have < 0 ? 0 : a.free_cap;
  }
  if (a.release) {
    for (int b0 = 0; b0 < a.B; b0 += kT) {
      const int n = min(kT, a.B - b0);
      int64_t pages = 0, total;
      if (tid < static_cast<uint32_t>(n) && (b0 == 0 ? rel0 : a.release[b0 + tid]) != 0) {
        const int32_t c = b0 == 0 ? ctx0 : a.ctx[b0 + tid];
        if (c < 0 || c > cap) {
          if (rank == 0) record_status(st, kStatusBadArg, 801);
        } else {
          pages = (static_cast<uint32_t>(c) + page - 1) / page;
        }
      }
      sm.need[tid] = clamp31(block_prefix<kT>(pages, total, sm.scan));
      __syncthreads();
      const int64_t room = a.free_cap - have;
      const uint32_t count = static_cast<uint32_t>(total < room ? total : room);
      move_pages(
          count, first, step,
          [&](uint32_t e) {
            const int i = find_owner(sm.need, n, e);
            return a.table[static_cast<int64_t>(b0 + i) * a.max_blocks + (e - sm.need[i])];
          },
          [&](uint32_t e) { return a.free_pages + have + e; });
      if (total > room && first == 0) record_status(st, kStatusBadArg, 802);
      have += count;
      __syncthreads();
    }
  }
  sync();
  int64_t cu0 = 0, need0 = 0, taken = 0;  // sums over the blocks of requests before this one
  for (int b0 = 0; b0 < a.B; b0 += kT) {
    const int n = min(kT, a.B - b0), b = b0 + static_cast<int>(tid);
    const bool live = tid < static_cast<uint32_t>(n);
    int32_t c = 0;
    int64_t tokens = 0, own = 0;
    bool valid = false;
    if (live) {
      const bool gone = a.release && (b0 == 0 ? rel0 : a.release[b]) != 0;
      c = b0 == 0 ? ctx0 : a.ctx[b];
      const int32_t add = b0 == 0 ? add0 : a.add[b];
      valid = c >= 0 && c <= cap && add >= 0;
      if (!valid && rank == 0) record_status(st, kStatusBadArg, 803);
      c = gone || c < 0 ? 0 : (c > cap ? cap : c);
      if (valid) tokens = add;
    }
    int64_t cu_total, need_total;
    const int64_t cu = block_prefix<kT>(tokens, cu_total, sm.scan);
    // a request that cannot fit (its table row, the step's tokens) asks for no page
    bool ok = valid && c + tokens <= cap && cu0 + cu + tokens <= a.max_tokens;
    const uint32_t held = (static_cast<uint32_t>(c) + page - 1) / page;
    if (ok) own = (static_cast<uint32_t>(c) + static_cast<uint32_t>(tokens) + page - 1) / page - held;
    if (tid == 0) sm.got = 0;
    const int64_t before = block_prefix<kT>(own, need_total, sm.scan);
    ok = ok && (own == 0 || need0 + before + own <= have);
    // granted requests that need pages are a prefix of those that do
    if (ok && own > 0) atomicMax(&sm.got, static_cast<uint32_t>(before + own));
    sm.cu[tid] = clamp31(cu);
    sm.need[tid] = clamp31(before);
    sm.ctx[tid] = c;
    sm.ok[tid] = ok;
    sync();  // every CTA has read this block's lengths: the outputs may be the same buffers
    if (rank == 0 && live) {
      a.seqlens[b] = c + (ok ? static_cast<int32_t>(tokens) : 0);
      a.granted[b] = ok ? static_cast<int32_t>(tokens) : 0;
      a.cu_new[b] = static_cast<int32_t>(clamp31(cu0 + cu));
    }
    // their pages are the `got` entries below `top` in the free list
    const int32_t* top = a.free_pages + (have - 1 - need0);
    const uint32_t got = sm.got;
    move_pages(
        got, first, step, [&](uint32_t e) { return top[-static_cast<int64_t>(e)]; },
        [&](uint32_t e) {
          const int i = find_owner(sm.need, n, e);
          const uint32_t blk = (static_cast<uint32_t>(sm.ctx[i]) + page - 1) / page + (e - sm.need[i]);
          return a.table + static_cast<int64_t>(b0 + i) * a.max_blocks + blk;
        });
    if (a.map) {
      sync();
      map_tokens(
          a, cu0, cu0, min(cu0 + cu_total, static_cast<int64_t>(a.max_tokens)), first, step, sm.cu, n,
          [&](int i, int32_t& had) {
            had = sm.ctx[i];
            return sm.ok[i] != 0;
          },
          [&](int i) { return a.table + static_cast<int64_t>(b0 + i) * a.max_blocks; }, st);
    }
    cu0 += cu_total;
    need0 += need_total;
    taken += got;
    __syncthreads();
  }
  if (a.map) map_padding(a, min(cu0, static_cast<int64_t>(a.max_tokens)), first, step);
  // every CTA has read free_count (before the barriers above): it may be free_count_out
  if (first == 0) {
    a.cu_new[a.B] = static_cast<int32_t>(clamp31(cu0));
    *a.free_count_out = static_cast<int32_t>(have - taken);
  }
}

// The slots and positions of a step with many tokens, from what the plan left: a request's
// length before the step is its length after it less what it was granted.
__global__ void __launch_bounds__(256) map_tokens_kernel(const PlanArgs a, DeviceStatus* st) {
  __shared__ int32_t held[kMapRequests];
  grid_dependency_wait();
  const bool fits = a.B <= kMapRequests;
  if (fits)
    for (int i = threadIdx.x; i < a.B; i += 256) held[i] = a.cu_new[i];
  __syncthreads();
  const int64_t t1 = min(a.cu_new[a.B], a.max_tokens);
  const uint32_t first = blockIdx.x * 256 + threadIdx.x, step = gridDim.x * 256;
  auto length = [&](int i, int32_t& had) {
    const int32_t got = a.granted[i];
    had = a.seqlens[i] - got;
    return got > 0;
  };
  auto row = [&](int i) { return a.table + static_cast<int64_t>(i) * a.max_blocks; };
  if (fits) map_tokens(a, 0, 0, t1, first, step, held, a.B, length, row, st);
  else map_tokens(a, 0, 0, t1, first, step, a.cu_new, a.B, length, row, st);
  map_padding(a, t1, first, step);
}

template <int kT>
cudaError_t launch_plan(const PlanArgs& a, unsigned ranks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_assign_kernel<kT>, a, device_status_ptr());
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
template <typename T, int D, bool kAdjacent>
__global__ void __launch_bounds__(128) rope_append_kernel(const AppendArgs a, DeviceStatus* st) {
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
  auto stream = [&](const T* src, int from, int to, int heads, auto first, auto work) {
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
    stream(static_cast<const T*>(a.q) + tok * a.q_stride, g0, min(g1, gq), a.Hq, make_angles,
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
  auto store_codes = [&](int8_t* pages, float* scales, int h, const float (&x)[4], const float (&y)[4]) {
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
      const int64_t row = row0 + static_cast<int64_t>(h) * a.page;
      *reinterpret_cast<uint32_t*>(pages + row * D + ea) = ca;
      *reinterpret_cast<uint32_t*>(pages + row * D + eb) = cb;
      if (l == 0) scales[row] = rs.s;
    }
  };
  const int ka = max(g0 - gq, 0), kb = min(g1 - gq, gk);
  if (ka < kb)
    stream(static_cast<const T*>(a.k) + tok * a.k_stride, ka, kb, a.Hkv, make_angles,
           [&](int h, float (&x)[4], float (&y)[4]) {
             rotate(x, y);
             store_codes(a.k_pages, a.k_scale, h, x, y);
           });
  const int va = max(g0 - gq - gk, 0), vb = g1 - gq - gk;
  if (va < vb)
    stream(static_cast<const T*>(a.v) + tok * a.v_stride, va, vb, a.Hkv, [] {},
           [&](int h, float (&x)[4], float (&y)[4]) { store_codes(a.v_pages, a.v_scale, h, x, y); });
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

// (y0, y1) = (y0 - 8388736, y1 - 8388736) r, each operation rounded to fp32, two at a time.
__device__ __forceinline__ void codes_times(float& y0, float& y1, float r) {
  asm("{\n\t.reg .b64 y, c;\n\tmov.b64 y, {%0, %1};\n\tmov.b64 c, {%3, %3};\n\tadd.rn.f32x2 y, y, c;\n\t"
      "mov.b64 c, {%2, %2};\n\tmul.rn.f32x2 y, y, c;\n\tmov.b64 {%0, %1}, y;\n\t}"
      : "+f"(y0), "+f"(y1)
      : "f"(r), "f"(-8388736.0f));
}

// Per-channel bounds of a page's keys.  With S the largest row scale among the page's
// valid rows, row t's keys are code * (s_t / S) in steps of S; the bounds are the floor
// of the least and the ceiling of the largest, so lo S <= k <= hi S holds for every key
// (up to the rounding of s_t / S and of the product).  A warp per (page, kv head): D / 8
// lanes hold a row, 8 channels each, and the rows run over the remaining lanes, kBatch of a
// lane's rows on their way at once.  Small calls are bound by the latency of the chain
// length -> page id -> rows, large ones by instruction issue, so a row's ratio is divided by
// one lane and shuffled to the others, products go two at a time and extrema take two rows
// at once; four warps a CTA, so that a CTA's slots are free again sooner: 4.7 us for one page
// of 64 rows in each of 64 sequences (8 kv heads, d = 128), 11.3 for the 16-row pages of four
// chunks of 4k to 8k tokens, whose bytes take 4.8 (7.2 and 16.4 without these four).
template <int D>
__global__ void __launch_bounds__(128, 8) page_bounds_kernel(const BoundsArgs a, DeviceStatus* st) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 8;
  constexpr int kSpan = kBatch * kRows, kScales = (kSpan + 31) / 32;  // rows of a batch; scales a lane holds of them
  const int lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * 4 + (threadIdx.x >> 5);
  const uint32_t u = w / static_cast<uint32_t>(a.Hkv), h = w - u * a.Hkv;
  const uint32_t b = u / static_cast<uint32_t>(a.per_seq), i = u - b * a.per_seq;
  if (b >= static_cast<uint32_t>(a.B)) return;
  const int32_t cap = a.max_blocks * a.page;  // below 2^31
  int32_t L = a.seqlens[b];
  bool bad = L < 0 || L > cap;
  L = L < 0 ? 0 : (L > cap ? cap : L);
  int32_t add = L;
  if (a.add) {
    add = a.add[b];
    bad = bad || add < 0 || add > L || add > a.max_new;
    add = add < 0 ? 0 : (add > L ? L : add);
    if (add > a.max_new) add = a.max_new;
  }
  if (bad && i == 0 && h == 0 && lane == 0) record_status(st, kStatusBadArg, 820);
  const uint32_t blk = static_cast<uint32_t>(L - add) / static_cast<uint32_t>(a.page) + i;
  if (add == 0 || blk * static_cast<uint64_t>(a.page) >= static_cast<uint32_t>(L)) return;
  const int n = min(a.page, L - static_cast<int32_t>(blk) * a.page);
  int32_t pg = a.table[static_cast<int64_t>(b) * a.max_blocks + blk];
  if (pg < 0 || pg >= a.num_pages) {
    if (lane == 0) record_status(st, kStatusBadArg, 821);
    return;
  }
  const int64_t ph = static_cast<int64_t>(pg) * a.Hkv + h;
  const int8_t* codes = a.k_pages + ph * a.page * D;
  const float* ks = a.k_scale + ph * a.page;
  const int l = lane % kLanes, sub = lane / kLanes;
  uint2 v[kBatch];
  float f[kScales];
  auto fetch = [&](int t0) {  // rows past n repeat the last one
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      v[j] = *reinterpret_cast<const uint2*>(codes + static_cast<int64_t>(min(t0 + sub + j * kRows, n - 1)) * D + 8 * l);
#pragma unroll
    for (int i = 0; i < kScales; ++i) f[i] = ks[min(t0 + 32 * i + lane, n - 1)];
  };
  fetch(0);
  float S = 0.0f;
#pragma unroll
  for (int i = 0; i < kScales; ++i) S = fmaxf(S, f[i]);
  for (int t = 32 * kScales + lane; t < n; t += 32) S = fmaxf(S, ks[t]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) S = fmaxf(S, __shfl_xor_sync(0xffffffffu, S, o));
  float lo[8], hi[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo[e] = INFINITY;
    hi[e] = -INFINITY;
  }
  for (int t0 = 0; t0 < n; t0 += kSpan) {
    if (t0 != 0) fetch(t0);
#pragma unroll
    for (int i = 0; i < kScales; ++i) f[i] = S > 0.0f && S < INFINITY ? __fdiv_rn(f[i], S) : 0.0f;
#pragma unroll
    for (int j = 0; j < kBatch; j += 2) {  // two rows at a time: least and largest of three
      float r[2], y[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) r[i] = __shfl_sync(0xffffffffu, f[(j + i) * kRows / 32], ((j + i) * kRows + sub) & 31);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // code + 128 as the low bits of 2^23 + code + 128: exact, without a conversion
          const uint32_t x = (e < 4 ? v[j + i].x : v[j + i].y) ^ 0x80808080u;
          y[i][0] = __uint_as_float(prmt(x, 0x4b000000u, 0x7650 + e % 4));
          y[i][1] = __uint_as_float(prmt(x, 0x4b000000u, 0x7651 + e % 4));
          codes_times(y[i][0], y[i][1], r[i]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          asm("min.f32 %0, %0, %1, %2;" : "+f"(lo[e + c]) : "f"(y[0][c]), "f"(y[1][c]));
          asm("max.f32 %0, %0, %1, %2;" : "+f"(hi[e + c]) : "f"(y[0][c]), "f"(y[1][c]));
        }
      }
    }
  }
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
      hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
    }
  }
  if (lane < kLanes) {
    uint32_t a2[2] = {0, 0}, b2[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a2[e / 4] |= static_cast<uint32_t>(static_cast<int>(floorf(lo[e])) & 0xff) << (8 * (e % 4));
      b2[e / 4] |= static_cast<uint32_t>(static_cast<int>(ceilf(hi[e])) & 0xff) << (8 * (e % 4));
    }
    int8_t* dst = a.bounds + ph * 2 * D + 8 * l;
    *reinterpret_cast<uint2*>(dst) = make_uint2(a2[0], a2[1]);
    *reinterpret_cast<uint2*>(dst + D) = make_uint2(b2[0], b2[1]);
    if (lane == 0) a.scale[ph] = S;
  }
}

template <typename T, int D>
cudaError_t launch_append_td(const AppendArgs& a, bool adjacent, unsigned grid, cudaStream_t s) {
  if (adjacent) rope_append_kernel<T, D, true><<<grid, 128, 0, s>>>(a, device_status_ptr());
  else rope_append_kernel<T, D, false><<<grid, 128, 0, s>>>(a, device_status_ptr());
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
  PlanArgs a{ctx_lens, new_lens, release, B, page_size, max_blocks, block_table, free_pages, free_capacity,
             free_count, free_count_out, max_tokens, seqlens, granted, cu_new, slot_map, token_pos,
             ((reinterpret_cast<uintptr_t>(slot_map) | reinterpret_cast<uintptr_t>(token_pos)) & 15u) == 0, true,
             (uint32_t(1) << 31) / static_cast<uint32_t>(page_size)};
  // a small step: one small CTA, whose barriers cost least (8 requests of one token: 5.1 us, and
  // 6.7 with a cluster), unless it may have many pages to push
  if (B <= 256 && max_tokens <= 1024 && (!release || static_cast<int64_t>(B) * max_blocks <= 16384))
    return launch_plan<256>(a, 1, s);
  // many tokens are mapped by a kernel of their own, on every SM (256 requests, 254,000 tokens:
  // 12 us instead of 23)
  a.map = max_tokens <= 16384;
  const cudaError_t e = launch_plan<1024>(a, kPlanCluster, s);
  if (a.map || e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((static_cast<int64_t>(max_tokens) + 1023) / 1024, 8ll * num_sms()));
  return launch_pdl(map_tokens_kernel, dim3(grid), dim3(256), 0, s, a, device_status_ptr());
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
  const int32_t groups = (r.Hq + rows_at_once - 1) / rows_at_once + 2 * ((r.Hkv + rows_at_once - 1) / rows_at_once);
  const int64_t fill = 32ll * num_sms();
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(groups, fill / r.T));
  a.iters = static_cast<int32_t>((groups + parts - 1) / parts);
  a.parts = (groups + a.iters - 1) / a.iters;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(r.T) * a.parts + 3) / 4);
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
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(B) * per_seq * Hkv + 3) / 4);
  switch (d) {
    case 32: page_bounds_kernel<32><<<grid, 128, 0, s>>>(a, device_status_ptr()); break;
    case 64: page_bounds_kernel<64><<<grid, 128, 0, s>>>(a, device_status_ptr()); break;
    case 128: page_bounds_kernel<128><<<grid, 128, 0, s>>>(a, device_status_ptr()); break;
    case 256: page_bounds_kernel<256><<<grid, 128, 0, s>>>(a, device_status_ptr()); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace sl8
