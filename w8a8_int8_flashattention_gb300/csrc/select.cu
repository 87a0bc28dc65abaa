// Page selection for sparse decode attention over the paged int8 cache, for sm_103a.
//
// For every query row and kv head, each page of the sequence gets a score: an upper bound
// of the attention logits its keys can reach, from the page's per-channel key bounds
// (page_bounds).  With q's int8 codes c and scale s_q, and the page's bound codes lo, hi
// and scale S,
//   score = max over the group's query heads of
//           float(sum_i max(c_i lo_i, c_i hi_i)) * S * s_q
//         = the same with sum_i (min(c_i, 0) lo_i + max(c_i, 0) hi_i):
// one int8 dot of 2 d terms per page and query head, exact in int32, then two fp32
// products in this order, so that the selection is the same on every run and for every
// grid.  The max_sel best pages are kept, the first and last ones always, ties to the
// lowest index, and listed in ascending order.
//
// GB300 design: the bounds are read once (2 d + 4 bytes per page and kv head), which is
// the bound for long contexts; for short ones it is the latency of the chain page id ->
// bounds -> scores -> radix passes -> list.  A cluster serves one (query row, kv head); its CTAs
// split the pages.  The dots run as int8 m16n8k32 MMAs (16 pages x 8 query heads): this
// part's int8 tensor rate is low, but a page's row enters as it lies in memory, straight
// into the A fragments, and at 3.6 cycles a page (d = 128, 8 heads) it stays below the
// 11 cycles that its bytes take at an SM's share of HBM.  The keys of the scores stay in
// shared memory, where the cluster finds the max_sel-th largest by a radix select (8 bits
// a pass, histograms added up over distributed shared memory).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "sl8_internal.h"

namespace cg = cooperative_groups;

namespace sl8 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kForced = 0xffffffffu;  // key of a page that is always kept

struct SelectArgs {
  const void* q;
  sl8_dtype q_dtype;
  const int8_t* bounds;   // [num_pages][Hkv][2][d]
  const float* scale;     // [num_pages][Hkv]
  int32_t num_pages, page;
  const int32_t* table;   // [B][max_blocks]
  int32_t max_blocks;
  const int32_t* seqlens;
  int32_t B, T, Hq, Hkv;
  int32_t max_sel, first, last;
  int32_t *blocks, *pages, *lens;
  float* scores;          // nullable
  int32_t cap;            // pages of a row that one CTA of the cluster can hold
};

struct SelectSmem {
  uint32_t hist[256];
  uint32_t sum[2];    // keys above the threshold, keys equal to it, in this CTA
  uint32_t digit, above;
  uint32_t warp_sum[kWarps];
};

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Order-preserving map of a float to an unsigned; + 0 turns a -0 into 0, so equal scores
// have equal keys.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t k = u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
  return k == kForced ? kForced - 1 : k;
}

// D: head dim; kTiles: 8-head tiles of the group when that is 1 (query fragments then stay
// in registers), else 0.
template <int D, int kTiles>
__global__ void __launch_bounds__(kThreads) page_select_kernel(const SelectArgs a, DeviceStatus* st) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ SelectSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x / ranks;  // (b, t, kv head)
  const int h = static_cast<int>(row % a.Hkv);
  const int64_t bt = row / a.Hkv;
  const int b = static_cast<int>(bt / a.T), t = static_cast<int>(bt - static_cast<int64_t>(b) * a.T);
  const int G = a.Hq / a.Hkv, tiles = kTiles ? kTiles : (G + 7) / 8;
  const int64_t cap_tokens = static_cast<int64_t>(a.max_blocks) * a.page;
  int64_t L = a.seqlens[b];
  if (L < 0 || L > cap_tokens) {
    if (tid == 0 && rank == 0) record_status(st, kStatusBadArg, 830);
    L = L < 0 ? 0 : cap_tokens;
  }
  L = max(static_cast<int64_t>(0), L - a.T + 1 + t);
  const int n = static_cast<int>((L + a.page - 1) / a.page);
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_blocks;
  int32_t* out_blocks = a.blocks + row * a.max_sel;
  int32_t* out_pages = a.pages + row * a.max_sel;
  const bool all = n <= a.max_sel;  // every page is kept
  if (all) {
    for (int i = rank * kThreads + tid; i < a.max_sel; i += ranks * kThreads) {
      out_blocks[i] = i < n ? i : -1;
      out_pages[i] = i < n ? table[i] : -1;
    }
    if (rank == 0 && tid == 0) a.lens[row] = static_cast<int32_t>(L);
    if (!a.scores) return;  // the same for every CTA of the cluster
  }

  // ---- the query heads' codes as rows [min(c, 0) | max(c, 0)] of 2 d, and their scales
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
  int8_t* qrows = reinterpret_cast<int8_t*>(smem + (static_cast<size_t>(a.cap) * 4 + 15) / 16 * 16);
  float* qscale = reinterpret_cast<float*>(qrows + tiles * 8 * 2 * D);
  for (int c = warp; c < tiles * 8; c += kWarps) {
    constexpr int E = D / 32;
    float v[E], amax = 0.0f;
    const int64_t base = (bt * a.Hq + h * G + c) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[e] = 0.0f;
      if (c < G)
        v[e] = a.q_dtype == SL8_F32    ? static_cast<const float*>(a.q)[base + e]
               : a.q_dtype == SL8_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[base + e])
                                       : __half2float(static_cast<const __half*>(a.q)[base + e]);
      amax = fmaxf(amax, fabsf(v[e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float sc = __fdiv_rn(amax, 127.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      int code = 0;
      if (sc != 0.0f) code = max(-127, min(127, __float2int_rn(__fdiv_rn(v[e], sc))));
      qrows[c * 2 * D + lane * E + e] = static_cast<int8_t>(min(code, 0));
      qrows[c * 2 * D + D + lane * E + e] = static_cast<int8_t>(max(code, 0));
    }
    if (lane == 0) qscale[c] = sc;
  }
  __syncthreads();

  // ---- scores: a warp takes 16 pages at a time.  Lane (g, tq) = (lane / 4, lane % 4) holds
  // 16-byte chunk tq of every 64-byte segment of rows g and g + 8; the same choice of
  // channels for the query rows keeps the dot whole.
  const int per = (n + ranks - 1) / ranks;
  const int p0 = min(n, rank * per), p1 = min(n, p0 + per);
  constexpr int kSeg = 2 * D / 64;
  const int g = lane >> 2, tq = lane & 3;
  uint4 qf[kTiles ? kSeg : 1];
  float qs[2] = {0.0f, 0.0f};
  if constexpr (kTiles != 0) {
#pragma unroll
    for (int s = 0; s < kSeg; ++s) qf[s] = *reinterpret_cast<const uint4*>(qrows + g * 2 * D + 64 * s + 16 * tq);
    qs[0] = qscale[2 * tq];
    qs[1] = qscale[2 * tq + 1];
  }
  auto page_at = [&](int p) {
    int32_t pg = table[min(p, p1 - 1)];
    if (pg < 0 || pg >= a.num_pages) {
      if (p < p1) record_status(st, kStatusBadArg, 831);
      pg = 0;
    }
    return pg;
  };
  int pa = 0, pb = 0;
  int p = p0 + 16 * warp;
  if (p < p1) {
    pa = page_at(p + g);
    pb = page_at(p + g + 8);
  }
  for (; p < p1; p += 16 * kWarps) {
    const int64_t ia = static_cast<int64_t>(pa) * a.Hkv + h, ib = static_cast<int64_t>(pb) * a.Hkv + h;
    uint4 ra[kSeg], rb[kSeg];
#pragma unroll
    for (int s = 0; s < kSeg; ++s) {
      ra[s] = __ldg(reinterpret_cast<const uint4*>(a.bounds + ia * 2 * D + 64 * s + 16 * tq));
      rb[s] = __ldg(reinterpret_cast<const uint4*>(a.bounds + ib * 2 * D + 64 * s + 16 * tq));
    }
    const float sa = __ldg(a.scale + ia), sb = __ldg(a.scale + ib);
    const int next = p + 16 * kWarps;
    if (next < p1) {
      pa = page_at(next + g);
      pb = page_at(next + g + 8);
    }
    float best_a = -INFINITY, best_b = -INFINITY;
    for (int nt = 0; nt < tiles; ++nt) {
      int d0[4] = {0, 0, 0, 0}, d1[4] = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < kSeg; ++s) {
        uint4 w;
        if constexpr (kTiles != 0) w = qf[s];
        else w = *reinterpret_cast<const uint4*>(qrows + (nt * 8 + g) * 2 * D + 64 * s + 16 * tq);
        mma_s8(d0, ra[s].x, rb[s].x, ra[s].y, rb[s].y, w.x, w.y);
        mma_s8(d1, ra[s].z, rb[s].z, ra[s].w, rb[s].w, w.z, w.w);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int head = nt * 8 + 2 * tq + c;
        float sq;
        if constexpr (kTiles != 0) sq = qs[c];
        else sq = qscale[head];
        if (head < G) {
          best_a = fmaxf(best_a, static_cast<float>(d0[c] + d1[c]) * sa * sq);
          best_b = fmaxf(best_b, static_cast<float>(d0[2 + c] + d1[2 + c]) * sb * sq);
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      best_a = fmaxf(best_a, __shfl_xor_sync(0xffffffffu, best_a, o));
      best_b = fmaxf(best_b, __shfl_xor_sync(0xffffffffu, best_b, o));
    }
    if (tq < 2) {
      const int pp = p + g + 8 * tq;
      const float x = tq ? best_b : best_a;
      if (pp < p1) {
        if (!all) keys[pp - p0] = pp < a.first || pp >= n - a.last ? kForced : key_of(x);
        if (a.scores) a.scores[row * a.max_blocks + pp] = x;
      }
    }
  }
  if (all) return;

  // ---- radix select of the max_sel-th largest key over the cluster
  const int m = p1 - p0;
  uint32_t prefix = 0, want = static_cast<uint32_t>(a.max_sel);  // keys to take from those that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    sm.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kThreads) {
      const uint32_t k = keys[i];
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&sm.hist[(k >> shift) & 255u], 1u);
    }
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    // bin 255 - tid: its count over the cluster, then the counts of the bins above it
    uint32_t count = 0;
    for (int r = 0; r < ranks; ++r) count += ranks > 1 ? *cluster.map_shared_rank(&sm.hist[255 - tid], r) : sm.hist[255 - tid];
    uint32_t incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += sm.warp_sum[w];
    const uint32_t above = before + incl - count;
    if (above < want && above + count >= want) {
      sm.digit = static_cast<uint32_t>(255 - tid);
      sm.above = above;
    }
    if (ranks > 1) cluster.sync();  // every CTA has read the histograms
    else __syncthreads();
    prefix |= sm.digit << shift;
    want -= sm.above;
    __syncthreads();
  }
  // prefix is now the threshold key; `want` pages with that very key are kept, lowest first

  // ---- the list, ascending: each thread takes a run of pages
  const int run = (m + kThreads - 1) / kThreads;
  const int i0 = min(m, tid * run), i1 = min(m, i0 + run);
  uint32_t gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    gt += keys[i] > prefix;
    eq += keys[i] == prefix;
  }
  // exclusive prefixes of both counts over the block (a CTA holds fewer than 2^16 pages)
  const uint32_t mine = (gt << 16) | eq;
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  __syncthreads();
  uint32_t before = incl - mine;
  for (int w = 0; w < warp; ++w) before += sm.warp_sum[w];
  if (tid == kThreads - 1) {
    sm.sum[0] = (before + mine) >> 16;
    sm.sum[1] = (before + mine) & 0xffffu;
  }
  if (ranks > 1) cluster.sync();
  else __syncthreads();
  uint32_t gt0 = before >> 16, eq0 = before & 0xffffu;
  for (int r = 0; r < rank; ++r) {
    gt0 += *cluster.map_shared_rank(&sm.sum[0], r);
    eq0 += *cluster.map_shared_rank(&sm.sum[1], r);
  }
  uint32_t at = gt0 + min(eq0, want);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = keys[i];
    bool take = k > prefix;
    if (k == prefix) take = eq0++ < want;
    const int blk = p0 + i;
    if (take) {
      out_blocks[at] = blk;
      out_pages[at] = table[blk];
      ++at;
    }
    // the row's last page decides how many tokens the list holds
    if (blk == n - 1)
      a.lens[row] = static_cast<int32_t>(static_cast<int64_t>(a.max_sel) * a.page -
                                         (take ? static_cast<int64_t>(n) * a.page - L : 0));
  }
  if (ranks > 1) cluster.sync();  // no CTA leaves while another reads its sums
}

size_t select_smem(int32_t cap, int32_t d, int32_t tiles) {
  return (static_cast<size_t>(cap) * 4 + 15) / 16 * 16 + static_cast<size_t>(tiles) * 8 * (2 * d + 4);
}

template <int D, int kTiles>
cudaError_t launch_select_dt(const SelectArgs& a, unsigned rows, unsigned ranks, size_t smem, cudaStream_t s) {
  auto kern = page_select_kernel<D, kTiles>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, device_status_ptr());
}
template <int D>
cudaError_t launch_select_d(const SelectArgs& a, unsigned rows, unsigned ranks, size_t smem, cudaStream_t s) {
  return a.Hq / a.Hkv <= 8 ? launch_select_dt<D, 1>(a, rows, ranks, smem, s)
                           : launch_select_dt<D, 0>(a, rows, ranks, smem, s);
}

constexpr size_t kSelectSmemMax = 200 * 1024;

// CTAs of a row's cluster: as many as keep the device busy, at least 256 pages each, and
// enough that each CTA's keys fit its shared memory; 0 if eight cannot hold them.
int select_ranks(int64_t rows, int32_t max_blocks, int32_t d, int32_t tiles) {
  int ranks = 1;
  while (ranks < kMaxCluster && rows * ranks < num_sms() && max_blocks / (2 * ranks) >= 256) ranks *= 2;
  while (ranks <= kMaxCluster && select_smem((max_blocks + ranks - 1) / ranks, d, tiles) > kSelectSmemMax) ranks *= 2;
  return ranks <= kMaxCluster ? ranks : 0;
}

}  // namespace

bool page_select_fits(int64_t rows, int32_t max_blocks, int32_t d, int32_t group) {
  return select_ranks(rows, max_blocks, d, (group + 7) / 8) != 0;
}

cudaError_t launch_page_select(const void* q, sl8_dtype q_dtype, const int8_t* bounds, const float* bound_scale,
                               int32_t num_pages, int32_t page_size, const int32_t* block_table, int32_t max_blocks,
                               const int32_t* seqlens, int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t d,
                               int32_t max_sel, int32_t first, int32_t last, int32_t* sel_blocks, int32_t* sel_pages,
                               int32_t* sel_lens, float* scores, cudaStream_t s) {
  TraceScope tr("page_select", s);
  const int64_t rows = static_cast<int64_t>(B) * T * Hkv;
  const int32_t tiles = (Hq / Hkv + 7) / 8;
  const int ranks = select_ranks(rows, max_blocks, d, tiles);
  if (ranks == 0) return cudaErrorInvalidValue;
  SelectArgs a{q, q_dtype, bounds, bound_scale, num_pages, page_size, block_table, max_blocks, seqlens, B, T, Hq, Hkv,
               max_sel, first, last, sel_blocks, sel_pages, sel_lens, scores, 0};
  a.cap = (max_blocks + ranks - 1) / ranks;
  const size_t smem = select_smem(a.cap, d, tiles);
  switch (d) {
    case 32: return launch_select_d<32>(a, static_cast<unsigned>(rows), ranks, smem, s);
    case 64: return launch_select_d<64>(a, static_cast<unsigned>(rows), ranks, smem, s);
    case 128: return launch_select_d<128>(a, static_cast<unsigned>(rows), ranks, smem, s);
    case 256: return launch_select_d<256>(a, static_cast<unsigned>(rows), ranks, smem, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sl8
