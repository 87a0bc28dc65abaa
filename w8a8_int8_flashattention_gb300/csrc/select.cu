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
// GB300 design: one kernel.  A CTA (a cluster of CTAs where there are few rows) serves one
// (query row, kv head): it reads the bounds of the row's pages once (2 d + 4 bytes each),
// keeps the scores' keys in shared memory, finds the threshold and writes the list.  What
// passes kHeld pages a CTA is read back from `scores`: keys held for every block of a wide
// table would cost resident CTAs (64 x 8 rows of 256 to 1,024 pages: 22.6 us with a table of
// 4,096 blocks, 23.6 with 65,536, and 27 / 61 / 100 with 8,192 / 32,768 / 65,536 if all are
// held).  Long contexts and large batches are bound by the bounds' bytes, small calls by the latency of
// the chain length -> page id -> bounds -> threshold -> list, so every row of a batch runs
// at once.  Measured against two kernels (scores, then lists) for 64 sequences of 8k to 32k
// tokens in 32-token pages, 8 kv heads, d = 128: 26.6 us against 33, and 9.9 against 12 for
// one sequence of 2,048 pages.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "decode_unit.cuh"
#include "sl8_internal.h"

namespace cg = cooperative_groups;

namespace sl8 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kForced = 0xffffffffu;  // key of a page that is always kept
constexpr int kBins = 4 * kThreads;        // bins of one narrowing step, four per thread
constexpr int kCand = kThreads;            // keys that are ranked against each other
constexpr int kHeld = kPageSelectHeld;     // keys that a CTA holds in shared memory
static_assert(kMaxCluster <= kWarps, "a warp collects each CTA's candidates");

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
  float* scores;          // nullable while no table is wider than kHeld
  int32_t cap;            // pages whose keys a CTA holds in shared memory
  uint32_t ranks;         // CTAs of the cluster
};

struct __align__(16) SelectSmem {
  uint32_t hist[kBins];
  // [r]: from CTA r of the cluster, which writes it into every CTA before a barrier, so that
  // nothing is fetched after it
  uint32_t cand[kMaxCluster][kCand];  // its keys of the threshold's bin
  uint32_t n_cand[kMaxCluster];
  uint32_t sum[kMaxCluster][2];  // its keys above the threshold, and equal to it
  uint32_t all[kCand];           // the candidates, one after another
  uint32_t own_cand;
  uint32_t bin, above, count;    // the threshold's bin: its number, the keys above it, its keys
  uint32_t key, want;            // the threshold key, and how many of the keys equal to it to keep
  uint2 warp_sum[kWarps];
};

// Order-preserving map of a float to an unsigned above 0 and below kForced; + 0 turns a -0
// into 0, so equal scores have equal keys.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t k = u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
  return min(max(k, 1u), kForced - 1);
}
// The bin of a key in the histogram that the scoring fills: 32 bins per octave of positive
// scores from 2^-16 to 2^16, all lower keys in bin 0 and all higher ones in the last.
constexpr int kFirstShift = 18;  // sign, exponent and 5 bits of the mantissa
constexpr uint32_t kFirstBase = (256 + 127 - 16) * 32;
static_assert(kBins == 32 * 32, "32 octaves of 32 bins");
__device__ __forceinline__ uint32_t first_bin(uint32_t k) {
  const uint32_t b = k >> kFirstShift;
  return b <= kFirstBase ? 0u : min(b - kFirstBase, static_cast<uint32_t>(kBins - 1));
}

// A lane's share of a bounds row: 32 contiguous bytes of every 128 (16 of the 64 at d = 32), so
// that the four lanes of a row read whole cache lines.
template <int D>
struct RowCfg {
  static constexpr int kBytes = D == 32 ? 16 : 32;
  static constexpr int kSeg = 2 * D / (4 * kBytes);  // segments of a row
  static constexpr int kWords = kBytes / 4;
  static constexpr int kStride = 2 * D + 16;         // query rows in shared memory: 16 bytes of
                                                     // padding keep the rows off each other's banks
};
template <int kWords>
__device__ __forceinline__ void load_words(const int8_t* p, uint32_t (&w)[kWords]) {
  if constexpr (kWords == 8)
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  else
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
}
// The negative and the positive codes among four: min(c, 0) and max(c, 0) per byte.
__device__ __forceinline__ uint32_t negatives(uint32_t c) { return c & __vcmplts4(c, 0u); }
__device__ __forceinline__ uint32_t positives(uint32_t c) { return c & ~__vcmplts4(c, 0u); }

// Index arithmetic is 32-bit throughout: divisions of 64 bits by numbers known only at run
// time cost more than the rest of the prologue.
// kWide: a CTA's pages can pass kHeld; built apart, since the reading back costs 0.6 us of 26.4
// where it is not needed.
template <int D, bool kWide>
__global__ void __launch_bounds__(kThreads, D == 256 ? 2 : 4) page_select_kernel(const SelectArgs a, DeviceStatus* st) {
  using R = RowCfg<D>;
  constexpr int kSeg = R::kSeg, kWords = R::kWords, kRuns = D / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ SelectSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t ranks = a.ranks, row = blockIdx.x / ranks, rank = blockIdx.x - row * ranks;  // row: (b, t, kv head)
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bt = row / static_cast<uint32_t>(a.Hkv), h = row - bt * a.Hkv;
  const uint32_t b = a.T == 1 ? bt : bt / static_cast<uint32_t>(a.T), t = bt - b * a.T;
  const int G = a.Hq / a.Hkv, tiles = (G + 7) / 8;
  // four query rows a warp, eight lanes each, D / 32 runs of four channels; the first ones are
  // on their way while the length is read
  const int qr = 4 * warp + (lane >> 3), ql = lane & 7;
  float x[kRuns][4] = {};
  auto load_q = [&](int c) {
    if (c < G) load_runs<kRuns>(a.q, a.q_dtype, (static_cast<int64_t>(bt) * a.Hq + h * G + c) * D + 4 * ql, 32, x);
  };
  load_q(qr);
  // so are the ids of the warp's first 16 pages, where they do not depend on the length
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_blocks;
  const int g = lane >> 2, tq = lane & 3;
  int32_t pa = 0, pb = 0;  // checked where they are used, so that nothing waits for them here
  int p = 16 * warp;
  if (ranks == 1) {
    if (p + g < a.max_blocks) pa = table[p + g];
    if (p + g + 8 < a.max_blocks) pb = table[p + g + 8];
  }
  const int32_t cap = a.max_blocks * a.page;  // below 2^31
  int32_t L = a.seqlens[b];
  if (L < 0 || L > cap) {
    if (tid == 0 && rank == 0) record_status(st, kStatusBadArg, 830);
    L = L < 0 ? 0 : cap;
  }
  L = max(0, L - (a.T - 1 - static_cast<int32_t>(t)));
  const int n = static_cast<int>((static_cast<uint32_t>(L) + a.page - 1) / static_cast<uint32_t>(a.page));
  int32_t* out_blocks = a.blocks + static_cast<int64_t>(row) * a.max_sel;
  int32_t* out_pages = a.pages + static_cast<int64_t>(row) * a.max_sel;
  if (n <= a.max_sel) {  // every page is kept; the same for every CTA of the cluster
    for (int i = rank * kThreads + tid; i < a.max_sel; i += ranks * kThreads) {
      out_blocks[i] = i < n ? i : -1;
      out_pages[i] = i < n ? table[i] : -1;
    }
    if (rank == 0 && tid == 0) a.lens[row] = L;
    return;
  }

  // the pages of this CTA; lanes past the last one score page 0 and store nothing
  const int per = ranks == 1 ? n : static_cast<int>((n + ranks - 1) / ranks);
  const int p0 = min(n, static_cast<int>(rank) * per), p1 = min(n, p0 + per), m = p1 - p0;
  p += p0;
  if (ranks > 1 && p < p1) {
    pa = table[min(p + g, p1 - 1)];
    pb = table[min(p + g + 8, p1 - 1)];
  }
  if (p + g >= p1) pa = 0;
  if (p + g + 8 >= p1) pb = 0;

  // ---- the query heads' codes as rows [min(c, 0) | max(c, 0)] of 2 d, and their scales
  uint2* keys = reinterpret_cast<uint2*>(smem);  // key and page id of this CTA's first pages
  auto score_at = [&](int pp) { return a.scores + static_cast<int64_t>(row) * a.max_blocks + pp; };
  auto forced = [&](int pp) { return pp < a.first || pp >= n - a.last; };
  auto key_at = [&](int i) {  // of this CTA's page i
    return !kWide || i < a.cap ? keys[i].x : forced(p0 + i) ? kForced : key_of(__ldcg(score_at(p0 + i)));
  };
  int8_t* qrows = reinterpret_cast<int8_t*>(smem + (static_cast<size_t>(a.cap) * 8 + 15) / 16 * 16);
  float* qscale = reinterpret_cast<float*>(qrows + tiles * 8 * R::kStride);
  for (int c = qr; c < tiles * 8; c += 4 * kWarps) {
    if (c != qr) {
#pragma unroll
      for (int i = 0; i < kRuns; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.0f;
      load_q(c);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[i][e]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const RowScale rs = row_scale(amax);
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const uint32_t code = quant4(x[i], rs);
      *reinterpret_cast<uint32_t*>(qrows + c * R::kStride + 32 * i + 4 * ql) = negatives(code);
      *reinterpret_cast<uint32_t*>(qrows + c * R::kStride + D + 32 * i + 4 * ql) = positives(code);
    }
    if (ql == 0) qscale[c] = rs.s;
  }
  for (int i = tid; i < kBins; i += kThreads) sm.hist[i] = 0;
  if (tid == 0) sm.own_cand = 0;
  __syncthreads();

  // ---- scores: a warp takes 16 pages at a time.  Lane (g, tq) = (lane / 4, lane % 4) holds
  // chunk tq of every segment of pages g and g + 8 as the A fragments of int8 m16n8k32 MMAs
  // (16 pages x 8 query heads), straight from memory; the same choice of channels for the
  // query rows keeps the dot whole.  This part's int8 rate is low (4 cycles an MMA and SM),
  // yet 8 MMAs per 16 pages (d = 128) are a fifth of the time that their 4 KB take at an
  // SM's share of HBM.
  for (; p < p1; p += 16 * kWarps) {
    if (static_cast<uint32_t>(pa) >= static_cast<uint32_t>(a.num_pages) ||
        static_cast<uint32_t>(pb) >= static_cast<uint32_t>(a.num_pages)) {
      record_status(st, kStatusBadArg, 831);  // page 0 is scored in its place
      pa = static_cast<uint32_t>(pa) < static_cast<uint32_t>(a.num_pages) ? pa : 0;
      pb = static_cast<uint32_t>(pb) < static_cast<uint32_t>(a.num_pages) ? pb : 0;
    }
    const int64_t ia = static_cast<int64_t>(pa) * a.Hkv + h, ib = static_cast<int64_t>(pb) * a.Hkv + h;
    uint32_t ra[kSeg][kWords], rb[kSeg][kWords];
#pragma unroll
    for (int s = 0; s < kSeg; ++s) {
      load_words<kWords>(a.bounds + ia * 2 * D + R::kBytes * (4 * s + tq), ra[s]);
      load_words<kWords>(a.bounds + ib * 2 * D + R::kBytes * (4 * s + tq), rb[s]);
    }
    const float sa = __ldg(a.scale + ia), sb = __ldg(a.scale + ib);
    const int next = p + 16 * kWarps;
    int32_t na = 0, nb = 0;
    if (next < p1) {
      na = table[min(next + g, p1 - 1)];
      nb = table[min(next + g + 8, p1 - 1)];
    }
    float best_a = -INFINITY, best_b = -INFINITY;
    for (int nt = 0; nt < tiles; ++nt) {
      int d0[4] = {0, 0, 0, 0}, d1[4] = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < kSeg; ++s) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          const uint4 w =
              *reinterpret_cast<const uint4*>(qrows + (nt * 8 + g) * R::kStride + R::kBytes * (4 * s + tq) + 4 * i);
          mma_s8(d0, ra[s][i], rb[s][i], ra[s][i + 1], rb[s][i + 1], w.x, w.y);
          mma_s8(d1, ra[s][i + 2], rb[s][i + 2], ra[s][i + 3], rb[s][i + 3], w.z, w.w);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int head = nt * 8 + 2 * tq + c;
        if (head < G) {
          const float sq = qscale[head];
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
      const float score = tq ? best_b : best_a;
      if (pp < p1) {
        const bool always = forced(pp);
        const uint32_t k = always ? kForced : key_of(score);
        if (!kWide || pp - p0 < a.cap) keys[pp - p0] = make_uint2(k, static_cast<uint32_t>(tq ? pb : pa));
        if (!always) atomicAdd(&sm.hist[first_bin(k)], 1u);
        if (a.scores) *score_at(pp) = score;
      }
    }
    pa = na;
    pb = nb;
  }

  // ---- the threshold: the want-th largest key of those that are not forced.  The range
  // [lo, hi] that holds it is cut into kBins bins (the first time as first_bin does), the
  // one that holds it becomes the next range, until the bin is kept whole, has few enough
  // keys to rank against each other (the usual end of the first step), or is a single key.
  uint32_t lo = 0, hi = kForced - 1, want = static_cast<uint32_t>(a.max_sel - a.first - a.last), thr = kForced - 1;
  // no narrowing, so no barrier yet: every CTA has to be there before its memory is written below
  if (want == 0 && ranks > 1) cluster.sync();
  for (bool start = true; want > 0; start = false) {
    const int shift = start ? kFirstShift : max(0, (32 - __clz(hi - lo)) - (31 - __clz(kBins)));
    if (!start) {
      for (int i = tid; i < m; i += kThreads) {
        const uint32_t k = key_at(i);
        if (k >= lo && k <= hi) atomicAdd(&sm.hist[(k - lo) >> shift], 1u);
      }
    }
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    // thread tid: bins kBins - 4 - 4 tid .. + 3, from the top; their counts over the cluster
    const int b0 = kBins - 4 - 4 * tid;
    uint4 c4 = *reinterpret_cast<const uint4*>(&sm.hist[b0]);
    if (ranks > 1) {
      uint4 o4[kMaxCluster - 1];  // the others', all on their way at once
#pragma unroll
      for (int i = 0; i < kMaxCluster - 1; ++i)
        if (i < static_cast<int>(ranks) - 1)
          o4[i] = *reinterpret_cast<const uint4*>(
              cluster.map_shared_rank(&sm.hist[b0], rank + 1 + i >= ranks ? rank + 1 + i - ranks : rank + 1 + i));
#pragma unroll
      for (int i = 0; i < kMaxCluster - 1; ++i) {
        if (i < static_cast<int>(ranks) - 1) {
          c4.x += o4[i].x;
          c4.y += o4[i].y;
          c4.z += o4[i].z;
          c4.w += o4[i].w;
        }
      }
    }
    uint32_t incl = c4.x + c4.y + c4.z + c4.w;
    const uint32_t mine = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm.warp_sum[warp].x = incl;
    __syncthreads();
    uint32_t above = incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? sm.warp_sum[lane].x : 0u);
    const uint32_t cnt[4] = {c4.w, c4.z, c4.y, c4.x};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (above < want && above + cnt[j] >= want) {
        sm.bin = static_cast<uint32_t>(b0 + 3 - j);
        sm.above = above;
        sm.count = cnt[j];
      }
      above += cnt[j];
    }
    __syncthreads();
    const uint32_t bin = sm.bin, count = sm.count;
    if (start) {
      lo = bin == 0 ? 0u : (bin + kFirstBase) << kFirstShift;
      hi = bin == kBins - 1 ? kForced - 1 : ((bin + 1 + kFirstBase) << kFirstShift) - 1u;
    } else {
      lo += bin << shift;
      hi = min(hi, lo + ((1u << shift) - 1u));
    }
    want -= sm.above;
    if (want == count) {  // the whole bin is kept: everything above the key below it
      thr = lo > 0 ? lo - 1 : 0;
      want = 0;
      break;
    }
    if (shift == 0) {  // a single key
      thr = lo;
      break;
    }
    if (count <= kCand) {
      for (int i = tid; i < m; i += kThreads) {
        const uint32_t k = key_at(i);
        if (k >= lo && k <= hi) sm.cand[rank][atomicAdd(&sm.own_cand, 1u)] = k;
      }
      __syncthreads();
      if (ranks > 1) {
        // warp r sends this CTA's to CTA r, and packs what CTA r sent
        if (warp < ranks && warp != rank) {
          for (uint32_t i = lane; i < sm.own_cand; i += 32) *cluster.map_shared_rank(&sm.cand[rank][i], warp) = sm.cand[rank][i];
        }
        if (warp < ranks && lane == 0) *cluster.map_shared_rank(&sm.n_cand[rank], warp) = sm.own_cand;
        cluster.sync();
        const uint32_t nr = lane < ranks ? sm.n_cand[lane] : 0u;
        const uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? nr : 0u);
        const uint32_t own = __shfl_sync(0xffffffffu, nr, warp);
        for (uint32_t i = lane; i < own; i += 32) sm.all[at + i] = sm.cand[warp][i];
        __syncthreads();
      }
      const uint32_t* cand = ranks > 1 ? sm.all : sm.cand[0];
      if (tid < count) {
        const uint32_t k = cand[tid];
        uint32_t above_k = 0, equal = 0;
        for (uint32_t i = 0; i < count; ++i) {
          above_k += cand[i] > k;
          equal += cand[i] == k;
        }
        if (above_k < want && above_k + equal >= want) {  // equal keys all write the same
          sm.key = k;
          sm.want = want - above_k;
        }
      }
      __syncthreads();
      thr = sm.key;
      want = sm.want;
      break;
    }
    // narrow: clear the bins once every CTA has read them
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) sm.hist[i] = 0;
    __syncthreads();
  }

  // ---- the list, ascending: keys above thr, and the first `want` that equal it.  Each thread
  // takes a run of pages; exclusive prefixes of both counts place its entries.
  const int run = (m + kThreads - 1) / kThreads;
  const int i0 = min(m, static_cast<int>(tid) * run), i1 = min(m, i0 + run);
  uint32_t gt = 0, eq = 0;
  __syncthreads();  // the keys; the narrowing is done with warp_sum
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    gt += k > thr;
    eq += k == thr;
  }
  uint32_t gt0 = gt, eq0 = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, gt0, o), y = __shfl_up_sync(0xffffffffu, eq0, o);
    if (lane >= o) {
      gt0 += x;
      eq0 += y;
    }
  }
  if (lane == 31) sm.warp_sum[warp] = make_uint2(gt0, eq0);
  __syncthreads();
  const uint2 before = lane < warp ? sm.warp_sum[lane] : make_uint2(0u, 0u);
  gt0 += __reduce_add_sync(0xffffffffu, before.x) - gt;
  eq0 += __reduce_add_sync(0xffffffffu, before.y) - eq;
  if (ranks > 1) {  // those of the CTAs before this one count too
    if (tid == kThreads - 1) {
      for (uint32_t r = rank + 1; r < ranks; ++r) {
        uint32_t* sum = cluster.map_shared_rank(sm.sum[rank], r);
        sum[0] = gt0 + gt;
        sum[1] = eq0 + eq;
      }
    }
    cluster.sync();  // the last one: no CTA reads or writes another's memory after it
    gt0 += __reduce_add_sync(0xffffffffu, lane < rank ? sm.sum[lane][0] : 0u);
    eq0 += __reduce_add_sync(0xffffffffu, lane < rank ? sm.sum[lane][1] : 0u);
  }
  uint32_t at = gt0 + min(eq0, want);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    bool take = k > thr;
    if (k == thr) take = eq0++ < want;
    const int blk = p0 + i;
    if (take) {
      int32_t pg;
      if (!kWide || i < a.cap) {
        pg = static_cast<int32_t>(keys[i].y);
      } else {
        pg = table[blk];
        if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(a.num_pages)) pg = 0;
      }
      out_blocks[at] = blk;
      out_pages[at] = pg;
      ++at;
    }
    // the row's last page decides how many tokens the list holds
    if (blk == n - 1) a.lens[row] = a.max_sel * a.page - (take ? n * a.page - L : 0);
  }
}

size_t select_smem(int32_t cap, int32_t d, int32_t tiles) {
  return (static_cast<size_t>(cap) * 8 + 15) / 16 * 16 + static_cast<size_t>(tiles) * 8 * (2 * d + 16 + 4);
}

template <int D, bool kWide>
cudaError_t launch_select_w(const SelectArgs& a, unsigned rows, size_t smem, cudaStream_t s) {
  auto kern = page_select_kernel<D, kWide>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * a.ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, device_status_ptr());
}

template <int D>
cudaError_t launch_select_d(const SelectArgs& a, unsigned rows, size_t smem, cudaStream_t s) {
  const bool wide = (a.max_blocks + static_cast<int64_t>(a.ranks) - 1) / a.ranks > a.cap;
  return wide ? launch_select_w<D, true>(a, rows, smem, s) : launch_select_w<D, false>(a, rows, smem, s);
}

// CTAs of a row's cluster: as many as there are SMs for, at least 128 pages each.
int select_ranks(int64_t rows, int32_t max_blocks) {
  int ranks = 1;
  while (ranks < kMaxCluster && rows * ranks * 2 <= num_sms() && max_blocks / (2 * ranks) >= 128) ranks *= 2;
  return ranks;
}

}  // namespace

cudaError_t launch_page_select(const void* q, sl8_dtype q_dtype, const int8_t* bounds, const float* bound_scale,
                               int32_t num_pages, int32_t page_size, const int32_t* block_table, int32_t max_blocks,
                               const int32_t* seqlens, int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t d,
                               int32_t max_sel, int32_t first, int32_t last, int32_t* sel_blocks, int32_t* sel_pages,
                               int32_t* sel_lens, float* scores, cudaStream_t s) {
  TraceScope tr("page_select", s);
  const int64_t rows = static_cast<int64_t>(B) * T * Hkv;
  const int32_t tiles = (Hq / Hkv + 7) / 8;
  const int ranks = select_ranks(rows, max_blocks);
  SelectArgs a{q, q_dtype, bounds, bound_scale, num_pages, page_size, block_table, max_blocks, seqlens, B, T, Hq, Hkv,
               max_sel, first, last, sel_blocks, sel_pages, sel_lens, scores, 0, 0};
  a.cap = std::min((max_blocks + ranks - 1) / ranks, kHeld);
  a.ranks = static_cast<uint32_t>(ranks);
  const size_t smem = select_smem(a.cap, d, tiles);
  switch (d) {
    case 32: return launch_select_d<32>(a, static_cast<unsigned>(rows), smem, s);
    case 64: return launch_select_d<64>(a, static_cast<unsigned>(rows), smem, s);
    case 128: return launch_select_d<128>(a, static_cast<unsigned>(rows), smem, s);
    case 256: return launch_select_d<256>(a, static_cast<unsigned>(rows), smem, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sl8
