// Sparse decode: attention of one query row over a page list of its own per kv head of the
// paged int8 cache, for sm_103a.  The arithmetic is the split-KV decode's (decode.cu):
//   x_t = int32(q_i8 . k_i8[t]) * s_q * s_k[t] / sqrt(d),  p = softmax(x),
//   O = sum_t p_t * s_v[t] * v_i8[t]
// over the tokens of the listed pages.
//
// GB300 design.  A list is short (some thousand tokens) and there are many, so the kernel
// is not persistent: a cluster of S CTAs serves one list, each CTA a contiguous run of its
// stages of 64 tokens, and two to five CTAs share an SM, one's start and end hidden behind
// the others' streams.  The S partial results meet over distributed shared memory, so one
// launch does everything and no workspace or counter is shared between launches.
//  * The last warp loads: per stage, one lane per piece of 64, 32 or 16 rows (the largest
//    that divides the page) issues the piece's K and V tiles (TMA, 128-byte swizzle for
//    d >= 128) and its two scale rows; page ids are read 32 pieces ahead.
//  * Warps 0..3 take 16 tokens of every stage each, with an online-softmax state of their
//    own.  S^T[16 tokens x 8 q] = K Q^T runs as int8 m16n8k32 MMAs, whose A operand is the K
//    rows as they lie in memory (this part's int8 rate is low, 4 cycles an MMA and SM, but 4
//    MMAs per 16 tokens at d = 128 take 16 of the 180 cycles that their bytes need);
//    O^T[d x 8 q] += V^T P'^T as fp16 MMAs on V codes biased by 128 (P' = p * s_v * 2^-E
//    rounded to fp16, off by 2^-11 of itself, 2^-22 for fp32 outputs (kFine), or by 2^-24 of the
//    list's largest p * s_v; E follows that weight, see grow_column; sums and the output
//    accumulate in fp32).
// HBM is the bound; the listed pages are read once per group of at most 8 query heads of a kv
// head.  64 rows x 8 kv heads x 4,096 tokens (d = 128) take 87.9 us, 6.2 TB/s, 0.91 of the measured
// copy rate; 32 lists of 512 tokens 6.3 us, mostly launch, prologue and merge.  (The split kernel
// and the combine over the same lists: 152 and 14.4 us.)  At d = 64 a stage is half the bytes for
// the same chain of steps: 600 lists of 4,096 tokens take 61 us, 0.80 of the copy rate.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>

#include "decode_unit.cuh"
#include "sl8_internal.h"

namespace cg = cooperative_groups;

namespace sl8 {

namespace {

constexpr int kMaxSplits = 8;                // CTAs per list (portable cluster size)

constexpr int kWarps = 4, kCThreads = 32 * kWarps;  // compute warps
constexpr int kThreads = kCThreads + 32;            // and the loader
constexpr int kTok = 16 * kWarps;                   // tokens per stage

// kCtas CTAs share an SM: list_ctas(d), or one more at d = 64 and 128, with fewer registers and
// stages, which only run unsplit lists and so carry no merge.
constexpr int list_ctas(int d) { return d == 256 ? 2 : d == 128 ? 3 : 4; }
template <int D, int kCtas>
struct LCfg {
  static constexpr bool kMerge = kCtas == list_ctas(D);
  static constexpr int kBW = D < 128 ? D : 128;  // bytes in one row of a TMA box
  static constexpr int kBoxes = D / kBW;
  static constexpr bool kSwz = D >= 128;
  static constexpr int kTile = kTok * D;
  static constexpr int kSK = 0, kSV = kTile, kSKs = 2 * kTile, kSVs = kSKs + kTok * 4;
  static constexpr int kAlign = kSwz ? 1024 : 128;  // swizzled tiles need 1024-byte alignment
  static constexpr int kStageBytes = (kSVs + kTok * 4 + kAlign - 1) / kAlign * kAlign;
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? (kMerge ? 4 : 3) : kMerge ? 6 : 4;
  // after the loop the ring holds the warps' O^T [warp][D][8] and the CTA's [8][D], fp32
  static constexpr int kRed = 0, kPart = kWarps * D * 32;
  static_assert(kPart + D * 32 <= kStages * kStageBytes, "the merge fits the ring");
  static constexpr int kQc = kStages * kStageBytes;       // [8][D] query codes
  static constexpr int kQs = kQc + 8 * D;                 // [8] scales
  static constexpr int kStat = kQs + 32;                  // [warp][8][2]: max (log2), sum
  static constexpr int kWt = kStat + kWarps * 64;        // [warp][8] weights of the warps
  static constexpr int kMl = kWt + kWarps * 32;          // [8] max, [8] sum of the CTA
  static constexpr int kBar = kMl + 64;
  static constexpr int kBytes = kBar + 2 * kStages * 8 + 1024;  // + alignment slack
  static_assert(!kSwz || kTile % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  // an SM has 228 KB, of which each CTA takes one more for itself
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "kCtas CTAs fit an SM");
};

// Byte offset of (row r, 16-byte chunk c of the row) in a stage tile of kBoxes boxes.
template <int D>
__device__ __forceinline__ uint32_t ltile_off(int r, int c) {
  using C = LCfg<D, 2>;  // the tile is the same for all
  constexpr int cpb = C::kBW / 16;
  const int b = c / cpb, cc = c % cpb;
  return static_cast<uint32_t>(b * (kTok * C::kBW) + r * C::kBW + 16 * (C::kSwz ? (cc ^ (r & 7)) : cc));
}

// kFine: P' goes to the MMAs as two fp16 terms, its rounding and what that left, which keeps 22
// bits of it; for fp32 outputs.  The second half of the P V MMAs costs an eighth of the time at
// worst (512 lists of 4,096 tokens, d = 128: 93.1 us instead of 88.4; 256 of them with 16 query
// heads: 92.8 instead of 82.2), and bf16 and fp16 outputs round to 8 and 11 bits themselves.
template <int D, int kCtas, bool kFine>
__global__ void __launch_bounds__(kThreads, kCtas)
    list_decode_kernel(const ListDecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, DeviceStatus* st, uint64_t limit_ns) {
  using C = LCfg<D, kCtas>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBar);
  uint64_t* empty = full + kStages;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = C::kMerge ? a.splits : 1, rank = S > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // list v = row * Hkv + kv head; its G query heads are cut into groups of GC <= 8
  const int vg = static_cast<int>(blockIdx.x / static_cast<unsigned>(S));
  const int v = vg / a.groups, grp = vg - v * a.groups;
  const int G = a.Hq / a.Hkv, GC = G / a.groups;
  const int64_t row0 = static_cast<int64_t>(v) * G + grp * GC;  // first of the GC rows of q and out

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_barrier_init();
  }
  int L = a.lens[v];
  const int cap = a.max_sel * a.page;
  if (L < 0 || L > cap) {
    if (threadIdx.x == 0) record_status(st, kStatusBadArg, 840);
    L = L < 0 ? 0 : cap;
  }
  // this CTA's stages of the list, and its tokens [t0, t1)
  const int n_all = (L + kTok - 1) / kTok;  // below 2^25
  const int s0 = static_cast<int>(static_cast<uint32_t>(n_all * rank) / static_cast<uint32_t>(S));
  const int s1 = static_cast<int>(static_cast<uint32_t>(n_all * (rank + 1)) / static_cast<uint32_t>(S));
  const int t0 = s0 * kTok, t1 = min(L, s1 * kTok), n = s1 - s0;
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ loader
    const int pieces = kTok / a.box;
    const int head = v % a.Hkv;
    const int32_t* list = a.list + static_cast<int64_t>(v) * a.max_sel;
    // page ids come 32 pieces at a time, read one batch ahead; pieces past t1 are not loaded
    const int n_pieces = (t1 - t0 + a.box - 1) / a.box;
    auto ids_at = [&](int j) { return j + lane < n_pieces ? list[(t0 + (j + lane) * a.box) / a.page] : 0; };
    int32_t ids = n > 0 ? ids_at(0) : 0, next_ids = n > 0 ? ids_at(32) : 0;
    if (lane == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
    int k = 0;
    for (; k < n; ++k) {
      const int j = k * pieces;  // the stage's first piece; pieces divides 32
      if (k > 0 && j % 32 == 0) {
        ids = next_ids;
        next_ids = ids_at(j + 32);
      }
      int32_t pg = __shfl_sync(0xffffffffu, ids, (j + lane) & 31);
      const int stg = k % kStages;
      if (k >= kStages && !warp_wait(&empty[stg], ((k / kStages) - 1) & 1, limit_ns, st, 850)) break;
      uint8_t* base = smem + stg * C::kStageBytes;
      const int tok = t0 + k * kTok;
      const int live = (min(kTok, t1 - tok) + a.box - 1) / a.box;
      if (lane == 0) mbar_arrive_expect_tx(&full[stg], static_cast<uint32_t>(live * a.box * 2 * (D + 4)));
      __syncwarp();
      if (lane < live) {
        if (pg < 0 || pg >= a.num_pages) {
          record_status(st, kStatusBadArg, 851);
          pg = 0;
        }
        const int64_t prow = (static_cast<int64_t>(pg) * a.Hkv + head) * a.page + (tok + lane * a.box) % a.page;
#pragma unroll
        for (int b = 0; b < C::kBoxes; ++b) {
          const uint32_t dst = static_cast<uint32_t>(b * kTok * C::kBW + lane * a.box * C::kBW);
          tma_load_3d(base + C::kSK + dst, &kmap, &full[stg], b * C::kBW, static_cast<int>(prow), 0);
          tma_load_3d(base + C::kSV + dst, &vmap, &full[stg], b * C::kBW, static_cast<int>(prow), 0);
        }
        bulk_load(base + C::kSKs + lane * a.box * 4, a.k_scale + prow, static_cast<uint32_t>(a.box * 4), &full[stg]);
        bulk_load(base + C::kSVs + lane * a.box * 4, a.v_scale + prow, static_cast<uint32_t>(a.box * 4), &full[stg]);
      }
    }
    // after a wait that gave up: the copies in flight land before the CTA may end
    if (k < n)
      for (int i = max(0, k - kStages); i < k; ++i) warp_wait(&full[i % kStages], (i / kStages) & 1, limit_ns, st, 852);
  } else {
    // ------------------------------------------------------------ compute warps
    const int g = lane >> 2, t = lane & 3;
    const int u0 = 16 * warp;
    int8_t* qc = reinterpret_cast<int8_t*>(smem + C::kQc);
    float* qsc = reinterpret_cast<float*>(smem + C::kQs);
    // the query rows: eight lanes a row, D / 32 runs of four channels each
    if (warp < 2) {
      const int c = 4 * warp + (lane >> 3), l8 = lane & 7;
      float x[D / 32][4] = {}, amax = 0.0f;
      if (c < GC) load_runs<D / 32>(a.q, a.q_dtype, (row0 + c) * D + 4 * l8, 32, x);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[i][e]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const RowScale rs = row_scale(amax);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) *reinterpret_cast<uint32_t*>(qc + c * D + 32 * i + 4 * l8) = quant4(x[i], rs);
      if (l8 == 0) qsc[c] = rs.s;
    }
    named_bar_sync(1, kCThreads);
    // B fragments of Q^T: query column g, the 16-byte chunks (8 bytes at d = 32) that the
    // lane reads of the K rows
    constexpr int kH = D >= 64 ? D / 64 : 1;
    uint4 qf[kH];
    if constexpr (D == 32) {
      const uint2 w = *reinterpret_cast<const uint2*>(qc + g * D + 8 * t);
      qf[0] = make_uint4(w.x, w.y, 0u, 0u);
    } else {
#pragma unroll
      for (int h = 0; h < kH; ++h) qf[h] = *reinterpret_cast<const uint4*>(qc + g * D + 64 * h + 16 * t);
    }
    const float log2e_over_sqrtd = 1.4426950408889634f / sqrtf(static_cast<float>(D));
    const float qsa = qsc[2 * t] * log2e_over_sqrtd, qsb = qsc[2 * t + 1] * log2e_over_sqrtd;

    // S^T row r (and r + 8) holds unit token tok(r) (and tok(r) + 8): the permutation that
    // keeps the K and V reads off each other's banks (two ways at d = 64)
    auto tok = [](int r) {
      if constexpr (C::kSwz) return (r >> 1) + 4 * (r & 1);
      if constexpr (D == 32) return (r & 1) ? 4 + (((r >> 1) + 2) & 3) : (r >> 1);
      return (r & 1) ? 4 + ((r >> 1) ^ 1) : (r >> 1);
    };
    const int pi = tok(g);
    uint32_t offk[kH][2];
    if constexpr (D == 32) {
      offk[0][0] = static_cast<uint32_t>((u0 + pi) * 32 + 8 * t);
      offk[0][1] = static_cast<uint32_t>((u0 + pi + 8) * 32 + 8 * t);
    } else {
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        offk[h][0] = ltile_off<D>(u0 + pi, 4 * h + t);
        offk[h][1] = ltile_off<D>(u0 + pi + 8, 4 * h + t);
      }
    }
    // V rows of the lane: unit tokens tok(2t), tok(2t + 1) and the same + 8, chunk pi
    uint32_t offv[C::kBoxes][4];
#pragma unroll
    for (int b = 0; b < C::kBoxes; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int row = u0 + tok(2 * t + (c & 1)) + 8 * (c >> 1);
        offv[b][c] = D == 32   ? static_cast<uint32_t>(row * 32 + 4 * pi)
                     : D == 64 ? static_cast<uint32_t>(row * 64 + 8 * pi)
                               : ltile_off<D>(row, 8 * b + pi);
      }

    float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.0f, l_b = 0.0f;
    float tha = -INFINITY, thb = -INFINITY;  // max + lazy headroom
    float inv_a = pow2i(126), inv_b = inv_a;  // P' carries s_v * 2^-E, inv = 2^-E (see grow_column)
    float vlim = scale_limit(inv_a, inv_b);
    float o[D / 16][4], osum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    for (int k = 0; k < n; ++k) {
      const int stg = k % kStages;
      if (!warp_wait(&full[stg], (k / kStages) & 1, limit_ns, st, 853)) break;
      const uint8_t* base = smem + stg * C::kStageBytes;
      const int nv = t1 - (t0 + k * kTok) - u0;  // valid tokens of this warp's unit
      if (nv > 0) {
        const uint8_t* sk = base + C::kSK;
        const uint8_t* sv = base + C::kSV;
        const float* sks = reinterpret_cast<const float*>(base + C::kSKs);
        const float* svs = reinterpret_cast<const float*>(base + C::kSVs);
        int i0[4] = {0, 0, 0, 0}, i1[4] = {0, 0, 0, 0};
        if constexpr (D == 32) {
          const uint2 wa = *reinterpret_cast<const uint2*>(sk + offk[0][0]);
          const uint2 wb = *reinterpret_cast<const uint2*>(sk + offk[0][1]);
          mma_s8(i0, wa.x, wb.x, wa.y, wb.y, qf[0].x, qf[0].y);
        } else {
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            const uint4 wa = *reinterpret_cast<const uint4*>(sk + offk[h][0]);
            const uint4 wb = *reinterpret_cast<const uint4*>(sk + offk[h][1]);
            mma_s8(i0, wa.x, wb.x, wa.y, wb.y, qf[h].x, qf[h].y);
            mma_s8(i1, wa.z, wb.z, wa.w, wb.w, qf[h].z, qf[h].w);
          }
        }
        const float d00 = static_cast<float>(i0[0] + i1[0]), d01 = static_cast<float>(i0[1] + i1[1]);
        const float d10 = static_cast<float>(i0[2] + i1[2]), d11 = static_cast<float>(i0[3] + i1[3]);
        const int rA = u0 + pi, rB = rA + 8;
        const bool vA = pi < nv, vB = pi + 8 < nv;
        // ---- online softmax (log2 units), lazily rescaled; rows past the list weigh 0,
        // whatever their scales hold
        const float ksA = vA ? sks[rA] : 0.0f, ksB = vB ? sks[rB] : 0.0f;
        const float vsA = vA ? svs[rA] : 0.0f, vsB = vB ? svs[rB] : 0.0f;
        const float xa0 = vA ? d00 * (ksA * qsa) : -INFINITY, xa1 = vA ? d01 * (ksA * qsb) : -INFINITY;
        const float xb0 = vB ? d10 * (ksB * qsa) : -INFINITY, xb1 = vB ? d11 * (ksB * qsb) : -INFINITY;
        const bool grow = (fmaxf(xa0, xb0) > tha) || (fmaxf(xa1, xb1) > thb) || (fmaxf(vsA, vsB) > vlim);
        if (__any_sync(0xffffffffu, grow)) {
          const float fa = grow_column(xa0, xb0, vsA, vsB, m_a, tha, l_a, inv_a);
          const float fb = grow_column(xa1, xb1, vsA, vsB, m_b, thb, l_b, inv_b);
          vlim = scale_limit(inv_a, inv_b);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[j][0] *= fa;
            o[j][2] *= fa;
            o[j][1] *= fb;
            o[j][3] *= fb;
          }
          osum[0] *= fa;
          osum[2] *= fa;
          osum[1] *= fb;
          osum[3] *= fb;
        }
        const float ra = m_a == -INFINITY ? 0.0f : m_a, rb = m_b == -INFINITY ? 0.0f : m_b;
        const float pa0 = ex2(xa0 - ra), pa1 = ex2(xa1 - rb), pb0 = ex2(xb0 - ra), pb1 = ex2(xb1 - rb);
        l_a += pa0 + pb0;
        l_b += pa1 + pb1;
        uint32_t pb0r, pb1r, lo0, lo1;
        weights_f16x2(pa0, pa1, vsA, inv_a, inv_b, pb0r, lo0);
        weights_f16x2(pb0, pb1, vsB, inv_a, inv_b, pb1r, lo1);
        pb0r = movm_t(pb0r);
        pb1r = movm_t(pb1r);
        if constexpr (kFine) {
          lo0 = movm_t(lo0);
          lo1 = movm_t(lo1);
        }
        // ---- O'^T += V_biased^T . P'^T (V codes + 128 as fp16 subnormals), the row sums of
        // P' from an all-ones A for the offset
        auto pv = [&](float (&acc)[4], uint32_t x01, uint32_t x23) {
          x01 ^= 0x80808080u;
          x23 ^= 0x80808080u;
          const uint32_t a0 = prmt(x01, 0u, 0x4140), a1 = prmt(x01, 0u, 0x4342);
          const uint32_t a2 = prmt(x23, 0u, 0x4140), a3 = prmt(x23, 0u, 0x4342);
          mma_f16(acc, a0, a1, a2, a3, pb0r, pb1r);
          if constexpr (kFine) mma_f16(acc, a0, a1, a2, a3, lo0, lo1);
        };
        if constexpr (D == 32) {
          uint32_t w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint32_t*>(sv + offv[0][c]);
          pv(o[0], prmt(w[0], w[1], 0x5140), prmt(w[2], w[3], 0x5140));
          pv(o[1], prmt(w[0], w[1], 0x7362), prmt(w[2], w[3], 0x7362));
        } else if constexpr (D == 64) {
          uint2 w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint2*>(sv + offv[0][c]);
          pv(o[0], prmt(w[0].x, w[1].x, 0x5140), prmt(w[2].x, w[3].x, 0x5140));
          pv(o[1], prmt(w[0].x, w[1].x, 0x7362), prmt(w[2].x, w[3].x, 0x7362));
          pv(o[2], prmt(w[0].y, w[1].y, 0x5140), prmt(w[2].y, w[3].y, 0x5140));
          pv(o[3], prmt(w[0].y, w[1].y, 0x7362), prmt(w[2].y, w[3].y, 0x7362));
        } else {
#pragma unroll
          for (int b = 0; b < C::kBoxes; ++b) {
            uint4 w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint4*>(sv + offv[b][c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w0 = i == 0 ? w[0].x : i == 1 ? w[0].y : i == 2 ? w[0].z : w[0].w;
              const uint32_t w1 = i == 0 ? w[1].x : i == 1 ? w[1].y : i == 2 ? w[1].z : w[1].w;
              const uint32_t w2 = i == 0 ? w[2].x : i == 1 ? w[2].y : i == 2 ? w[2].z : w[2].w;
              const uint32_t w3 = i == 0 ? w[3].x : i == 1 ? w[3].y : i == 2 ? w[3].z : w[3].w;
              pv(o[8 * b + 2 * i], prmt(w0, w1, 0x5140), prmt(w2, w3, 0x5140));
              pv(o[8 * b + 2 * i + 1], prmt(w0, w1, 0x7362), prmt(w2, w3, 0x7362));
            }
          }
        }
        mma_f16(osum, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pb0r, pb1r);
        if constexpr (kFine) mma_f16(osum, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, lo0, lo1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stg]);
    }
    // ---- this warp's state: per query column its max and sum, and
    // O = (2^24 O' - 128 rowsum(P')) * 2^E.  The ring is free once every warp is here.
    l_a = col_sum(l_a);
    l_b = col_sum(l_b);
    m_a = keep_nan(m_a, l_a);
    m_b = keep_nan(m_b, l_b);
    named_bar_sync(1, kCThreads);
    float* stat = reinterpret_cast<float*>(smem + C::kStat);
    float* red = reinterpret_cast<float*>(smem + C::kRed);
    float* wt = reinterpret_cast<float*>(smem + C::kWt);
    float* ml = reinterpret_cast<float*>(smem + C::kMl);
    if (g == 0) {
      *reinterpret_cast<float4*>(stat + (warp * 8 + 2 * t) * 2) = make_float4(m_a, l_a, m_b, l_b);
    }
    const float pea = pow2_inverse(inv_a), peb = pow2_inverse(inv_b);  // 2^E
    constexpr float k2p24 = 16777216.0f;
    const float ca = -128.0f * osum[0], cb = -128.0f * osum[1];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      int dim;  // rows g and g + 8 of m-tile j are channels dim and dim + 1
      if constexpr (D == 32) dim = 4 * pi + 2 * j;
      else if constexpr (D == 64) dim = 8 * pi + 4 * (j >> 1) + 2 * (j & 1);
      else dim = 128 * (j >> 3) + 16 * pi + 4 * ((j & 7) >> 1) + 2 * (j & 1);
      float* r = red + (warp * D + dim) * 8 + 2 * t;
      *reinterpret_cast<float2*>(r) = make_float2(fmaf(o[j][0], k2p24, ca) * pea, fmaf(o[j][1], k2p24, cb) * peb);
      *reinterpret_cast<float2*>(r + 8) = make_float2(fmaf(o[j][2], k2p24, ca) * pea, fmaf(o[j][3], k2p24, cb) * peb);
    }
    named_bar_sync(1, kCThreads);
    if (threadIdx.x < 8 * kWarps) {  // column c: the weight of warp w's state, and (w = 0) max and sum
      const int c = threadIdx.x & 7, w = threadIdx.x >> 3;
      float M = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) M = fmaxf(M, stat[(i * 8 + c) * 2]);
      const float mw = stat[(w * 8 + c) * 2];
      wt[w * 8 + c] = mw == -INFINITY ? 0.0f : ex2(mw - M);
      if (w == 0) {
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float mi = stat[(i * 8 + c) * 2];
          if (mi != -INFINITY) sum = fmaf(ex2(mi - M), stat[(i * 8 + c) * 2 + 1], sum);
        }
        ml[c] = M;
        ml[8 + c] = sum;
      }
    }
    named_bar_sync(1, kCThreads);
    // ---- the CTA's O over its warps: unit u = (channel u % D, columns 4 (u / D) ..)
    for (int u = threadIdx.x; u < 2 * D; u += kCThreads) {
      const int dim = u % D, h = u / D;
      if (4 * h >= GC) continue;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 r = *reinterpret_cast<const float4*>(red + (w * D + dim) * 8 + 4 * h);
        const float4 f = *reinterpret_cast<const float4*>(wt + w * 8 + 4 * h);
        acc.x = fmaf(r.x, f.x, acc.x);
        acc.y = fmaf(r.y, f.y, acc.y);
        acc.z = fmaf(r.z, f.z, acc.z);
        acc.w = fmaf(r.w, f.w, acc.w);
      }
      const float x[4] = {acc.x, acc.y, acc.z, acc.w};
      if (S > 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) reinterpret_cast<float*>(smem + C::kPart)[(4 * h + c) * D + dim] = x[c];
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float l = ml[8 + 4 * h + c];
          if (4 * h + c < GC)
            store_out(a.out, a.out_dtype, (row0 + 4 * h + c) * D + dim, l == 0.0f ? 0.0f : x[c] / l);
        }
      }
    }
    if (S == 1 && a.lse && threadIdx.x < GC) {
      const float l = ml[8 + threadIdx.x];
      a.lse[row0 + threadIdx.x] = l == 0.0f ? -INFINITY : (ml[threadIdx.x] + log2f(l)) * 0.6931471805599453f;
    }
  }
  if (S == 1) return;

  // ---- merge the S parts: each CTA takes every S-th run of (column, channel) units
  cluster.sync();
  for (int u = rank * kThreads + threadIdx.x; u < GC * D; u += S * kThreads) {
    const int c = u / D, dim = u % D;
    float m[kMaxSplits], l[kMaxSplits], x[kMaxSplits];  // all on their way at once
#pragma unroll
    for (int r = 0; r < kMaxSplits; ++r) {
      if (r < S) {
        const float* peer = reinterpret_cast<const float*>(cluster.map_shared_rank(smem, r));
        m[r] = peer[C::kMl / 4 + c];
        l[r] = peer[C::kMl / 4 + 8 + c];
        x[r] = peer[C::kPart / 4 + c * D + dim];
      }
    }
    float M = -INFINITY, sum = 0.0f, acc = 0.0f;
#pragma unroll
    for (int r = 0; r < kMaxSplits; ++r)
      if (r < S) M = fmaxf(M, m[r]);
#pragma unroll
    for (int r = 0; r < kMaxSplits; ++r) {
      if (r < S && m[r] != -INFINITY) {
        const float f = ex2(m[r] - M);
        sum = fmaf(f, l[r], sum);
        acc = fmaf(f, x[r], acc);
      }
    }
    store_out(a.out, a.out_dtype, (row0 + c) * D + dim, sum == 0.0f ? 0.0f : acc / sum);
    if (a.lse && dim == 0) a.lse[row0 + c] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
  }
  cluster.sync();  // no CTA leaves while another reads its part
}

template <int D, int kCtas, bool kFine>
cudaError_t launch_list_f(const ListDecodeArgs& a, cudaStream_t s) {
  using C = LCfg<D, kCtas>;
  auto kern = list_decode_kernel<D, kCtas, kFine>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), C::kBytes);
  if (e != cudaSuccess) return e;
  bool ok = true;
  const uint64_t rows = static_cast<uint64_t>(a.num_pages) * a.Hkv * a.page;
  const CUtensorMap km = make_tmap_3d(a.k_pages, CU_TENSOR_MAP_DATA_TYPE_UINT8, D, rows, 1, D, rows * D, C::kBW, a.box, 1,
                                      &ok, C::kSwz);
  const CUtensorMap vm = make_tmap_3d(a.v_pages, CU_TENSOR_MAP_DATA_TYPE_UINT8, D, rows, 1, D, rows * D, C::kBW, a.box, 1,
                                      &ok, C::kSwz);
  if (!ok) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * a.Hkv * a.groups * a.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, km, vm, device_status_ptr(), spin_limit_ns());
}

template <int D, int kCtas>
cudaError_t launch_list_d(const ListDecodeArgs& a, cudaStream_t s) {
  return a.out_dtype == SL8_F32 ? launch_list_f<D, kCtas, true>(a, s) : launch_list_f<D, kCtas, false>(a, s);
}

}  // namespace

int list_decode_max_splits() { return kMaxSplits; }

int list_decode_splits(int64_t lists, int64_t tokens, int32_t d) {
  const int64_t fit = list_ctas(d) * static_cast<int64_t>(num_sms());
  // few long lists: clusters of kMaxSplits CTAs would leave SMs without work (8 lists of
  // 65,536 tokens, d = 128: 81 us with 8 splits, 51 with 32; 1 list: 80 and 26 with 64)
  if (lists * kMaxSplits < num_sms() && tokens >= 4096 * kMaxSplits)
    return static_cast<int>(std::max<int64_t>(kMaxSplits + 1, std::min<int64_t>(64, 256 / lists)));
  // else as many splits as fit one wave, of 128 tokens at least
  int n = 1;
  while (n < kMaxSplits && lists * (n + 1) <= fit && tokens / (n + 1) >= 128) ++n;
  return n;
}

cudaError_t launch_list_decode(const ListDecodeArgs& args, int32_t d, cudaStream_t s) {
  TraceScope tr("list_decode", s);
  ListDecodeArgs a = args;
  // rows per TMA box: the largest of a stage's 64, 32 or 16 that divides the page, so that
  // no piece straddles two pages
  a.box = a.page % 64 == 0 ? 64 : a.page % 32 == 0 ? 32 : 16;
  // list_ctas(d) CTAs an SM or one more, whichever fills its last wave better: d = 128, 512 lists
  // of 4,096 tokens take 110 us with three and 87.5 with four, 512 of 1,024 tokens 35 and 27; 768
  // lists of 2,048 tokens 72 and 82, 448 of 4,096 76 and 74.  d = 64, 720 lists of 4,096 tokens:
  // 102 with four, 77 with five; 600 of them 61.4 and 62.5.
  const int64_t ctas = static_cast<int64_t>(a.rows) * a.Hkv * a.groups * a.splits;
  const int64_t w = static_cast<int64_t>(list_ctas(d)) * num_sms(), w1 = w + num_sms();
  const bool more = a.splits == 1 && ctas > w && (ctas + w1 - 1) / w1 * w1 < (ctas + w - 1) / w * w;
  switch (d) {
    case 32: return launch_list_d<32, list_ctas(32)>(a, s);
    case 64: return more ? launch_list_d<64, list_ctas(64) + 1>(a, s) : launch_list_d<64, list_ctas(64)>(a, s);
    case 128: return more ? launch_list_d<128, list_ctas(128) + 1>(a, s) : launch_list_d<128, list_ctas(128)>(a, s);
    case 256: return launch_list_d<256, list_ctas(256)>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sl8
