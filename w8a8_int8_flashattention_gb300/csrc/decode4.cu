// Decode attention over the paged 4-bit cache (rows as in cache4.cuh), for sm_103a: single queries
// and up to 32 drafts a sequence, causal or with tree masks.
//   x_t = s_q * sum_g s_k[t, g] * int32(q_i8[g] . c_k[t, g]) / sqrt(d),  p = softmax(x),
//   O   = sum_t p_t * s_v[t, g] * c_v[t]
// over the tokens t that the query sees, g the groups of 32 channels.
//
// GB300 design.  A column is one query row of a kv head: a draft and a query head.  A CTA takes
// up to 16 columns of one (sequence, kv head) and a contiguous run of its tokens; a cluster of S
// CTAs, or more with a combine, share a sequence.
//  * Four warps, each on its own: units of 16 tokens, taken in turn, arrive by 16-byte cp.async in a ring of the
//    warp's own, so that no warp waits for another before the end.  Page ids are read 32 units ahead.
//  * S[16 columns x 16 tokens] = Q K^T as fp16 m16n8k16 MMAs: a 4-bit code is or-ed into the
//    mantissa of 1024 (or, where it lies four bits higher, 16 times as much, against q / 16),
//    and what that adds, 1032 and 72 times the q's, is in the accumulator from the start: all are
//    integers below 2^23, so that the group's integer product is exact.  Each group's product meets its scale in fp32.
//  * O^T[d x 8 columns] += V^T P^T as bf16 MMAs: ldmatrix.trans hands each lane the four nibbles of
//    two tokens' channels, which are codes of bf16 after an or and a subtraction, both exact.  The weights p * s_v
//    of a group are a sum of bf16 terms, two (2^-17 of themselves left over; 16-bit outputs) or three (fp32).  They have
//    fp32's range, so that no scale, however far from the others, costs another one its bits.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "cache4.cuh"
#include "decode_unit.cuh"
#include "sl8_internal.h"

namespace cg = cooperative_groups;

namespace sl8 {

namespace {

constexpr int kMaxCluster = 8;  // CTAs of a cluster (portable)
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kUnit = 16;  // tokens that a warp takes at a time

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t a, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm2_t(uint32_t a, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(a) : "memory");
}
// d = a b + c in fp16 with fp32 sums.
__device__ __forceinline__ void mma_f16_from(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two nibbles (bits 0..3 of each half) as bf16 codes: 128 + n, less 136.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"((w & 0x000f000fu) | 0x43004300u), "r"(0x43084308u));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int kCols>
struct Cfg4 {
  static constexpr int kN = D / kGroup4;                  // groups (and 16-byte chunks) of a row
  static constexpr int kK = 0, kV = 8 * D, kKs = 16 * D, kVs = 17 * D, kUnitBytes = 18 * D;
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? (kCols == 8 ? 4 : 5) : D == 64 ? 6 : 8;
  static constexpr int kCtas = D == 256 ? 3 : D == 128 ? (kCols == 8 ? 4 : 3) : D == 64 ? (kCols == 8 ? 5 : 4) : 5;
  static constexpr int kRing = kWarps * kStages * kUnitBytes;
  // after the loop the ring holds the warps' O^T [warp][D][kCols] and the CTA's [kCols][D], fp32
  static constexpr int kRed = 0, kPart = kWarps * D * kCols * 4;
  static_assert(kPart + kCols * D * 4 <= kRing, "the merge fits the ring");
  static constexpr int kQc = kRing;                       // [kCols][D] query codes
  static constexpr int kQs = kQc + kCols * D;             // [kCols] scales
  static constexpr int kStat = kQs + kCols * 4;           // [warp][kCols][2]: max (log2), sum
  static constexpr int kWt = kStat + kWarps * kCols * 8;  // [warp][kCols] weights of the warps
  static constexpr int kMl = kWt + kWarps * kCols * 4;    // [kCols] max, [kCols] sum of the CTA
  static constexpr int kBytes = kMl + kCols * 8;
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "kCtas CTAs fit an SM");
};

// Row of a unit's tile in shared memory that token tau has: tokens 4 t, 4 t + 1 and 4 t + 2,
// 4 t + 3 of lane t's quad are rows 2 t, 2 t + 1 of the two halves, so that a lane's accumulators are four
// tokens in a row.
__device__ __forceinline__ int row_of(int tau) { return ((tau >> 1) & 1) * 8 + (tau >> 2) * 2 + (tau & 1); }
// Byte offset of chunk j of row r: eight rows' chunks j lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int r, int j) {
  constexpr int n = D / kGroup4, m = 8 / n;  // chunks of a row, rows in 128 bytes
  return static_cast<uint32_t>(r * (16 * n) + 16 * (j ^ (((r & 7) / m) & (n - 1))));
}

// kCols: 8 or 16 columns.  kTerms: bf16 terms of a weight.
template <int D, int kCols, int kTerms>
__global__ void __launch_bounds__(kThreads, Cfg4<D, kCols>::kCtas)
    decode4_kernel(const Decode4Args a, DeviceStatus* st) {
  using C = Cfg4<D, kCols>;
  constexpr int kN = C::kN, kStages = C::kStages, kH = kCols / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const bool clustered = a.splits <= kMaxCluster;
  const int S = a.splits;
  const unsigned item = blockIdx.x / static_cast<unsigned>(S);
  const int rank = static_cast<int>(blockIdx.x - item * S);
  const unsigned bh = item / static_cast<unsigned>(a.groups);
  const int b = static_cast<int>(bh / static_cast<unsigned>(a.Hkv)), head = static_cast<int>(bh - static_cast<unsigned>(b) * a.Hkv);
  const int G = a.Hq / a.Hkv;
  const int col0 = static_cast<int>(item - bh * a.groups) * a.cols;  // first of this CTA's columns
  const int GC = min(a.cols, a.T * G - col0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // row of q and out that column c stands for: its draft, its query head
  auto row_at = [&](int c) {
    const int dr = (col0 + c) / G;
    return (static_cast<int64_t>(b) * a.T + dr) * a.Hq + head * G + (col0 + c - dr * G);
  };

  int L = a.seqlens[b];
  const int cap = a.max_blocks * a.page;
  if (L < 0 || L > cap) {
    if (threadIdx.x == 0) record_status(st, kStatusBadArg, 870);
    L = L < 0 ? 0 : cap;
  }
  // this CTA's units of the sequence, [u0, u1); this warp's are u0 + warp, u0 + warp + 4, ...
  const int n_all = (L + kUnit - 1) / kUnit;  // below 2^27
  const int u0 = static_cast<int>(static_cast<int64_t>(n_all) * rank / S);
  const int u1 = static_cast<int>(static_cast<int64_t>(n_all) * (rank + 1) / S);
  const int n = max(0, (u1 - u0 - warp + kWarps - 1) / kWarps);
  const int first = u0 + warp;

  // ------------------------------------------------------------ loads
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_blocks;
  auto ids_at = [&](int k) { return k + lane < n ? table[(first + (k + lane) * kWarps) * kUnit / a.page] : 0; };
  int32_t ids = ids_at(0), next_ids = n > 32 ? ids_at(32) : 0;
  const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * kStages * C::kUnitBytes);
  // the lane's chunks of a unit: K's and V's 16 kN, then the scales' 2 kN each
  constexpr int kChunks = 16 * kN, kPer = kChunks >= 32 ? kChunks / 32 : 1;
  auto issue = [&](int k) {  // unit k of this warp
    if (k < n) {
      if (k > 0 && k % 32 == 0) {
        ids = next_ids;
        next_ids = ids_at(k + 32);
      }
      int32_t pg = __shfl_sync(0xffffffffu, ids, k & 31);
      if (pg < 0 || pg >= a.num_pages) {
        if (lane == 0) record_status(st, kStatusBadArg, 871);
        pg = 0;
      }
      const int64_t row = (static_cast<int64_t>(pg) * a.Hkv + head) * a.page + (first + k * kWarps) * kUnit % a.page;
      const uint32_t base = ring + static_cast<uint32_t>(k % kStages * C::kUnitBytes);
      const uint8_t* ksrc = a.k_pages + row * (D / 2);
      const uint8_t* vsrc = a.v_pages + row * (D / 2);
      if constexpr (kChunks >= 32) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int c = lane + 32 * i;
          const uint32_t dst = base + chunk_off<D>(row_of(c / kN), c % kN);
          cp_async16(dst + C::kK, ksrc + 16 * c);
          cp_async16(dst + C::kV, vsrc + 16 * c);
        }
      } else {
        const int c = lane & 15;
        cp_async16(base + (lane < 16 ? C::kK : C::kV) + chunk_off<D>(row_of(c), 0), (lane < 16 ? ksrc : vsrc) + 16 * c);
      }
      if (lane < 4 * kN) {  // scales: 32 kN bytes each
        const int c = lane % (2 * kN);
        const uint16_t* src = lane < 2 * kN ? a.k_scale : a.v_scale;
        cp_async16(base + (lane < 2 * kN ? C::kKs : C::kVs) + 16 * c, reinterpret_cast<const uint8_t*>(src + row * kN) + 16 * c);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue(k);

  // ------------------------------------------------------------ the query columns: eight lanes a row
  int8_t* qc = reinterpret_cast<int8_t*>(smem + C::kQc);
  float* qsc = reinterpret_cast<float*>(smem + C::kQs);
  if (4 * warp < kCols) {
    const int c = 4 * warp + (lane >> 3), l8 = lane & 7;
    float x[D / 32][4] = {}, amax = 0.0f;
    if (c < GC) load_runs<D / 32>(a.q, a.q_dtype, row_at(c) * D + 4 * l8, 32, x);
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
  __syncthreads();
  // A fragments: rows g and g + 8 are columns; word t of a group's chunk holds channels 8 t .. 8 t + 7,
  // of which the even ones meet one MMA, the odd ones (whose nibbles stand 16 times as high) another
  uint32_t qa[kN][2][2 * kH];
  float bias[kN][4];
  float qs[kH];
  uint32_t seen[kH];  // drafts that the column sees
#pragma unroll
  for (int h = 0; h < kH; ++h) {
    const int c = g + 8 * h;
    qs[h] = qsc[c] * (1.4426950408889634f / sqrtf(static_cast<float>(D)));
    const int dr = c < GC ? (col0 + c) / G : 0;
    seen[h] = a.mask ? a.mask[static_cast<int64_t>(b) * a.T + dr] : 0xffffffffu >> (31 - dr);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const uint2 w = *reinterpret_cast<const uint2*>(qc + c * D + 32 * j + 8 * t);
      float x[8];
      float even = 0.0f, odd = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = static_cast<float>(static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3))));
        if (i & 1) odd += x[i], x[i] *= 0.0625f;
        else even += x[i];
      }
      qa[j][0][h] = f16x2_of(x[0], x[4]);
      qa[j][0][kH + h] = f16x2_of(x[2], x[6]);
      qa[j][1][h] = f16x2_of(x[1], x[5]);
      qa[j][1][kH + h] = f16x2_of(x[3], x[7]);
      float f = -(1032.0f * even + 72.0f * odd);
      f += __shfl_xor_sync(0xffffffffu, f, 1);
      f += __shfl_xor_sync(0xffffffffu, f, 2);
      bias[j][2 * h] = bias[j][2 * h + 1] = f;
      if (kH == 1) bias[j][2] = bias[j][3] = 0.0f;
    }
  }

  // ------------------------------------------------------------ the tokens
  const int lr = lane & 7, lm = lane >> 3;  // ldmatrix: row and matrix that the lane's address is for
  float m[kH], th[kH], l[kH];
  float o[D / 16][kH][4];
#pragma unroll
  for (int h = 0; h < kH; ++h) m[h] = th[h] = -INFINITY, l[h] = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int h = 0; h < kH; ++h) o[i][h][0] = o[i][h][1] = o[i][h][2] = o[i][h][3] = 0.0f;
  const int base_tok = L - a.T;  // position of the first draft

  auto unit = [&](uint32_t base, int tok, auto masked) {
    constexpr bool kMasked = decltype(masked)::value;
    // the lane's tokens tok + 4 t + i; seen or not by each of its columns
    bool vis[kH][4];
    if constexpr (kMasked) {
#pragma unroll
      for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = tok + 4 * t + i;
          vis[h][i] = p < base_tok || (p < L && ((seen[h] >> (p - base_tok)) & 1u));
        }
    }
    // ---- logits
    uint32_t kw[2][kN];
    if constexpr (kN == 1) {
      ldsm2(base + C::kK + chunk_off<D>(8 * (lm & 1) + lr, 0), kw[0][0], kw[1][0]);
    } else if constexpr (kN == 2) {
      ldsm4(base + C::kK + chunk_off<D>(8 * (lm >> 1) + lr, lm & 1), kw[0][0], kw[0][1], kw[1][0], kw[1][1]);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < kN; j += 4)
          ldsm4(base + C::kK + chunk_off<D>(8 * s + lr, lm + j), kw[s][j], kw[s][j + 1], kw[s][j + 2], kw[s][j + 3]);
    }
    float ks[4][kN];
    auto scales_at = [&](uint32_t off, float (&f)[4][kN]) {
      uint32_t w[2 * kN];
      const uint8_t* p = smem + (base - smem_u32(smem)) + off + 8 * kN * t;
#pragma unroll
      for (int i = 0; i < 2 * kN; i += 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p + 4 * i);
        w[i] = v.x, w[i + 1] = v.y;
      }
#pragma unroll
      for (int i = 0; i < 4 * kN; ++i) f[i / kN][i % kN] = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    };
    scales_at(C::kKs, ks);
    float x[kH][4] = {};
#pragma unroll
    for (int j = 0; j < kN; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t w0 = kw[s][j], w8 = w0 >> 8;
        float acc[4];
        mma_f16_from(acc, bias[j], qa[j][0][0], kH == 2 ? qa[j][0][1] : 0u, qa[j][0][kH], kH == 2 ? qa[j][0][3] : 0u,
                     (w0 & 0x000f000fu) | 0x64006400u, (w8 & 0x000f000fu) | 0x64006400u);
        mma_f16(acc, qa[j][1][0], kH == 2 ? qa[j][1][1] : 0u, qa[j][1][kH], kH == 2 ? qa[j][1][3] : 0u,
                (w0 & 0x00f000f0u) | 0x64006400u, (w8 & 0x00f000f0u) | 0x64006400u);
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) x[h][2 * s + i] = fmaf(acc[2 * h + i], ks[2 * s + i][j], x[h][2 * s + i]);
      }
    // ---- online softmax (log2 units), lazily rescaled
    bool grow = false;
#pragma unroll
    for (int h = 0; h < kH; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[h][i] *= qs[h];
        if constexpr (kMasked) x[h][i] = vis[h][i] ? x[h][i] : -INFINITY;
      }
      grow = grow || fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3])) > th[h];
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        float mx = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        float f = 1.0f;
        if (mx > th[h]) {
          f = ex2(m[h] - mx);
          m[h] = mx;
          th[h] = mx + kLazy;
          l[h] *= f;
        }
        const float fa = __shfl_sync(0xffffffffu, f, 8 * t), fb = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][h][0] *= fa;
          o[i][h][1] *= fb;
          o[i][h][2] *= fa;
          o[i][h][3] *= fb;
        }
      }
    }
    float p[kH][4];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      const float ref = m[h] == -INFINITY ? 0.0f : m[h];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[h][i] = ex2(x[h][i] - ref);
        l[h] += p[h][i];
      }
    }
    // ---- output
    uint32_t vw[2][kN];
    if constexpr (kN == 1) {
      ldsm2_t(base + C::kV + chunk_off<D>(8 * (lm & 1) + lr, 0), vw[0][0], vw[1][0]);
    } else if constexpr (kN == 2) {
      ldsm4_t(base + C::kV + chunk_off<D>(8 * (lm >> 1) + lr, lm & 1), vw[0][0], vw[0][1], vw[1][0], vw[1][1]);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < kN; j += 4)
          ldsm4_t(base + C::kV + chunk_off<D>(8 * s + lr, lm + j), vw[s][j], vw[s][j + 1], vw[s][j + 2], vw[s][j + 3]);
    }
    float vs[4][kN];
    scales_at(C::kVs, vs);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      uint32_t wt[kH][kTerms][2];
#pragma unroll
      for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float w0 = p[h][2 * s] * vs[2 * s][j], w1 = p[h][2 * s + 1] * vs[2 * s + 1][j];
          if constexpr (kMasked) {  // whatever the scales of rows that are not seen hold
            w0 = vis[h][2 * s] ? w0 : 0.0f;
            w1 = vis[h][2 * s + 1] ? w1 : 0.0f;
          }
#pragma unroll
          for (int e = 0; e < kTerms; ++e) {
            const uint32_t r = bf16x2_of(w0, w1);
            wt[h][e][s] = r;
            w0 -= __uint_as_float(r << 16);
            w1 -= __uint_as_float(r & 0xffff0000u);
          }
        }
#pragma unroll
      for (int y = 0; y < 2; ++y) {  // channels 32 j + 4 g + 2 y and + 1
        const uint32_t a0 = codes_bf16x2(vw[0][j] >> (8 * y)), a1 = codes_bf16x2(vw[0][j] >> (8 * y + 4));
        const uint32_t a2 = codes_bf16x2(vw[1][j] >> (8 * y)), a3 = codes_bf16x2(vw[1][j] >> (8 * y + 4));
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int e = 0; e < kTerms; ++e) mma_bf16(o[2 * j + y][h], a0, a1, a2, a3, wt[h][e][0], wt[h][e][1]);
      }
    }
  };

  for (int k = 0; k < n; ++k) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue(k + kStages - 1);  // into the stage that the last iteration read
    const uint32_t base = ring + static_cast<uint32_t>(k % kStages * C::kUnitBytes);
    const int tok = (first + k * kWarps) * kUnit;
    if (tok + kUnit > base_tok) unit(base, tok, std::true_type{});
    else unit(base, tok, std::false_type{});
    __syncwarp();
  }
  cp_async_wait<0>();

  // ------------------------------------------------------------ the CTA's state from its warps'
  float* stat = reinterpret_cast<float*>(smem + C::kStat);
  float* red = reinterpret_cast<float*>(smem + C::kRed);
  float* wt = reinterpret_cast<float*>(smem + C::kWt);
  float* ml = reinterpret_cast<float*>(smem + C::kMl);
  float* part = reinterpret_cast<float*>(smem + C::kPart);
  __syncthreads();  // the rings are free
#pragma unroll
  for (int h = 0; h < kH; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    m[h] = keep_nan(m[h], l[h]);
    if (t == 0) *reinterpret_cast<float2*>(stat + (warp * kCols + g + 8 * h) * 2) = make_float2(m[h], l[h]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {  // rows g and g + 8 of tile i
      float* r = red + (warp * D + 16 * i + g) * kCols + 8 * h + 2 * t;
      *reinterpret_cast<float2*>(r) = make_float2(o[i][h][0], o[i][h][1]);
      *reinterpret_cast<float2*>(r + 8 * kCols) = make_float2(o[i][h][2], o[i][h][3]);
    }
  }
  __syncthreads();
  if (threadIdx.x < kCols * kWarps) {  // column c: the weight of warp w's state, and (w = 0) max and sum
    const int c = threadIdx.x % kCols, w = threadIdx.x / kCols;
    float M = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) M = fmaxf(M, stat[(i * kCols + c) * 2]);
    const float mw = stat[(w * kCols + c) * 2];
    wt[w * kCols + c] = mw == -INFINITY ? 0.0f : ex2(mw - M);
    if (w == 0) {
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float mi = stat[(i * kCols + c) * 2];
        if (mi != -INFINITY) sum = fmaf(ex2(mi - M), stat[(i * kCols + c) * 2 + 1], sum);
      }
      ml[c] = M;
      ml[kCols + c] = sum;
    }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < D * (kCols / 4); u += kThreads) {  // row u % D, columns 4 (u / D) ..
    const int r = u % D, q4 = u / D;
    const int dim = 32 * (r >> 5) + 4 * (r & 7) + 2 * ((r >> 4) & 1) + ((r >> 3) & 1);
    if (4 * q4 >= GC) continue;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(red + (w * D + r) * kCols + 4 * q4);
      const float4 f = *reinterpret_cast<const float4*>(wt + w * kCols + 4 * q4);
      acc.x = fmaf(v.x, f.x, acc.x);
      acc.y = fmaf(v.y, f.y, acc.y);
      acc.z = fmaf(v.z, f.z, acc.z);
      acc.w = fmaf(v.w, f.w, acc.w);
    }
    part[(4 * q4 + 0) * D + dim] = acc.x;
    part[(4 * q4 + 1) * D + dim] = acc.y;
    part[(4 * q4 + 2) * D + dim] = acc.z;
    part[(4 * q4 + 3) * D + dim] = acc.w;
  }

  if (!clustered) {  // to the workspace, for the combine
    __syncthreads();
    for (int u = threadIdx.x; u < GC * D; u += kThreads) {
      const int c = u / D;
      a.part_o[(row_at(c) * S + rank) * D + u % D] = part[u];
      if (u % D == 0) a.part_ml[row_at(c) * S + rank] = make_float2(ml[c], ml[kCols + c]);
    }
    return;
  }
  // ------------------------------------------------------------ merge the S parts of the cluster
  if (S > 1) cluster.sync();
  else __syncthreads();
  for (int u = rank * kThreads + threadIdx.x; u < GC * D; u += S * kThreads) {
    const int c = u / D, dim = u % D;
    float mr[kMaxCluster], lr2[kMaxCluster], x[kMaxCluster];  // all on their way at once
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r < S) {
        const float* peer = reinterpret_cast<const float*>(S > 1 ? cluster.map_shared_rank(smem, r) : smem);
        mr[r] = peer[C::kMl / 4 + c];
        lr2[r] = peer[C::kMl / 4 + kCols + c];
        x[r] = peer[C::kPart / 4 + c * D + dim];
      }
    }
    float M = -INFINITY, sum = 0.0f, acc = 0.0f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < S) M = fmaxf(M, mr[r]);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r < S && mr[r] != -INFINITY) {
        const float f = ex2(mr[r] - M);
        sum = fmaf(f, lr2[r], sum);
        acc = fmaf(f, x[r], acc);
      }
    }
    const int64_t row = row_at(c);
    store_out(a.out, a.out_dtype, row * D + dim, sum == 0.0f ? 0.0f : acc / sum);
    if (a.lse && dim == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
  }
  if (S > 1) cluster.sync();  // no CTA leaves while another reads its part
}

// The S parts of each row from the workspace: one warp a row and 32 channels.
template <int D>
__global__ void __launch_bounds__(128) decode4_combine_kernel(const Decode4Args a, int64_t rows) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t row = w / (D / 32);
  if (row >= rows) return;
  const int dim = static_cast<int>(w % (D / 32)) * 32 + lane;
  const float2* ml = a.part_ml + row * a.splits;
  float M = -INFINITY;
  for (int r = lane; r < a.splits; r += 32) M = fmaxf(M, ml[r].x);
  M = warp_max_f(M);
  float sum = 0.0f, acc = 0.0f;
#pragma unroll 4
  for (int r = 0; r < a.splits; ++r) {
    const float2 v = ml[r];
    const float x = a.part_o[(row * a.splits + r) * D + dim];
    if (v.x != -INFINITY) {
      const float f = ex2(v.x - M);
      sum = fmaf(f, v.y, sum);
      acc = fmaf(f, x, acc);
    }
  }
  store_out(a.out, a.out_dtype, row * D + dim, sum == 0.0f ? 0.0f : acc / sum);
  if (a.lse && dim == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

template <int D, int kCols, int kTerms>
cudaError_t launch_t(const Decode4Args& a, cudaStream_t s) {
  using C = Cfg4<D, kCols>;
  auto kern = decode4_kernel<D, kCols, kTerms>;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), C::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.Hkv * a.groups * a.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.splits <= kMaxCluster ? a.splits : 1;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, device_status_ptr());
}

template <int D, int kCols>
cudaError_t launch_c(const Decode4Args& a, cudaStream_t s) {
  return a.out_dtype == SL8_F32 ? launch_t<D, kCols, 3>(a, s) : launch_t<D, kCols, 2>(a, s);
}

template <int D>
cudaError_t launch_d(const Decode4Args& a, cudaStream_t s) {
  cudaError_t e;
  if constexpr (D == 256) e = launch_c<D, 8>(a, s);
  else e = a.cols > 8 ? launch_c<D, 16>(a, s) : launch_c<D, 8>(a, s);
  if (e != cudaSuccess || a.splits <= kMaxCluster) return e;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.Hq;
  const unsigned grid = static_cast<unsigned>((rows * (D / 32) + 3) / 4);
  return launch_pdl(decode4_combine_kernel<D>, dim3(grid), dim3(128), 0, s, a, rows);
}

}  // namespace

int decode4_max_cluster() { return kMaxCluster; }
int32_t decode4_max_columns(int32_t d) { return d == 256 ? 8 : 16; }

int decode4_splits(int64_t items, int64_t tokens, int32_t d) {
  const int64_t fit = 4 * static_cast<int64_t>(num_sms());
  if (items * kMaxCluster < num_sms() && tokens >= 4096 * kMaxCluster)
    return static_cast<int>(std::max<int64_t>(kMaxCluster + 1, std::min<int64_t>(64, fit / items)));
  int n = 1;
  while (n < kMaxCluster && items * (n + 1) <= fit && tokens / (n + 1) >= 128) ++n;
  return n;
}

cudaError_t launch_decode4(const Decode4Args& a, int32_t d, cudaStream_t s) {
  TraceScope tr("decode_int4", s);
  switch (d) {
    case 32: return launch_d<32>(a, s);
    case 64: return launch_d<64>(a, s);
    case 128: return launch_d<128>(a, s);
    case 256: return launch_d<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sl8
