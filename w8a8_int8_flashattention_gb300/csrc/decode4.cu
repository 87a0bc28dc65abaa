// Decode attention over the paged 4-bit cache (rows as in cache4.cuh), for sm_103a: single queries
// and up to 32 drafts a sequence, causal or with tree masks.
//   x_t = s_q * sum_g s_k[t, g] * int32(q_i8[g] . c_k[t, g]) / sqrt(d),  p = softmax(x),
//   O   = sum_t p_t * s_v[t, g] * c_v[t]
// over the tokens t that the query sees, g the groups of 32 channels.
//
// GB300 design.  A column is one query row of a kv head: a draft and a query head.  A CTA takes
// up to 16 columns of one (sequence, kv head) and a contiguous run of its tokens; a cluster of S
// CTAs, or more with a combine, share a sequence.
//  * Four warps, each on its own: units of 16 tokens, taken in turn, arrive by 16-byte cp.async in a ring of
//    the warp's own, so that no warp waits for another before the end.  Page ids are read 32 units ahead.
//  * S[16 tokens x 8 columns] = K Q^T as fp16 m16n8k16 MMAs on the nibbles where they lie, which are
//    fp16 subnormals, n 2^-24 (or, four bits higher, 16 times that, against q / 16); 8 times the sum of the
//    q's comes off again.  All partial sums are whole multiples of 2^-24 below 2^17 of them, so that a
//    group's integer product is exact.  It meets its scale in fp32.  (The int8 MMA that would take the codes as
//    they are takes 17 cycles an SM on this part, where the fp16 one takes 2 and does half; e4m3
//    operands, in which nibbles are numbers too, are converted to fp16 one by one.)
//  * O^T[d x 8 columns] += V^T P^T as bf16 MMAs: ldmatrix.trans hands each lane the four nibbles of
//    two tokens' channels; where they lie they are bf16 numbers too, and one fma makes codes of them.  The
//    weights p * s_v of a group are sums of bf16 terms, two (2^-17 of themselves left over; 16-bit
//    outputs) or three (fp32).  They have fp32's range, so that no scale, however far from the
//    others, costs another one its bits.
//  * The logits of the next unit are computed beside the output of this one, so that neither
//    chain waits alone; the units that end behind the first draft, at most one a warp, come last, with masks.
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

// N 16-bit values from shared memory, as words (N = 1: in the low half).
template <int N, int M>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[M]) {
  if constexpr (N == 1) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    w[0] = v;
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a) : "memory");
  } else if constexpr (N == 4) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; i += 4)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]) : "r"(a + 4 * i) : "memory");
  }
}
__device__ __forceinline__ void cp_async16_if(bool on, uint32_t dst, const void* src) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst), "l"(src),
               "r"(static_cast<uint32_t>(on))
               : "memory");
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
// d = a b in fp16 with fp32 sums, and d += a b.
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// (x0, x1) += (a0, a1) in fp32, as one instruction.
__device__ __forceinline__ void add_pair(float& x0, float& x1, float a0, float a1) {
  asm("{\n\t.reg .b64 x, a;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tadd.rn.f32x2 x, x, a;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a0), "f"(a1));
}
// Nibbles where they lie in a 16-bit word are bf16 numbers, n 2^-133 (bits 0..3) and n 2^-129
// (bits 4..7, since the exponents 0 and 1 have the same step): times 2^127 and less 8 such, codes.
constexpr uint32_t k2p127 = 0x7f007f00u, kLow8 = 0xbe00be00u, kHigh8 = 0xc000c000u;  // 2^127, -8 2^-6, -8 2^-2
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int kCols>
struct Cfg4 {
  static constexpr int kN = D / kGroup4;                  // groups (and 16-byte chunks) of a row
  static constexpr int kK = 0, kV = 8 * D, kKs = 16 * D, kVs = 17 * D, kUnitBytes = 18 * D;
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? 5 : D == 64 ? 6 : 8;
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
  constexpr int kN = C::kN, kStages = C::kStages, kT = kCols / 8;  // tiles of eight columns
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
  // the sixteenth of a row index at which unit k + lane lies
  auto rows_at = [&](int k) -> uint32_t {
    if (k + lane >= n) return 0;
    const int tok = (first + (k + lane) * kWarps) * kUnit, blk = tok / a.page;
    int32_t pg = table[blk];
    if (pg < 0 || pg >= a.num_pages) {
      record_status(st, kStatusBadArg, 871);
      pg = 0;
    }
    return (static_cast<uint32_t>(pg) * a.Hkv + head) * (a.page / kUnit) + (tok - blk * a.page) / kUnit;
  };
  uint32_t rows = rows_at(0), next_rows = n > 32 ? rows_at(32) : 0;
  // The lane's chunks of a unit: c0, c0 + 32, ... of K's and V's 16 kN, then one of the scales' 2 kN each.
  // 32 chunks further is 512 bytes further, at d = 256 (four rows) with another swizzle.
  constexpr int kChunks = 16 * kN, kPer = kChunks >= 32 ? kChunks / 32 : 1;
  const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * kStages * C::kUnitBytes);
  const int c0 = kChunks >= 32 ? lane : lane & 15;
  const uint32_t dst = (kChunks >= 32 || lane < 16 ? C::kK : C::kV) + chunk_off<D>(c0 / kN, c0 % kN);
  const uint8_t* const src = (kChunks >= 32 || lane < 16 ? a.k_pages : a.v_pages) + 16 * c0;
  const uint8_t* const src_v = a.v_pages + 16 * lane;
  const uint8_t* const src_s = reinterpret_cast<const uint8_t*>(lane < 2 * kN ? a.k_scale : a.v_scale) + 16 * (lane % (2 * kN));
  const uint32_t dst_s = (lane < 2 * kN ? C::kKs : C::kVs) + 16 * (lane % (2 * kN));
  int issued = 0;
  uint32_t in = ring;  // the stage that takes the next unit
  auto issue = [&] {
    {
      const bool on = issued < n;
      if ((issued & 31) == 0 && issued > 0) {
        rows = next_rows;
        next_rows = rows_at(issued + 32);
      }
      const uint64_t row = __shfl_sync(0xffffffffu, rows, issued & 31);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t to = in + (kN == 8 ? dst ^ (64 * (i & 1)) : dst) + 512 * i;
        cp_async16_if(on, to, src + row * (8 * D) + 512 * i);
        if constexpr (kChunks >= 32) cp_async16_if(on, to + (C::kV - C::kK), src_v + row * (8 * D) + 512 * i);
      }
      cp_async16_if(on && lane < 4 * kN, in + dst_s, src_s + row * D);
    }
    cp_async_commit();
    ++issued;
    in += C::kUnitBytes;
    if (in == ring + kStages * C::kUnitBytes) in = ring;
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue();

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
  // B fragments of Q^T: word t of a group's chunk holds channels 8 t .. 8 t + 7 of column g, of which
  // the even ones meet one MMA, the odd ones (whose nibbles stand 16 times as high) another
  uint32_t qb[kN][kT][2][2];
  float bias[kN][kT][2], qs[kT][2];  // of the lane's accumulator columns 2 t and 2 t + 1
#pragma unroll
  for (int h = 0; h < kT; ++h) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {  // logits in units of log2, from products of 2^-24; all are 0 where the scale is 0
      const float s = qsc[8 * h + 2 * t + c];
      qs[h][c] = s == 0.0f ? 1.0f : s * (0x1p24f * 1.4426950408889634f / sqrtf(static_cast<float>(D)));
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const uint2 w = *reinterpret_cast<const uint2*>(qc + (g + 8 * h) * D + 32 * j + 8 * t);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = static_cast<float>(static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3))));
        if (i & 1) x[i] *= 0.0625f;
      }
      qb[j][h][0][0] = f16x2_of(x[0], x[4]);
      qb[j][h][0][1] = f16x2_of(x[2], x[6]);
      qb[j][h][1][0] = f16x2_of(x[1], x[5]);
      qb[j][h][1][1] = f16x2_of(x[3], x[7]);
      int sum = __dp4a(static_cast<int>(w.x), 0x01010101, __dp4a(static_cast<int>(w.y), 0x01010101, 0));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const float f = -8.0f * 0x1p-24f * static_cast<float>(sum);
      bias[j][h][0] = __shfl_sync(0xffffffffu, f, 8 * t);
      bias[j][h][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }
  }

  // ------------------------------------------------------------ the tokens
  const int lr = lane & 7, lm = lane >> 3;  // ldmatrix: row and matrix that the lane's address is for
  // columns 2 t and 2 t + 1 of each tile: what the exponents are relative to (0 before there is a
  // token), the logit up to which it stays, and the sum over the lane's tokens
  float ref[kT][2], th[kT][2], l[kT][2];
  float o[D / 16][kT][4];
#pragma unroll
  for (int h = 0; h < kT; ++h)
#pragma unroll
    for (int c = 0; c < 2; ++c) th[h][c] = -INFINITY, ref[h][c] = l[h][c] = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int h = 0; h < kT; ++h) o[i][h][0] = o[i][h][1] = o[i][h][2] = o[i][h][3] = 0.0f;
  const int base_tok = L - a.T;  // position of the first draft
  const uint32_t frag = kN == 1   ? chunk_off<D>(8 * (lm & 1) + lr, 0)
                        : kN == 2 ? chunk_off<D>(8 * (lm >> 1) + lr, lm & 1)
                                  : chunk_off<D>(lr, lm);

  // Logits of a unit before the scale qs: x[h][0], [1] of token g, [2], [3] of token g + 8.
  auto logits = [&](uint32_t base, float (&x)[kT][4]) {
    uint32_t kw[2][kN], s0[(kN + 1) / 2], s1[(kN + 1) / 2];
    if constexpr (kN == 1) {
      ldsm2(base + C::kK + frag, kw[0][0], kw[1][0]);
    } else if constexpr (kN == 2) {
      ldsm4(base + C::kK + frag, kw[0][0], kw[0][1], kw[1][0], kw[1][1]);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < kN; j += 4)
          ldsm4(base + C::kK + (frag ^ (16 * j)) + 16 * D / 4 * s, kw[s][j], kw[s][j + 1], kw[s][j + 2], kw[s][j + 3]);
    }
    lds_words<kN>(base + C::kKs + 2 * kN * g, s0);
    lds_words<kN>(base + C::kKs + 2 * kN * (g + 8), s1);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const uint32_t u0 = kw[0][j], u1 = kw[1][j], v0 = u0 >> 8, v1 = u1 >> 8;
      float acc[kT][4];
#pragma unroll
      for (int h = 0; h < kT; ++h) {
        mma_f16_new(acc[h], u0 & 0x000f000fu, u1 & 0x000f000fu, v0 & 0x000f000fu, v1 & 0x000f000fu, qb[j][h][0][0], qb[j][h][0][1]);
        mma_f16_add(acc[h], u0 & 0x00f000f0u, u1 & 0x00f000f0u, v0 & 0x00f000f0u, v1 & 0x00f000f0u, qb[j][h][1][0], qb[j][h][1][1]);
      }
      const float f0 = __uint_as_float((j & 1) ? s0[j / 2] & 0xffff0000u : s0[j / 2] << 16);
      const float f1 = __uint_as_float((j & 1) ? s1[j / 2] & 0xffff0000u : s1[j / 2] << 16);
#pragma unroll
      for (int h = 0; h < kT; ++h) {
        add_pair(acc[h][0], acc[h][1], bias[j][h][0], bias[j][h][1]);
        add_pair(acc[h][2], acc[h][3], bias[j][h][0], bias[j][h][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[h][i] = j == 0 ? acc[h][i] * (i < 2 ? f0 : f1) : fmaf(acc[h][i], i < 2 ? f0 : f1, x[h][i]);
      }
    }
  };

  // Online softmax, lazily rescaled: where a logit passes its column's limit, the reference moves.
  auto move_maxima = [&](const float (&x)[kT][4]) {
    bool grow = false;
#pragma unroll
    for (int h = 0; h < kT; ++h) grow = grow || fmaxf(x[h][0], x[h][2]) > th[h][0] || fmaxf(x[h][1], x[h][3]) > th[h][1];
    if (!__any_sync(0xffffffffu, grow)) return;
#pragma unroll
    for (int h = 0; h < kT; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float mx = col_max(fmaxf(x[h][c], x[h][2 + c])), y = mx * qs[h][c];
        if (!(mx > th[h][c]) || isnan(y)) continue;
        const float f = th[h][c] == -INFINITY ? 0.0f : ex2(ref[h][c] - y);
        ref[h][c] = y;
        th[h][c] = (y + kLazy) / qs[h][c];
        l[h][c] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][h][c] *= f;
          o[i][h][2 + c] *= f;
        }
      }
  };

  // O += the unit's weighted rows.  vis: masks of the V scales of column g + 8 h's token pairs (masked).
  auto output = [&](uint32_t base, const float (&x)[kT][4], const bool masked, const uint32_t (&vis)[kT][2]) {
    uint32_t vw[2][kN], sc[2][kN];
    if constexpr (kN == 1) {
      ldsm2_t(base + C::kV + frag, vw[0][0], vw[1][0]);
    } else if constexpr (kN == 2) {
      ldsm4_t(base + C::kV + frag, vw[0][0], vw[0][1], vw[1][0], vw[1][1]);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < kN; j += 4)
          ldsm4_t(base + C::kV + (frag ^ (16 * j)) + 16 * D / 4 * s, vw[s][j], vw[s][j + 1], vw[s][j + 2], vw[s][j + 3]);
    }
    // scales of tokens 2 t, 2 t + 1 (and + 8), words of two groups a token; below a word of two tokens a group
    lds_words<2 * kN>(base + C::kVs + 4 * kN * t, sc[0]);
    lds_words<2 * kN>(base + C::kVs + 4 * kN * (t + 4), sc[1]);
    // p as bf16 terms, transposed: column g, tokens 2 t and 2 t + 1 (and + 8)
    uint32_t p[kT][kTerms][2];
#pragma unroll
    for (int h = 0; h < kT; ++h) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float pa = ex2(fmaf(x[h][2 * s], qs[h][0], -ref[h][0])), pb = ex2(fmaf(x[h][2 * s + 1], qs[h][1], -ref[h][1]));
        add_pair(l[h][0], l[h][1], pa, pb);
#pragma unroll
        for (int e = 0; e < kTerms; ++e) {
          const uint32_t r = bf16x2_of(pa, pb);
          p[h][e][s] = movm_t(r);
          pa -= __uint_as_float(r << 16);
          pb -= __uint_as_float(r & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      uint32_t wt[kT][kTerms][2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t pair = kN == 1 ? sc[s][0] : prmt(sc[s][j / 2], sc[s][(kN + j) / 2], (j & 1) ? 0x7632 : 0x5410);
#pragma unroll
        for (int h = 0; h < kT; ++h) {
          const uint32_t f = masked ? pair & vis[h][s] : pair;
          if constexpr (kTerms == 2) {
            // p0 s less its rounding is exact in bf16, and p1 s joins it
            wt[h][0][s] = mul_bf16x2(p[h][0][s], f);
            wt[h][1][s] = fma_bf16x2(p[h][1][s], f, fma_bf16x2(p[h][0][s], f, mul_bf16x2(p[h][0][s] ^ 0x80008000u, f)));
          } else {
            float w0 = 0.0f, w1 = 0.0f;
#pragma unroll
            for (int e = kTerms - 1; e >= 0; --e) {
              w0 += __uint_as_float(p[h][e][s] << 16);
              w1 += __uint_as_float(p[h][e][s] & 0xffff0000u);
            }
            w0 *= __uint_as_float(f << 16);
            w1 *= __uint_as_float(f & 0xffff0000u);
#pragma unroll
            for (int e = 0; e < kTerms; ++e) {
              const uint32_t r = bf16x2_of(w0, w1);
              wt[h][e][s] = r;
              w0 -= __uint_as_float(r << 16);
              w1 -= __uint_as_float(r & 0xffff0000u);
            }
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {  // channels 32 j + 4 g + 2 y and + 1
        const uint32_t u0 = y ? vw[0][j] >> 8 : vw[0][j], u1 = y ? vw[1][j] >> 8 : vw[1][j];
        const uint32_t a0 = fma_bf16x2(u0 & 0x000f000fu, k2p127, kLow8), a1 = fma_bf16x2(u0 & 0x00f000f0u, k2p127, kHigh8);
        const uint32_t a2 = fma_bf16x2(u1 & 0x000f000fu, k2p127, kLow8), a3 = fma_bf16x2(u1 & 0x00f000f0u, k2p127, kHigh8);
#pragma unroll
        for (int h = 0; h < kT; ++h)
#pragma unroll
          for (int e = 0; e < kTerms; ++e) mma_bf16(o[2 * j + y][h], a0, a1, a2, a3, wt[h][e][0], wt[h][e][1]);
      }
    }
  };

  const uint32_t no_mask[kT][2] = {};
  auto next_stage = [&](uint32_t p) { return p + C::kUnitBytes == ring + kStages * C::kUnitBytes ? ring : p + C::kUnitBytes; };
  // this warp's last unit can reach past the first draft's position (a sequence has at most three such units)
  const int whole = n > 0 && (first + (n - 1) * kWarps + 1) * kUnit > base_tok ? n - 1 : n;
  uint32_t at = ring;
  float x[kT][4];
  if (n > 0) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    logits(at, x);
  }
  for (int k = 0; k < whole; ++k) {
    move_maxima(x);
    cp_async_wait<kStages - 3>();
    __syncwarp();  // the next unit's bytes are here for all, and the last one's stage is read
    issue();
    const uint32_t next = next_stage(at);
    float y[kT][4];
    logits(next, y);  // of the masked unit, or of a stage that holds none: those are not used
    output(at, x, false, no_mask);
#pragma unroll
    for (int h = 0; h < kT; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[h][i] = y[h][i];
    at = next;
  }
  if (whole < n) {
    const int tok = (first + whole * kWarps) * kUnit;
    // the drafts that column c sees
    auto seen = [&](int c) {
      const int dr = c < GC ? (col0 + c) / G : 0;
      return a.mask ? a.mask[static_cast<int64_t>(b) * a.T + dr] : 0xffffffffu >> (31 - dr);
    };
    auto visible = [&](uint32_t drafts, int p) { return p < base_tok || (p < L && ((drafts >> (p - base_tok)) & 1u)); };
    uint32_t vis[kT][2];
#pragma unroll
    for (int h = 0; h < kT; ++h) {
      const uint32_t da = seen(8 * h + 2 * t), db = seen(8 * h + 2 * t + 1), dg = seen(8 * h + g);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int p = tok + g + 8 * s, q = tok + 2 * t + 8 * s;
        if (!visible(da, p)) x[h][2 * s] = -INFINITY;
        if (!visible(db, p)) x[h][2 * s + 1] = -INFINITY;
        vis[h][s] = (visible(dg, q) ? 0xffffu : 0u) | (visible(dg, q + 1) ? 0xffff0000u : 0u);
      }
    }
    move_maxima(x);
    output(at, x, true, vis);
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
  for (int h = 0; h < kT; ++h) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      l[h][c] = col_sum(l[h][c]);
      ref[h][c] = keep_nan(th[h][c] == -INFINITY ? -INFINITY : ref[h][c], l[h][c]);
    }
    if (g == 0) *reinterpret_cast<float4*>(stat + (warp * kCols + 8 * h + 2 * t) * 2) = make_float4(ref[h][0], l[h][0], ref[h][1], l[h][1]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {  // rows g and g + 8 of tile i
      float* r = red + (warp * D + 16 * i + g) * kCols + 8 * h + 2 * t;
      *reinterpret_cast<float2*>(r) = make_float2(o[i][h][0] * 64.0f, o[i][h][1] * 64.0f);
      *reinterpret_cast<float2*>(r + 8 * kCols) = make_float2(o[i][h][2] * 4.0f, o[i][h][3] * 4.0f);
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
