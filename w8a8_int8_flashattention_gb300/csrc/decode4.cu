// Decode attention over the paged 4-bit cache (rows as in cache4.cuh), for sm_103a: single queries
// and up to 32 drafts a sequence, causal or with tree masks.
//   x_t = s_q * sum_g s_k[t, g] * int32(q_i8[g] . c_k[t, g]) / sqrt(d),  p = softmax(x),
//   O   = sum_t p_t * s_v[t, g] * c_v[t]
// over the tokens t that the query sees, g the groups of 32 channels.
//
// GB300 design.  A column is one query row of a kv head: a draft and a query head.  A CTA takes up to 24 columns
// (8 at d = 256, whose outputs fill the registers) of one (sequence, kv head) and a run of its tokens.
//  * Four warps, each on its own: steps of 32 tokens (16 at d = 256, and at d = 128 with 24 columns), every fourth of
//    the run, arrive by 16-byte cp.async in a ring of the warp's own, the keys of the next step and the values of this one,
//    so that no warp waits for another before the end.  Page ids are read 32 units of 16 tokens ahead.
//  * S[16 tokens x 8 columns] = K Q^T as fp16 m16n8k16 MMAs on the nibbles where they lie, which are
//    fp16 subnormals, n 2^-24 (or, four bits higher, 16 times that, against q / 16); their sums start at -8 times the sum of the
//    q's, which is what the stored offset of 8 adds.  All partial sums are whole multiples of 2^-24 below 2^17 of them, so that a
//    group's integer product is exact.  It meets its scale in fp32.  (The int8 MMA that would take the codes as
//    they are takes 17 cycles an SM on this part, where the fp16 one takes 2 and does half; e4m3
//    operands, in which nibbles are numbers too, are converted to fp16 one by one.)
//  * O^T[d x 8 columns] += V^T P^T as MMAs: ldmatrix.trans hands each lane the four nibbles of two tokens' channels; where
//    they lie they are numbers too, and one fma makes codes of them.  The weight of a row in a group is p * s_v, formed in fp32,
//    two columns at a time, and transposed between lanes in 16 bits.  16-bit outputs take it as one fp16 number, relative
//    to a power of two that follows the largest weight so far, 2^-11 of itself; fp32 outputs as three bf16 terms, which have
//    fp32's range, so that no scale, however far from the others, costs another one its bits.
//  * The logits of the next step are computed beside the output of this one, so that neither
//    chain waits alone; the steps that end behind the first draft, at most one a warp, come last, with masks.
//  * Few tokens: a cluster of up to 8 CTAs a sequence, which send their parts to one another's shared memory.  Many: all
//    sequences' steps are shared out evenly over the CTAs that fit the device, and a second kernel joins what the
//    shares cut (64 sequences of 1,024 to 8,192 tokens, 8 x 4 heads, d = 128: 72 us, and 87 with a cluster of 2 each).
// Bound by the warps' own latency, not by HBM: the accumulators leave 2 to 3.6 warps a scheduler, which wait for the last
// instruction's result or for a turn at a pipe.  At 8 columns and d = 128 issue is at 61 %, the busiest pipe (logic, shifts,
// conversions) at 54 %, the tensor cores at 28 %; at 24 columns at 41, 27 and 29 %.
// 76 sequences of 8,192 tokens, 8 kv heads: 126 us at d = 128 with up to 8 columns, 0.84 of the copy rate
// for codes and scales; 192 with 16 and 257 with 24, where 8 at a time would take 251 and 377; 165 with fp32 outputs.
// d = 64: 91 us, 110, 155; d = 32: 67, 73, 101; d = 256: 241, 0.87 of the copy rate, and 318 with fp32 outputs.
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
// d = c + a b in fp16 with fp32 sums, and d += a b.
__device__ __forceinline__ void mma_f16_on(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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
// (x0, x1) += (a0, a1) in fp32, as one instruction.
__device__ __forceinline__ void add_pair(float& x0, float& x1, float a0, float a1) {
  asm("{\n\t.reg .b64 x, a;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tadd.rn.f32x2 x, x, a;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a0), "f"(a1));
}
template <int kA>
__device__ __forceinline__ float bf16_half(uint32_t a) {  // as fp32
  const uint16_t x = static_cast<uint16_t>(kA ? a >> 16 : a);
  float d;
  asm("add.rn.f32.bf16 %0, %1, %2;" : "=f"(d) : "h"(x), "f"(-0.0f));
  return d;
}
// (x0, x1) *= (f0, f1).
__device__ __forceinline__ void scale_pair(float& x0, float& x1, float f0, float f1) {
  asm("{\n\t.reg .b64 x, f;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 f, {%2, %3};\n\tmul.rn.f32x2 x, x, f;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(f0), "f"(f1));
}
// (x0, x1) = (a0, a1) f, and (x0, x1) += (a0, a1) f.
__device__ __forceinline__ void mul_pair(float& x0, float& x1, float a0, float a1, float f) {
  asm("{\n\t.reg .b64 x, a, f;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\tmul.rn.f32x2 x, a, f;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(f));
}
__device__ __forceinline__ void fma_pair(float& x0, float& x1, float a0, float a1, float f) {
  asm("{\n\t.reg .b64 x, a, f;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\tfma.rn.f32x2 x, a, f, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a0), "f"(a1), "f"(f));
}
// Nibbles where they lie in a 16-bit word are bf16 numbers, n 2^-133 (bits 0..3) and n 2^-129
// (bits 4..7, since the exponents 0 and 1 have the same step): times 2^127 and less 8 such, codes.
// As fp16 numbers they are n 2^-24 and n 2^-20, times 2^15 less 8 such.
template <bool kHalf>
struct Codes4 {
  static constexpr uint32_t kUp = kHalf ? 0x78007800u : 0x7f007f00u;     // 2^15, 2^127
  static constexpr uint32_t kLow8 = kHalf ? 0xa400a400u : 0xbe00be00u;   // -8 2^-9, -8 2^-6
  static constexpr uint32_t kHigh8 = kHalf ? 0xb400b400u : 0xc000c000u;  // -8 2^-5, -8 2^-2
  static constexpr float kLow = kHalf ? 512.0f : 64.0f, kHigh = kHalf ? 32.0f : 4.0f;  // what takes codes of them
  static __device__ __forceinline__ uint32_t low(uint32_t w) { return fma(w & 0x000f000fu, kLow8); }
  static __device__ __forceinline__ uint32_t high(uint32_t w) { return fma(w & 0x00f000f0u, kHigh8); }
  static __device__ __forceinline__ uint32_t fma(uint32_t w, uint32_t less) {
    uint32_t r;
    if constexpr (kHalf) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(kUp), "r"(less));
    else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(kUp), "r"(less));
    return r;
  }
};
// The magnitude's bits of the bf16 number in the low half of a word; 0 for infinities and NaN, which make their
// group's channels NaN whatever the others' weights are relative to.
__device__ __forceinline__ uint32_t finite_scale(uint32_t w) {
  const uint32_t s = w & 0x7fffu;
  return s < 0x7f80u ? s : 0u;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int kCols>
struct Cfg4 {
  static constexpr int kN = D / kGroup4;  // groups (and 16-byte chunks) of a row
  static constexpr int kT = (kCols + 7) / 8;  // tiles of eight columns
  // Units of 16 tokens that a warp takes at a time, a step: two where the registers hold them (64 sequences of up to 8,192
  // tokens 71 us, and 77 with one; 16 x 5 drafts of 4 heads, 20 columns, at d = 128 46 with one and 51 with two).
  static constexpr int kU = D == 256 || (D == 128 && kCols > 16) ? 1 : 2;
  static constexpr int kStep = 16 * kU;
  static constexpr int kStart = D == 256 ? 16 : 512 / kStep;  // steps that a sequence's start and end are worth, see below
  static constexpr int kHalf = kU * 9 * D;  // a step's keys, or its values: codes [kU][16][D / 2], scales [kU][16][kN]
  static constexpr int kScales = kU * 8 * D;
  static constexpr int kRing = 4 * kHalf;  // of a warp: two steps' keys, two steps' values
  // as many CTAs an SM as their registers let, the accumulators being D kT / 4 a thread (48 sequences, 16 columns at
  // d = 64: with one more 37.0 us for 33.8, with one less 34.1; 64 at d = 128 with one less 71.8 for 71.3)
  static constexpr int kCtas = D == 256 ? 3 : D == 128 ? 5 - kT : 6 - kT;
  // after the loop the rings hold the warps' O^T [warp][D][kCols], fp32
  static constexpr int kRed = 0, kMerge = kWarps * D * kCols * 4;
  static constexpr int kQf = kWarps * kRing > kMerge ? kWarps * kRing : kMerge;  // [kN][kT][32] fragments of Q, 16 bytes
  static constexpr int kBias = kQf + kN * kT * 512;       // [kN][kT][4][4] -8 sum of q of columns 2 t, 2 t + 1, twice
  static constexpr int kQs = kBias + kN * kT * 64;        // [kCols] scales
  static constexpr int kQc = kQs + kCols * 4;             // [kCols][D] query codes
  static constexpr int kStat = kQc + kCols * D;           // [warp][kCols][2]: max (log2), sum
  // [warp][kCols] exponents of the warps' fp16 weights, then weights of the warps' parts, or of the CTAs'
  static constexpr int kWt = kStat + kWarps * kCols * 8;
  static constexpr int kRows = kWt + kMaxCluster * kCols * 4;  // [kCols] rows of q and out
  // what a cluster's CTAs send: [CTA][kCols][2] max and sum, and of each CTA its runs [CTA][run][32], four columns each
  static constexpr int kMl = kRows + kCols * 8;
  static constexpr int kIn = kMl + kMaxCluster * kCols * 8;
  static constexpr int kRuns = D * kCols / 128;  // of 32 rows of O^T and four columns
  static constexpr int kBytes = kIn + (kRuns + kMaxCluster - 1) * 512;
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "kCtas CTAs fit an SM");
};

// The work of a balanced launch: the (kv head, column group)s, each with all sequences in a row, each
// sequence kStart and its steps long, are cut evenly among `ctas` CTAs, but into no less than kLeast
// steps.  kStart stands for what a CTA spends on a sequence besides its steps, queries and merge; an empty
// sequence counts one step.  (Without kStart a CTA that had 32 sequences of one token ran five times as long as
// the others; with a sequence's heads in a row, two times with it.)
constexpr int kLeast = 4 * kWarps;
__device__ __forceinline__ int steps_of(int L, int step) { return max(1, (L + step - 1) / step); }

// Byte offset of chunk j of row r: eight rows' chunks j lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int r, int j) {
  constexpr int n = D / kGroup4, m = 8 / n;  // chunks of a row, rows in 128 bytes
  return static_cast<uint32_t>(r * (16 * n) + 16 * (j ^ (((r & 7) / m) & (n - 1))));
}

// A cluster's barrier: what a thread has written before it arrives is there for those that have waited.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Inclusive prefix over the CTA's threads of one value each.
__device__ __forceinline__ int64_t cta_prefix(int64_t x, int64_t* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += sm[w];
  return x;
}

// kCols: columns of a CTA.  kTerms: 1, weights as one fp16 number; 3, as three bf16 terms.
template <int D, int kCols, int kTerms>
__global__ void __launch_bounds__(kThreads, Cfg4<D, kCols>::kCtas)
    decode4_kernel(const Decode4Args a, DeviceStatus* st) {
  using C = Cfg4<D, kCols>;
  constexpr int kN = C::kN, kT = C::kT, kU = C::kU;
  constexpr bool kHalf = kTerms == 1;           // weights and value codes in fp16, else in bf16
  constexpr uint32_t kMinusOne = 0xbf80u;       // bf16
  using Codes = Codes4<kHalf>;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int G = a.Hq / a.Hkv, per_seq = a.Hkv * a.groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cap = a.max_blocks * a.page;
  auto checked = [&](int L) {
    if (L >= 0 && L <= cap) return L;
    if (threadIdx.x == 0) record_status(st, kStatusBadArg, 870);
    return L < 0 ? 0 : cap;
  };

  // ------------------------------------------------------------ this CTA's part of the work
  if (a.ctas) {
    grid_dependents_launch();  // the combine's CTAs may come as this grid's go
    if (threadIdx.x == 0) a.starts[blockIdx.x] = -1;  // the sequence that this CTA begins and does not end
  }
  const int S = a.ctas ? 1 : a.splits;
  if (S > 1) cluster_arrive();
  int rank = 0, b, inner;      // inner: kv head * groups + column group
  int64_t left = 1;            // balanced: what this CTA still has of its share
  int s0 = 0;                  // first step of the segment in its sequence; below 0: in its kStart
  if (a.ctas) {
    int64_t* scan = reinterpret_cast<int64_t*>(smem);
    // a thread's sequences, [i0, i1), and what they and all before them come to
    const int strip = (a.B + kThreads - 1) / kThreads;
    const int i0 = min(a.B, static_cast<int>(threadIdx.x) * strip), i1 = min(a.B, i0 + strip);
    int64_t x = 0;
    for (int i = i0; i < i1; ++i) x += C::kStart + steps_of(checked(a.seqlens[i]), C::kStep);
    const int64_t end = cta_prefix(x, scan);
    if (threadIdx.x == kThreads - 1) scan[kWarps] = end;
    __syncthreads();
    const int64_t all = scan[kWarps], total = all * per_seq;
    auto divide = [](int64_t x, int64_t y) {  // of numbers that mostly fit 32 bits
      return (x | y) >> 32 ? x / y : static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
    };
    // CTA i of `used` has [i q + min(i, r), ...) of the total, q r its quotient and remainder
    const int64_t used = max(int64_t(1), min(static_cast<int64_t>(a.ctas), total / kLeast));
    if (blockIdx.x >= used) return;
    const int64_t q = divide(total, used), r = total - q * used;
    const int64_t from = blockIdx.x * q + min(static_cast<int64_t>(blockIdx.x), r);
    left = q + (blockIdx.x < r ? 1 : 0);
    inner = static_cast<int>(divide(from, all));
    const int64_t off = from - inner * all;
    if (off >= end - x && off < end) {  // this thread has the sequence that `off` lies in
      int64_t at = end - x;
      int i = i0;
      for (;; ++i) {
        const int per = C::kStart + steps_of(checked(a.seqlens[i]), C::kStep);
        if (off < at + per) break;
        at += per;
      }
      scan[kWarps + 1] = i;
      scan[kWarps + 2] = at;
    }
    __syncthreads();
    b = static_cast<int>(scan[kWarps + 1]);
    s0 = static_cast<int>(off - scan[kWarps + 2]) - C::kStart;
    __syncthreads();
  } else {
    const unsigned item = blockIdx.x / static_cast<unsigned>(S);
    rank = static_cast<int>(blockIdx.x - item * S);
    b = static_cast<int>(item / static_cast<unsigned>(per_seq));
    inner = static_cast<int>(item - static_cast<unsigned>(b) * per_seq);
  }

  // ------------------------------------------------------------ what stays from segment to segment
  const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * C::kRing);
  // a lane's chunks of a unit's 16 kN: c0, c0 + 32, ..., 512 bytes apart (at d = 256, four rows on, with
  // another swizzle); of its scales' 2 kN: one, the units of a step side by side
  constexpr int kChunks = 16 * kN, kPer = kChunks >= 32 ? kChunks / 32 : 1;
  const uint32_t dst = chunk_off<D>((lane % kChunks) / kN, lane % kN);
  const uint32_t dst_s = C::kScales + 16 * (lane % (2 * kN * kU));
  const int lr = lane & 7, lm = lane >> 3;  // ldmatrix: row and matrix that the lane's address is for
  const uint32_t frag = kN == 1   ? chunk_off<D>(8 * (lm & 1) + lr, 0)
                        : kN == 2 ? chunk_off<D>(8 * (lm >> 1) + lr, lm & 1)
                                  : chunk_off<D>(lr, lm);
  const uint32_t qf = smem_u32(smem) + C::kQf + 16 * lane, qbias = smem_u32(smem) + C::kBias + 16 * t;

  for (;;) {
    const int head = inner / a.groups;
    const int col0 = (inner - head * a.groups) * a.cols;  // first of this segment's columns
    const int GC = min(a.cols, a.T * G - col0);
    int64_t* const row_of = reinterpret_cast<int64_t*>(smem + C::kRows);  // of q and out, for each column
    // The query columns, eight lanes a row, are asked for beside the length, and quantised while the first rows' pages
    // are looked up: a segment starts with a chain of loads that wait for one another.
    const int len = a.seqlens[b];
    constexpr int kPass = (8 * kCols + kThreads - 1) / kThreads;
    float qx[kPass][D / 32][4] = {};
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const int c = static_cast<int>(threadIdx.x >> 3) + i * (kThreads / 8);
      if (c < GC) {
        const int dr = (col0 + c) / G;  // its draft, its query head
        const int64_t at = (static_cast<int64_t>(b) * a.T + dr) * a.Hq + head * G + (col0 + c - dr * G);
        load_runs<D / 32>(a.q, a.q_dtype, at * D + 4 * (lane & 7), 32, qx[i]);
        if ((lane & 7) == 0) row_of[c] = at;
      }
    }
    const int L = checked(len), per = steps_of(L, C::kStep);
    int s1 = per;
    if (a.ctas) {
      s1 = static_cast<int>(min(static_cast<int64_t>(per), s0 + left));
      left -= s1 - s0;
      if (s1 <= 0) return;  // the share ends before the first step
      s0 = max(s0, 0);
    } else {
      s0 = static_cast<int>(static_cast<int64_t>(per) * rank / S);
      s1 = static_cast<int>(static_cast<int64_t>(per) * (rank + 1) / S);
    }
    // this warp's steps: first, first + kWarps, ...
    const int first = s0 + warp, n = max(0, (s1 - first + kWarps - 1) / kWarps);

    // ---------------------------------------------------------- loads
    const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_blocks;
    // the sixteenth of a row index at which a unit lies; lane i looks up unit i % kU of step k + i / kU.
    // Units past the end are row 0: loaded, and not used.
    auto rows_at = [&](int k) -> uint32_t {
      const int step = k + lane / kU;
      if (step >= n) return 0;
      const int tok = (first + step * kWarps) * C::kStep + lane % kU * 16;
      if (tok >= L) return 0;
      const int blk = tok / a.page;
      int32_t pg = table[blk];
      if (pg < 0 || pg >= a.num_pages) {
        record_status(st, kStatusBadArg, 871);
        pg = 0;
      }
      return (static_cast<uint32_t>(pg) * a.Hkv + head) * (a.page / 16) + (tok - blk * a.page) / 16;
    };
    constexpr int kBatch = 32 / kU;  // steps that a look-up covers
    uint32_t rows = rows_at(0), next_rows = n > kBatch ? rows_at(kBatch) : 0;
    uint32_t row[kU] = {};  // of the step whose keys were asked for last
    int looked = 0, at_lane = 0;
    // Lanes that have no chunk of their own repeat another's.
    auto ask = [&](uint32_t to, const uint8_t* codes, const uint16_t* scales) {
      if constexpr (kChunks >= 32) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const uint8_t* src = codes + static_cast<uint64_t>(row[u]) * (8 * D) + 16 * lane;
#pragma unroll
          for (int i = 0; i < kPer; ++i) cp_async16(to + u * 8 * D + (kN == 8 ? dst ^ (64 * (i & 1)) : dst) + 512 * i, src + 512 * i);
        }
      } else {  // d = 32: half a warp a unit
        const uint32_t r = lane < 16 ? row[0] : row[kU - 1];
        cp_async16(to + (lane >> 4) * 8 * D + dst, codes + static_cast<uint64_t>(r) * (8 * D) + 16 * (lane & 15));
      }
      const uint32_t r = kU == 2 && (lane & (2 * kN)) ? row[kU - 1] : row[0];
      cp_async16(to + dst_s, reinterpret_cast<const uint8_t*>(scales) + static_cast<uint64_t>(r) * D + 16 * (lane % (2 * kN)));
    };
    // the keys of the next step and the values of the one before it
    auto next_row = [&] {
      if (at_lane == 32) {
        looked += kBatch;
        rows = next_rows;
        next_rows = rows_at(looked + kBatch);
        at_lane = 0;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) row[u] = __shfl_sync(0xffffffffu, rows, at_lane + u);
      at_lane += kU;
    };
    auto issue = [&](uint32_t to_k, uint32_t to_v) {
      ask(to_v, a.v_pages, a.v_scale);
      next_row();
      ask(to_k, a.k_pages, a.k_scale);
      cp_async_commit();
    };
    // ---------------------------------------------------------- the query columns
    int8_t* qc = reinterpret_cast<int8_t*>(smem + C::kQc);
    float* qsc = reinterpret_cast<float*>(smem + C::kQs);
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int c = static_cast<int>(threadIdx.x >> 3) + p * (kThreads / 8), l8 = lane & 7;
      if (c >= kCols) break;
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(qx[p][i][e]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const RowScale rs = row_scale(amax);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) *reinterpret_cast<uint32_t*>(qc + c * D + 32 * i + 4 * l8) = quant4(qx[p][i], rs);
      if (l8 == 0) qsc[c] = rs.s;
    }
    next_row();
    ask(ring, a.k_pages, a.k_scale);
    cp_async_commit();
    issue(ring + C::kHalf, ring + 2 * C::kHalf);
    __syncthreads();
    // B fragments of Q^T: word t of a group's chunk holds channels 8 t .. 8 t + 7 of column g, of which
    // the even ones meet one MMA, the odd ones (whose nibbles stand 16 times as high) another
    for (int i = warp; i < kN * kT; i += kWarps) {
      const int j = i / kT, c = g + 8 * (i % kT);
      const uint2 w = *reinterpret_cast<const uint2*>(qc + c * D + 32 * j + 8 * t);
      const uint32_t lo = prmt(w.x ^ 0x80808080u, w.y ^ 0x80808080u, 0x5140), hi = prmt(w.x ^ 0x80808080u, w.y ^ 0x80808080u, 0x7362);
      auto sixteenth = [](uint32_t x) {
        uint32_t r;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x2c002c00u));
        return r;
      };
      *reinterpret_cast<uint4*>(smem + C::kQf + i * 512 + 16 * lane) =
          make_uint4(codes_f16x2(lo, 0x4140), codes_f16x2(hi, 0x4140), sixteenth(codes_f16x2(lo, 0x4342)), sixteenth(codes_f16x2(hi, 0x4342)));
      int sum = __dp4a(static_cast<int>(w.x), 0x01010101, __dp4a(static_cast<int>(w.y), 0x01010101, 0));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (t < 2) reinterpret_cast<float*>(smem + C::kBias)[i * 16 + 4 * (g >> 1) + 2 * t + (g & 1)] = -8.0f * 0x1p-24f * static_cast<float>(sum);
    }
    // of the lane's accumulator columns 2 t and 2 t + 1
    float qs[kT][2];
#pragma unroll
    for (int h = 0; h < kT; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // logits in units of log2, from products of 2^-24; all are 0 where the scale is 0
        const float s = qsc[8 * h + 2 * t + c];
        qs[h][c] = s == 0.0f ? 1.0f : s * (0x1p24f * 1.4426950408889634f / sqrtf(static_cast<float>(D)));
      }
    __syncthreads();

    // ---------------------------------------------------------- the tokens
    // columns 2 t and 2 t + 1 of each tile: what the exponents are relative to, the maximum (0 before there is a
    // token), the logit up to which it stays, and the sum over the lane's tokens
    float ref[kT][2], th[kT][2], l[kT][2];
    [[maybe_unused]] float inv[kT][2];             // fp16 weights are p s_v 2^-E: 2^-E
    [[maybe_unused]] uint32_t vlim = 0x7f800000u;  // and the V scale up to which they all fit
    float o[D / 16][kT][4];
#pragma unroll
    for (int h = 0; h < kT; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c) th[h][c] = -INFINITY, ref[h][c] = l[h][c] = 0.0f, inv[h][c] = 1.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int h = 0; h < kT; ++h) o[i][h][0] = o[i][h][1] = o[i][h][2] = o[i][h][3] = 0.0f;
    const int base_tok = L - a.T;  // position of the first draft

    // Logits of a step before the scale qs: x[u][h][0], [1] of token g of unit u, [2], [3] of token g + 8.
    auto logits = [&](uint32_t base, float (&x)[kU][kT][4]) {
      uint32_t kw[kU][2][kN], sc[kU][2][(kN + 1) / 2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t p = base + u * 8 * D + frag, q = base + C::kScales + u * D + 2 * kN * g;
        if constexpr (kN == 1) {
          ldsm2(p, kw[u][0][0], kw[u][1][0]);
        } else if constexpr (kN == 2) {
          ldsm4(p, kw[u][0][0], kw[u][0][1], kw[u][1][0], kw[u][1][1]);
        } else {
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < kN; j += 4)
              ldsm4((j ? p ^ (16 * j) : p) + 4 * D * s, kw[u][s][j], kw[u][s][j + 1], kw[u][s][j + 2], kw[u][s][j + 3]);
        }
        lds_words<kN>(q, sc[u][0]);
        lds_words<kN>(q + 16 * kN, sc[u][1]);
      }
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        uint32_t qb[kT][4];
        float bias[kT][4];
#pragma unroll
        for (int h = 0; h < kT; ++h) {
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(qb[h][0]), "=r"(qb[h][1]), "=r"(qb[h][2]), "=r"(qb[h][3]) : "r"(qf + (j * kT + h) * 512));
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(bias[h][0]), "=f"(bias[h][1]), "=f"(bias[h][2]), "=f"(bias[h][3]) : "r"(qbias + (j * kT + h) * 64));
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const uint32_t u0 = kw[u][0][j], u1 = kw[u][1][j], v0 = u0 >> 8, v1 = u1 >> 8;
          const float f0 = (j & 1) ? bf16_half<1>(sc[u][0][j / 2]) : bf16_half<0>(sc[u][0][j / 2]);
          const float f1 = (j & 1) ? bf16_half<1>(sc[u][1][j / 2]) : bf16_half<0>(sc[u][1][j / 2]);
#pragma unroll
          for (int h = 0; h < kT; ++h) {
            float acc[4];
            mma_f16_on(acc, u0 & 0x000f000fu, u1 & 0x000f000fu, v0 & 0x000f000fu, v1 & 0x000f000fu, qb[h][0], qb[h][1], bias[h]);
            mma_f16_add(acc, u0 & 0x00f000f0u, u1 & 0x00f000f0u, v0 & 0x00f000f0u, v1 & 0x00f000f0u, qb[h][2], qb[h][3]);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const float f = i < 2 ? f0 : f1;
              if (j == 0) mul_pair(x[u][h][i], x[u][h][i + 1], acc[i], acc[i + 1], f);
              else fma_pair(x[u][h][i], x[u][h][i + 1], acc[i], acc[i + 1], f);
            }
          }
        }
      }
    };

    // Online softmax, lazily rescaled: where a logit passes its column's limit, the reference moves.
    // fp16 weights w = p s_v 2^-E: without E a row of a huge scale would not fit, and with E following the scales
    // alone a row of a huge scale and no probability would push the others below fp16's range.  So E follows the
    // weights: it is about log2 of the column's largest p s_v, and moves where a logit is 2^kLazyLists above the
    // maximum, or a scale 2^10 above that weight.  The sum of the p knows nothing of it.
    auto move_maxima = [&](const float (&x)[kU][kT][4], uint32_t values) {
      bool grow = false;
      float mx[kT][2];
#pragma unroll
      for (int h = 0; h < kT; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[h][c] = fmaxf(x[0][h][c], x[0][h][2 + c]);
          if constexpr (kU == 2) mx[h][c] = fmaxf(mx[h][c], fmaxf(x[kU - 1][h][c], x[kU - 1][h][2 + c]));
          grow = grow || mx[h][c] > th[h][c];
        }
      if constexpr (kHalf) {  // each lane looks at its share of the step's scales
        constexpr int kMine = kU * D / 64;
        uint32_t w[(kMine + 1) / 2];
        lds_words<kMine>(values + C::kScales + 2 * kMine * lane, w);
        uint32_t s = w[0] << 16;
        if constexpr (kMine > 1) s = max(s, w[0] & 0xffff0000u);
        if constexpr (kMine > 2) s = max(s, max(w[(kMine - 1) / 2] << 16, w[(kMine - 1) / 2] & 0xffff0000u));
        if (!__any_sync(0xffffffffu, grow || s > vlim)) return;
        // The bits of an infinity, a NaN or a negative scale lie above any limit; here they count as below.
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) most = max(most, finite_scale((i & 1) ? w[i / 2] >> 16 : w[i / 2]));
        grow = grow || (most << 16) > vlim;
      }
      if (!__any_sync(0xffffffffu, grow)) return;
      [[maybe_unused]] float up[kU][2];  // log2 of the largest finite scale of tokens g and g + 8, rounded up
      if constexpr (kHalf) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            uint32_t w[(kN + 1) / 2], most = 0;
            lds_words<kN>(values + C::kScales + u * D + 2 * kN * (g + 8 * s), w);
#pragma unroll
            for (int j = 0; j < kN; ++j) most = max(most, finite_scale((j & 1) ? w[j / 2] >> 16 : w[j / 2]));
            up[u][s] = static_cast<float>(static_cast<int>(most >> 7) - 126);
          }
      }
      auto bounded = [](float v) { return fminf(fmaxf(v, -1048576.0f), 1048576.0f); };
#pragma unroll
      for (int h = 0; h < kT; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float m = col_max(mx[h][c]), y = m * qs[h][c];
          float heavy = 0.0f;
          if constexpr (kHalf) {
            heavy = -INFINITY;
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
              for (int s = 0; s < 2; ++s) heavy = fmaxf(heavy, bounded(x[u][h][2 * s + c] * qs[h][c]) + up[u][s]);
            heavy = col_max(heavy);
          }
          const bool first = th[h][c] == -INFINITY, higher = m > th[h][c];
          if ((first && !higher) || isnan(y) || (!kHalf && !higher)) continue;
          const float to = higher ? y : ref[h][c], shift = ref[h][c] - to, f = first ? 0.0f : ex2(shift);
          float fo = f;
          if constexpr (kHalf) {
            // what the earlier rows' largest weight has become, and this step's, in [2^(e - 1), 2^(e + 1))
            const int before = 127 - static_cast<int>(__float_as_uint(inv[h][c]) >> 23);
            const int kept = first ? -120 : before + __float2int_rd(fmaxf(shift, -252.0f));
            const int e = __float2int_ru(heavy - bounded(to)) - 1;
            const int E = max(-120, min(120, max(kept, e)));
            inv[h][c] = pow2i(-E);
            fo = f * pow2i(min(127, before - E));  // at most 2: f is 0 where before - E is above
          }
          ref[h][c] = to;
          if (higher) th[h][c] = (y + static_cast<float>(kHalf ? kLazyLists : static_cast<int>(kLazy))) / qs[h][c];
          l[h][c] *= f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[i][h][c] *= fo;
            o[i][h][2 + c] *= fo;
          }
        }
      if constexpr (kHalf) {  // the limit of the column that has the least weights
        int least = 120;
#pragma unroll
        for (int h = 0; h < kT; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (th[h][c] != -INFINITY) least = min(least, 127 - static_cast<int>(__float_as_uint(inv[h][c]) >> 23));
        least = min(least, __shfl_xor_sync(0xffffffffu, least, 1));
        least = min(least, __shfl_xor_sync(0xffffffffu, least, 2));
        vlim = static_cast<uint32_t>(min(127, least + 15 - kLazyLists) + 127) << 23;
      }
    };

    // O += a step's weighted rows.  vis (masked): which of the columns 2 t and 2 t + 1 see tokens g and g + 8; whatever the
    // scales of the others hold, they weigh nothing.
    auto output = [&](uint32_t base, const float (&x)[kU][kT][4], const bool masked, const uint32_t (&vis)[kU][kT][2]) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t q = base + u * 8 * D + frag, r = base + C::kScales + u * D + 2 * kN * g;
        uint32_t vw[2][kN], sc[2][(kN + 1) / 2];
        if constexpr (kN == 1) {
          ldsm2_t(q, vw[0][0], vw[1][0]);
        } else if constexpr (kN == 2) {
          ldsm4_t(q, vw[0][0], vw[0][1], vw[1][0], vw[1][1]);
        } else {
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < kN; j += 4)
              ldsm4_t((j ? q ^ (16 * j) : q) + 4 * D * s, vw[s][j], vw[s][j + 1], vw[s][j + 2], vw[s][j + 3]);
        }
        lds_words<kN>(r, sc[0]);
        lds_words<kN>(r + 16 * kN, sc[1]);
        float p[kT][2][2];  // of tokens g and g + 8 and columns 2 t and 2 t + 1
#pragma unroll
        for (int h = 0; h < kT; ++h)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            p[h][s][0] = ex2(fmaf(x[u][h][2 * s], qs[h][0], -ref[h][0]));
            p[h][s][1] = ex2(fmaf(x[u][h][2 * s + 1], qs[h][1], -ref[h][1]));
            add_pair(l[h][0], l[h][1], p[h][s][0], p[h][s][1]);
            if constexpr (kHalf) scale_pair(p[h][s][0], p[h][s][1], inv[h][0], inv[h][1]);
          }
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          uint32_t wt[kT][kTerms][2];  // the weights, transposed: column g, tokens 2 t and 2 t + 1 (and + 8)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const float f = (j & 1) ? bf16_half<1>(sc[s][j / 2]) : bf16_half<0>(sc[s][j / 2]);
#pragma unroll
            for (int h = 0; h < kT; ++h) {
              float w0, w1;
              mul_pair(w0, w1, p[h][s][0], p[h][s][1], f);
              if (masked) {
                w0 = (vis[u][h][s] & 1u) ? w0 : 0.0f;
                w1 = (vis[u][h][s] & 2u) ? w1 : 0.0f;
              }
              if constexpr (kHalf) {
                wt[h][0][s] = movm_t(f16x2_of(w0, w1));
              } else {
#pragma unroll
                for (int e = 0; e < kTerms; ++e) {
                  const uint32_t w = bf16x2_of(w0, w1);
                  wt[h][e][s] = movm_t(w);
                  if (e + 1 < kTerms) {
                    w0 = fma_mixed<0, 0>(w, kMinusOne, w0);
                    w1 = fma_mixed<1, 0>(w, kMinusOne, w1);
                  }
                }
              }
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // channels 32 j + 4 g + 2 y and + 1
            const uint32_t u0 = y ? vw[0][j] >> 8 : vw[0][j], u1 = y ? vw[1][j] >> 8 : vw[1][j];
            const uint32_t a0 = Codes::low(u0), a1 = Codes::high(u0), a2 = Codes::low(u1), a3 = Codes::high(u1);
#pragma unroll
            for (int h = 0; h < kT; ++h) {
              if constexpr (kHalf) {
                mma_f16_add(o[2 * j + y][h], a0, a1, a2, a3, wt[h][0][0], wt[h][0][1]);
              } else {
#pragma unroll
                for (int e = 0; e < kTerms; ++e) mma_bf16(o[2 * j + y][h], a0, a1, a2, a3, wt[h][e][0], wt[h][e][1]);
              }
            }
          }
        }
      }
    };

    const uint32_t no_mask[kU][kT][2] = {};
    // this warp's last step can reach past the first draft's position (a sequence has at most three such steps)
    const int whole = n > 0 && (first + (n - 1) * kWarps + 1) * C::kStep > base_tok ? n - 1 : n;
    uint32_t now = 0;  // half of the rings that this step's values are in, and its keys were
    float x[kU][kT][4];
    cp_async_wait<1>();
    __syncwarp();
    logits(ring, x);  // a warp without steps: of stale bytes, not used
    for (int k = 0; k < whole; ++k) {
      cp_async_wait<0>();
      __syncwarp();  // this step's values and the next one's keys are here for all, and what they replace is read
      move_maxima(x, ring + 2 * C::kHalf + now);
      const uint32_t then = C::kHalf - now;
      issue(ring + now, ring + 2 * C::kHalf + then);
      output(ring + 2 * C::kHalf + now, x, false, no_mask);
      logits(ring + then, x);  // of the masked step, or of one past the end, which are not used
      now = then;
    }
    cp_async_wait<0>();
    __syncwarp();
    if (whole < n) {
      const int tok = (first + whole * kWarps) * C::kStep;
      // the drafts that column c sees
      auto seen = [&](int c) {
        const int dr = c < GC ? (col0 + c) / G : 0;
        return a.mask ? a.mask[static_cast<int64_t>(b) * a.T + dr] : 0xffffffffu >> (31 - dr);
      };
      auto visible = [&](uint32_t drafts, int p) { return p < base_tok || (p < L && ((drafts >> (p - base_tok)) & 1u)); };
      uint32_t vis[kU][kT][2];
#pragma unroll
      for (int h = 0; h < kT; ++h) {
        const uint32_t da = seen(8 * h + 2 * t), db = seen(8 * h + 2 * t + 1);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int p = tok + 16 * u + g + 8 * s;
            const bool va = visible(da, p), vb = visible(db, p);
            if (!va) x[u][h][2 * s] = -INFINITY;
            if (!vb) x[u][h][2 * s + 1] = -INFINITY;
            vis[u][h][s] = (va ? 1u : 0u) | (vb ? 2u : 0u);
          }
      }
      move_maxima(x, ring + 2 * C::kHalf + now);
      output(ring + 2 * C::kHalf + now, x, true, vis);
    }

    // ---------------------------------------------------------- the CTA's state from its warps'
    float* stat = reinterpret_cast<float*>(smem + C::kStat);
    float* red = reinterpret_cast<float*>(smem + C::kRed);
    float* wt = reinterpret_cast<float*>(smem + C::kWt);
    __syncthreads();  // the rings are free
#pragma unroll
    for (int h = 0; h < kT; ++h) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[h][c] = col_sum(l[h][c]);
        ref[h][c] = keep_nan(th[h][c] == -INFINITY ? -INFINITY : ref[h][c], l[h][c]);
      }
      if (g == 0) *reinterpret_cast<float4*>(stat + (warp * kCols + 8 * h + 2 * t) * 2) = make_float4(ref[h][0], l[h][0], ref[h][1], l[h][1]);
      if (kHalf && g == 0) *reinterpret_cast<float2*>(wt + warp * kCols + 8 * h + 2 * t) = make_float2(pow2_inverse(inv[h][0]), pow2_inverse(inv[h][1]));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {  // rows g and g + 8 of tile i
        float* r = red + (warp * D + 16 * i + g) * kCols + 8 * h + 2 * t;
        *reinterpret_cast<float2*>(r) = make_float2(o[i][h][0] * Codes::kLow, o[i][h][1] * Codes::kLow);
        *reinterpret_cast<float2*>(r + 8 * kCols) = make_float2(o[i][h][2] * Codes::kHigh, o[i][h][3] * Codes::kHigh);
      }
    }
    __syncthreads();
    const bool cut = a.ctas && s1 - s0 < per;  // a part of a sequence, for the combine
    // The parts of a column, of maxima v.x and sums v.y: the joined ones, and weights of the parts' outputs.  A warp's
    // output is relative to 2^E (in wt) and not divided by anything yet, a CTA's is divided by its sum, so that
    // neither passes fp32 where the joined output does not.
    auto weigh = [&](int c, int n, const auto& v, bool ctas, float& M, float& sum) {
      constexpr int kMost = sizeof(v) / sizeof(v[0]);
      M = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < n) M = fmaxf(M, v[i].x);
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < n) {
          const float f = v[i].x == -INFINITY ? 0.0f : ex2(v[i].x - M);
          if (v[i].x != -INFINITY) sum = fmaf(f, v[i].y, sum);
          wt[i * kCols + c] = f * (ctas ? v[i].y : kHalf ? wt[i * kCols + c] : 1.0f);
        }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < n) wt[i * kCols + c] *= inv;
      M = keep_nan(M, sum);  // which stays beside the others' maxima
    };
    auto store_lse = [&](int c, float M, float sum) {
      if (a.lse && rank == 0) a.lse[row_of[c]] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
    };
    // slot 0 of a CTA's two parts where its work begins, else 1
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (s0 == 0 ? 1 : 0);
    if (S > 1) cluster_wait();  // all of the cluster have started
    if (threadIdx.x < GC) {
      const int c = threadIdx.x;
      float M, sum;
      float2 v[kWarps];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v[i] = *reinterpret_cast<const float2*>(stat + (i * kCols + c) * 2);
      weigh(c, kWarps, v, false, M, sum);
      if (S > 1) {
        for (int i = 0; i < S; ++i) *cluster.map_shared_rank(reinterpret_cast<float2*>(smem + C::kMl) + rank * kCols + c, i) = make_float2(M, sum);
      } else if (cut) a.part_ml[slot * kCols + c] = make_float2(M, sum);
      else store_lse(c, M, sum);
    }
    if (a.ctas && threadIdx.x == 0) {  // the CTAs that have the first and the last step
      int32_t* const ends = a.ends + 2 * (static_cast<int64_t>(b) * per_seq + inner);
      if (s0 == 0) ends[0] = static_cast<int32_t>(blockIdx.x);
      if (s1 == per) ends[1] = static_cast<int32_t>(blockIdx.x);
      if (s0 == 0 && cut) a.starts[blockIdx.x] = static_cast<int32_t>(b) * per_seq + inner;
    }
    __syncthreads();
    // O^T in runs of 32 rows (a warp's, of channels that lie in a row) and four columns
    const int runs = D / 32 * ((GC + 3) / 4), slots = (runs + S - 1) / S;
    auto dim_of = [](int r) { return 32 * (r >> 5) + 4 * (r & 7) + 2 * ((r >> 4) & 1) + ((r >> 3) & 1); };
    float4* const in = reinterpret_cast<float4*>(smem + C::kIn);
    for (int run = warp; run < runs; run += kWarps) {
      const int r = 32 * (run % (D / 32)) + lane, c = 4 * (run / (D / 32)), dim = dim_of(r);
      float acc[4] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(red + (w * D + r) * kCols + c);
        const float4 f = *reinterpret_cast<const float4*>(wt + w * kCols + c);
        acc[0] = fmaf(v.x, f.x, acc[0]);
        acc[1] = fmaf(v.y, f.y, acc[1]);
        acc[2] = fmaf(v.z, f.z, acc[2]);
        acc[3] = fmaf(v.w, f.w, acc[3]);
      }
      if (S > 1) {  // run i is joined by CTA i % S of the cluster
        const int to = run % S;
        cluster.map_shared_rank(in, to)[(rank * slots + run / S) * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        continue;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c + i >= GC) break;
        if (cut) a.part_o[(slot * kCols + c + i) * D + dim] = acc[i];
        else store_out(a.out, a.out_dtype, row_of[c + i] * D + dim, acc[i]);
      }
    }
    if (S > 1) {  // what the cluster's CTAs have sent
      cluster_arrive();
      cluster_wait();
      if (threadIdx.x < GC) {
        const int c = threadIdx.x;
        float M, sum;
        float2 v[kMaxCluster] = {};
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i)
          if (i < S) v[i] = reinterpret_cast<const float2*>(smem + C::kMl)[i * kCols + c];
        weigh(c, S, v, true, M, sum);
        store_lse(c, M, sum);
      }
      __syncthreads();
      for (int n = warp; n * S + rank < runs; n += kWarps) {
        const int run = n * S + rank, r = 32 * (run % (D / 32)) + lane, c = 4 * (run / (D / 32)), dim = dim_of(r);
        float acc[4] = {};
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i)
          if (i < S) {
            const float4 v = in[(i * slots + n) * 32 + lane], f = *reinterpret_cast<const float4*>(wt + i * kCols + c);
            acc[0] = fmaf(v.x, f.x, acc[0]);
            acc[1] = fmaf(v.y, f.y, acc[1]);
            acc[2] = fmaf(v.z, f.z, acc[2]);
            acc[3] = fmaf(v.w, f.w, acc[3]);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < GC) store_out(a.out, a.out_dtype, row_of[c + i] * D + dim, acc[i]);
      }
    }
    if (!a.ctas) return;
    if (left <= 0) return;
    s0 = -C::kStart;
    if (++b == a.B) b = 0, ++inner;
    __syncthreads();  // the parts are read
  }
}

// The parts of each (sequence, kv head, column group) of a balanced launch that was cut.  D / 4 threads, a row, hold a
// column; `stripes` rows share its parts, each taking kAhead of them at once, and a CTA has kRows / stripes columns
// of one item: each of them in turn (kEach) or, where there are more than CTAs of the kernel above, of the one that such
// a CTA began and did not end, if it did.
constexpr int kJoin = 256, kAhead = 4;
constexpr float kJoinScale = 0x1p-32f;  // of the outputs' sums over parts, which may otherwise pass fp32 where the outputs do not
template <int D, bool kEach>
__global__ void __launch_bounds__(kJoin) decode4_combine_kernel(const Decode4Args a, int pad, int stripes) {
  constexpr int kRow = D / 4;
  __shared__ float4 sm[kJoin];
  __shared__ float2 sums[kJoin / kRow];
  const int per_seq = a.Hkv * a.groups, G = a.Hq / a.Hkv;
  const int q = static_cast<int>(threadIdx.x) % kRow, r = static_cast<int>(threadIdx.x) / kRow;
  const int columns = kJoin / kRow / stripes, ctas = (a.cols + columns - 1) / columns;  // of a CTA, of an item
  const int which = static_cast<int>(blockIdx.x) / ctas;
  const int c = (static_cast<int>(blockIdx.x) - which * ctas) * columns + r / stripes, stripe = r % stripes;
  grid_dependency_wait();
  const int item = kEach ? which : a.starts[which];
  if (item < 0) return;
  const int2 ends = reinterpret_cast<const int2*>(a.ends)[item];
  const int i0 = ends.x, i1 = ends.y;
  if (i0 == i1) return;  // written by that CTA
  const int b = item / per_seq, inner = item - b * per_seq;
  const int head = inner / a.groups, col0 = (inner - head * a.groups) * a.cols;
  const bool mine = c < min(a.cols, a.T * G - col0);
  auto slot_of = [&](int i) { return static_cast<int64_t>(2 * i + (i == i0 ? 1 : 0)); };
  float M = -INFINITY, sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = i0 + stripe; mine && i <= i1; i += kAhead * stripes) {
    float2 v[kAhead];
    float4 x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int j = i + k * stripes;
      const int64_t slot = slot_of(min(j, i1));
      v[k] = a.part_ml[slot * pad + c];
      x[k] = *reinterpret_cast<const float4*>(a.part_o + (slot * pad + c) * D + 4 * q);
      if (j > i1) v[k].x = -INFINITY;
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) top = fmaxf(top, v[k].x);
    const float keep = M == -INFINITY ? 0.0f : ex2(M - top);
    M = top;
    sum *= keep;
    acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (v[k].x == -INFINITY) continue;
      const float w = ex2(v[k].x - M) * v[k].y, f = w * kJoinScale;
      sum += w;
      acc.x = fmaf(f, x[k].x, acc.x);
      acc.y = fmaf(f, x[k].y, acc.y);
      acc.z = fmaf(f, x[k].z, acc.z);
      acc.w = fmaf(f, x[k].w, acc.w);
    }
  }
  if (stripes > 1) {
    sm[threadIdx.x] = acc;
    if (q == 0) sums[r] = make_float2(keep_nan(M, sum), sum);
    __syncthreads();
    if (stripe == 0) {
      for (int i = 1; i < stripes; ++i) M = fmaxf(M, sums[r + i].x);
      sum = 0.0f;
      acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int i = 0; i < stripes; ++i) {
        const float2 v = sums[r + i];
        if (v.x == -INFINITY) continue;
        const float f = ex2(v.x - M);
        const float4 x = sm[threadIdx.x + i * kRow];
        sum = fmaf(f, v.y, sum);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
      }
    }
  }
  if (!mine || stripe > 0) return;
  const int dr = (col0 + c) / G;
  const int64_t row = (static_cast<int64_t>(b) * a.T + dr) * a.Hq + head * G + (col0 + c - dr * G);
  const float x[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) store_out(a.out, a.out_dtype, row * D + 4 * q + i, sum == 0.0f ? 0.0f : x[i] / (sum * kJoinScale));
  if (a.lse && q == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

template <int D, int kCols, int kTerms>
cudaError_t launch_t(const Decode4Args& a, cudaStream_t s) {
  using C = Cfg4<D, kCols>;
  auto kern = decode4_kernel<D, kCols, kTerms>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), C::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned items = static_cast<unsigned>(a.B) * a.Hkv * a.groups;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas ? static_cast<unsigned>(a.ctas) : items * a.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.ctas ? 1 : a.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a, device_status_ptr());
  if (e != cudaSuccess || !a.ctas) return e;
  // rows of the combine that share a column's parts: as many as take them kMany times over at once, since lengths differ
  // (kMany 1, 2, 4, 8: 64 sequences of up to 8,192 tokens 70.6 us, 71.3, 73.2, 75.6; 48 of up to 16,384, d = 64, 34.4, 33.8, 34.1, 37.0)
  constexpr int kRows = kJoin / (D / 4), kMany = 2;
  const unsigned ctas = static_cast<unsigned>(a.ctas);
  int stripes = 1;
  while (stripes < kRows && stripes * kAhead < kMany * static_cast<int>(ctas / items + 2)) stripes *= 2;
  const unsigned each = (a.cols + kRows / stripes - 1) / (kRows / stripes);
  if (items <= ctas) return launch_pdl(decode4_combine_kernel<D, true>, dim3(items * each), dim3(kJoin), 0, s, a, kCols, stripes);
  return launch_pdl(decode4_combine_kernel<D, false>, dim3(ctas * each), dim3(kJoin), 0, s, a, kCols, stripes);
}

template <int D, int kCols>
cudaError_t launch_c(const Decode4Args& a, cudaStream_t s) {
  return a.out_dtype == SL8_F32 ? launch_t<D, kCols, 3>(a, s) : launch_t<D, kCols, 1>(a, s);
}

template <int D>
cudaError_t launch_d(const Decode4Args& a, cudaStream_t s) {
  if constexpr (D == 256) return launch_c<D, 8>(a, s);
  else return a.cols > 16 ? launch_c<D, 24>(a, s) : a.cols > 8 ? launch_c<D, 16>(a, s) : launch_c<D, 8>(a, s);
}

// CTAs of the kernel that fit the device at once.
template <int D>
int ctas_d(int32_t cols) {
  if constexpr (D == 256) return Cfg4<D, 8>::kCtas;
  else return cols > 16 ? Cfg4<D, 24>::kCtas : cols > 8 ? Cfg4<D, 16>::kCtas : Cfg4<D, 8>::kCtas;
}
int slots(int32_t d, int32_t cols) {
  return num_sms() * (d == 256 ? ctas_d<256>(cols) : d == 128 ? ctas_d<128>(cols) : d == 64 ? ctas_d<64>(cols) : ctas_d<32>(cols));
}

}  // namespace

int32_t decode4_max_columns(int32_t d) { return d == 256 ? 8 : 24; }

void decode4_plan_work(int64_t items, int64_t tokens, int32_t d, int32_t cols, int32_t num_splits, int32_t* splits,
                       int32_t* ctas) {
  const int64_t fit = slots(d, cols), many = 16ll * num_sms();
  *splits = 1;
  *ctas = 0;
  const bool counted = items < (int64_t(1) << 50) / (tokens + 1);  // steps and shares stay within 64 bits
  if (num_splits > kMaxCluster) {
    if (counted) *ctas = static_cast<int32_t>(std::min(items * std::min<int64_t>(num_splits, many), many));
    else *splits = kMaxCluster;
  } else if (num_splits > 0) {
    *splits = num_splits;
  } else {
    // A cluster for each item, of as many CTAs as fit one wave and have 128 tokens each, 1,024 where they are more than
    // two an SM, whose starts hold one another up (64 items of up to 1,024 tokens: 9.2 us with 4 CTAs each, 11.4 with 8); or even shares, if the table's
    // width says that a CTA's longest run could be longer than a share (of lengths that are five eighths of the width) by
    // what the second kernel and the ends of the shares cost: 1,000 tokens' time, 750 at d = 256.
    // One sequence, 8 heads: 8,192 tokens 13.8 us in clusters and 13.7 in shares, 65,536 53 and 27; 4,096 (512 a CTA) 10.3
    // and 12.8.  64 sequences of 256 to 2,048: 29.0 and 32.8, of 512 to 4,096: 50.7 and 47.4.  Only the device knows the
    // lengths: where tables are far wider, shares are taken that a cluster would beat (4 sequences of up to 2,048 tokens
    // 13.1 for 9.7 us, 64 of up to 512 22 for 14).
    while (*splits < kMaxCluster && items * (*splits + 1) <= fit && tokens / (*splits + 1) >= (items * (*splits + 1) <= 2 * num_sms() ? 128 : 1024))
      ++*splits;
    if (counted) {
      const int64_t share = items * tokens / fit, run = std::max(tokens / *splits, share);
      if (run - share * 5 / 8 >= (d == 256 ? 750 : 1000)) *splits = 1, *ctas = static_cast<int32_t>(fit);
    }
  }
}

size_t decode4_workspace(int64_t items, int32_t d, int32_t cols, int32_t ctas, size_t* ml, size_t* ends, size_t* starts) {
  const size_t slots = 2 * static_cast<size_t>(ctas), c = (cols + 7) / 8 * 8;
  *ml = slots * c * d * sizeof(float);
  *ends = *ml + slots * c * sizeof(float2);
  *starts = *ends + static_cast<size_t>(items) * 2 * sizeof(int32_t);
  return *starts + static_cast<size_t>(ctas) * sizeof(int32_t);
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
