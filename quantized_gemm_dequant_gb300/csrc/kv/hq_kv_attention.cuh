// Attention of one new token per sequence over a paged cache, split over the cache's length and joined.
//
//   s_j = scale (q . k_j);   m = max_j s_j;   l = sum_j exp(s_j - m);   o = (1 / l) sum_j exp(s_j - m) v_j
//
// in one pass over the cache: a part of the tokens keeps its own m, l and unnormalised o, and parts (m1, l1, o1),
// (m2, l2, o2) join to m = max(m1, m2), l = l1 e^(m1 - m) + l2 e^(m2 - m), o alike.  Everything is in powers of two
// (scores are multiplied by log2 e once), in fp32.
//
// What bounds it: the cache is read once and 4 G operations are done per key-value pair of elements for the G query
// heads that share a head.  bf16 and e4m3 caches are bound by memory up to G = 8 (with 12 and 16, on one or two CTAs per
// SM less, they reach 71% and 59% of the copy's rate), NVFP4 by the instructions that decode it.  The work is laid out to
// read the cache once:
//  - The tokens of all (sequence, head) pairs form one list of small units, cut into equal shares for a fixed number of
//    CTAs, whatever the lengths are.  A pair inside one share is finished there; one that crosses shares leaves fp32
//    partial results in the workspace, and the last CTA to arrive joins them in order.  The lengths are read on the
//    device, so a captured call follows them.
//  - The four warps of a CTA each stream every fourth chunk of 16 or 32 tokens through a ring of their own in shared
//    memory (cp.async, 16 bytes a lane); no barrier but the warp's own until a pair's parts are joined.  The ring runs
//    ahead across pairs.  Two or three CTAs per SM, as their registers allow, hide each other's ends of pairs.
//  - Products run on mma.sync m16n8k16 with 16 tokens as the rows and 8 query heads as the columns, s^T = K q^T and
//    o^T = V^T p^T: the codes are the A operand of both, so their decoding is shared by up to 16 heads, and a group of
//    8 heads wastes nothing.  Between the two, movmatrix turns p.  (A tcgen05 tile would need the decoded operands
//    back in shared memory; the legacy unit is at a fifth of its rate here.)
//  - 8- and 4-bit codes go from shared memory through ldmatrix to registers and become f16 there, exactly.  The
//    fragments' dims are permuted so that a lane's bytes are its own: the dot product does not care about the order of
//    dims if q follows it, and the output's order is undone when it is stored.
//  - e4m3: a token's key scale multiplies its score.  Its value scale v multiplies its weight, and a weight must fit
//    f16: o's weights are exp2(s_j - m + log2 v_j - d) with a running d of their own, the largest of what stands before
//    it, so that the largest weight times its scale is about one whatever the scales' range, while l sums exp2(s_j - m)
//    in fp32.  (By one maximum for both, a value scale 2^126 times the others before it took their weights out of l.)
//    A scale of zero has a weight of zero in o and its own in l; o / l is multiplied by 2^d at the end.
//  - nvfp4: code * block scale is exact in f16 (2 + 4 significant bits); the global scales go to q's scale and to o.
//  - Queries of the f16 kinds are scaled by a power of two per row that takes the largest element to [2^14, 2^15): a bf16
//    element keeps its bits down to 2^-31 of that one, loses them one by one below and is zero under 2^-39 of it.
//  - The running maximum only moves when a score exceeds it by 8 (powers of two): a vote finds that out, so that the
//    steady state has no shuffles and o is seldom rescaled; weights up to 2^8 fit the 16-bit types.  f16's are 2^7 times
//    that (what stands for the maximum is 7 less): they keep their bits down to 2^-21 of the largest and vanish under
//    2^-32 of it, beside a token that holds nearly all of the weight (l has them in fp32).  bf16 has 8 bits: a weight
//    is the sum of two of them, 15 bits, and the values are multiplied by both, which costs a kernel that waits for
//    memory nothing (24 ragged sequences: 43.1 us with one, 43.0 with two).  f16's 11 bits are one: what they round off
//    is an eighth of the output's own rounding.
//
// Measured on a GB300 (6.69 TB/s measured copy), 8 query heads of 128 dims per key-value head unless said: bf16, 24
// sequences of up to 5000 tokens, 4 query heads: 43.3 us, 88% of copy; e4m3, 64 of up to 16384: 93.9 us, 88%; e4m3, one
// of 131072, 4 query heads: 52.9 us, 78%; bf16, 33 with a window of 1024, 2 query heads of 256 dims: 27.4 us, 72%; NVFP4,
// 128 of up to 8192: 133 us, 69% (710 instructions per 32 tokens and warp, 2.1 issued a cycle, the integer pipe busy half
// of the time).  NVFP4 otherwise: heads of 64 dims 46%, 16 query heads 46 to 49%, 256 sequences of up to 600 tokens 35%.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../hq_launch.h"
#include "../hq_ptx.cuh"
#include "hq_kv.h"
#include "hq_kv_codec.cuh"

namespace hq {

constexpr int KA_WARPS = 4;
constexpr int KA_THREADS = 32 * KA_WARPS;
constexpr int KA_ROWS = 16;          // query heads of one row tile, at most
constexpr float KA_LAZY = 8.0f;      // the running maximum lags by at most this (log2)
constexpr float KA_LEAD = 7.0f;      // f16 weights are 2^7 times what they would be: 2^15 at most
constexpr int KA_GROUP = 16;         // CTAs whose parts of a pair with many are joined first, to one part
constexpr int KA_MANY = 24;          // parts from more than which that is done
constexpr int KA_MOST = 32 * KA_GROUP;  // CTAs, so that a join has 32 parts at most
constexpr float KA_NONE = -3.0e38f;  // the running maximum of no token

// 16-token blocks per chunk and unit of the list: two where a chunk's ring steps leave room for three of them (NVFP4 with
// one: 154 us instead of 133, the copies' bookkeeping); resident CTAs per SM: what the registers allow without spills
// (the batches above with two, three and four, which spill: NVFP4 147, 133, 155 us; bf16 45.4, 43.4, 49.9; e4m3 93.6,
// 94.0, 97.7).
__host__ __device__ constexpr int ka_blocks(int kind, int dim) {
  return kind == HQ_KV_NVFP4 ? (dim == 256 ? 1 : 2) : (kind == HQ_KV_E4M3 && dim == 64 ? 2 : 1);
}
__host__ __device__ constexpr int ka_ctas(int kind, int dim, int nt) {
  return dim == 256 ? 2 : (nt == 2 ? 2 : 3);
}

// Beginning and ending a pair costs a CTA about as long as streaming so many bytes (3 to 4 us): so many units of the list
// are the pair's own.  Without them the CTAs with more pairs were up to a fifth later than the others (a batch of 64 e4m3
// sequences: 99 us, with them 94 to 96).
__host__ __device__ constexpr int ka_extra(int kind, int dim) {
  return (kind == HQ_KV_NVFP4 ? 49152 : 81920) /
         (2 * ka_blocks(kind, dim) * KV_BLOCK * (kv_row_bytes(kind, dim) + kv_scale_bytes(kind, dim)));
}

// Workspace of a call, for the host (sizes) and the device: the status, then two slots per CTA for the parts of split
// pairs, then two counters per KA_GROUP CTAs, then one per (sequence, head, row tile).  The slots' room is that of the
// largest format, so that the counters, which have to be zero between calls, are at one place whatever the calls' shapes
// are.
constexpr size_t KA_SLOT_FLOATS = KA_ROWS * (256 + 3);  // o, then (m, l) and d of each row, of 16 heads of 256 dims
constexpr int KA_MOST_CTAS = 2;                         // per SM, of that size
constexpr size_t ka_group_counters_at(int sms) {
  return KV_HEADER_BYTES + 2 * (size_t)(KA_MOST_CTAS * sms) * KA_SLOT_FLOATS * sizeof(float);
}
constexpr size_t ka_counters_at(int sms) {
  return ka_group_counters_at(sms) + 2 * (KA_MOST / KA_GROUP) * sizeof(int);
}

template <int KIND, int D, int NT>
struct KaCfg {
  static constexpr int RB = kv_row_bytes(KIND, D), SB = kv_scale_bytes(KIND, D);
  static constexpr int TB = ka_blocks(KIND, D);      // 16-token blocks of one chunk
  static constexpr int BLOCK = 16 * (RB + SB);       // a block's codes, then its scales
  static constexpr int SIDE = TB * BLOCK;            // a chunk's keys, or its values
  // A ring step is a chunk's keys and values, one wait and one look at the table for both; of bf16, which has twice the
  // bytes, it is one side.  (Of e4m3 heads of 256 dims one side a step makes five steps of two: 80 us -> 86.)
  static constexpr bool PAIR = KIND != HQ_KV_BF16;
  static constexpr int STEP = PAIR ? 2 * SIDE : SIDE;
  static constexpr int SUMS = KIND == HQ_KV_BF16 ? 2 : 1;  // of a score: every other 16 dims of bf16 apart, a shorter chain
  static constexpr int EXTRA = ka_extra(KIND, D);
  static constexpr int CTAS = ka_ctas(KIND, D, NT);  // resident per SM
  static constexpr bool OD = KIND == HQ_KV_E4M3;     // o has a running maximum of its own, d over m
  static constexpr size_t PART = 8 * NT * (D + (OD ? 3 : 2));  // floats of a part: o, then (m, l), then d of each head
  static constexpr float LEAD = KIND == HQ_KV_NVFP4 ? KA_LEAD : 0.0f;  // m is the maximum less this; d: less KA_LEAD
  static constexpr int ML = OD ? 3 : 2;              // floats of a head in shared memory: m, l, d
  static_assert(CTAS * PART <= KA_MOST_CTAS * KA_SLOT_FLOATS, "workspace");
  static constexpr int PAD = 4;                      // floats: the lanes' stores of a head's dims meet no bank twice
  // heads of every warp that are joined at a time: with eight of 256 dims the ring of bf16 would have two steps instead
  // of three (33 sequences with a window of 1024: 28.1 us, so 27.4)
  static constexpr int JOIN = KIND == HQ_KV_BF16 && D == 256 && NT == 1 ? 4 : 8;
  static constexpr int MERGE = KA_WARPS * JOIN * (D + PAD) * 4;
  static constexpr bool QS = D == 256 && NT == 2;    // q's fragments in shared memory instead of registers
  static constexpr int QBYTES = QS ? D / 16 * NT * 256 : 0;
  static constexpr int FIXED = MERGE + QBYTES + 128 + KA_WARPS * 8 * ML * 4;
  static constexpr int LIMIT = (228 * 1024) / CTAS / 128 * 128 - 1024;  // shared memory of a CTA
  static constexpr int FIT = (LIMIT - FIXED) / (KA_WARPS * (STEP + 4));
  static constexpr int DEPTH = FIT < 2 ? 2 : (FIT > 12 ? 12 : FIT);  // ring steps
  static constexpr int SMEM = FIXED + KA_WARPS * DEPTH * (STEP + 4);
  static_assert(SMEM <= LIMIT, "shared memory");
  // unit u (16 bytes) of row r sits at u ^ ((r / RPL) & XM), so that eight rows' equal units lie in different banks
  static constexpr int UPR = RB / 16;
  static constexpr int RPL = UPR >= 8 ? 1 : 8 / UPR;  // rows of a 128-byte line
  static constexpr int XM = (UPR >= 8 ? 8 : UPR) - 1;
  static __device__ __forceinline__ uint32_t at(int r, int u) {
    return (uint32_t)(r * RB + ((u ^ ((r / RPL) & XM)) << 4));
  }
};

#ifdef __CUDACC__

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// transpose of an 8 x 8 matrix of 16-bit values, a row's pair per lane
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// the four bytes of x, two e2m1 codes each -> four f16x2
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t x, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "mov.b32 {t0, t1, t2, t3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t0;\n\tcvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, t2;\n\tcvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(x));
}
// both halves the low, or the high half
template <int HALF>
__device__ __forceinline__ uint32_t dup16(uint32_t x) {
  uint32_t d;
  if constexpr (HALF)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(d) : "r"(x));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(d) : "r"(x));
  return d;
}

// L2 line i of a range, if it has one
__device__ __forceinline__ void ka_prefetch(const void* p, int64_t bytes, int64_t i) {
  if (i * 128 < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"((const char*)p + i * 128));
}

// counter + 1, ordered after the CTA's writes (made visible by its barrier) and before its later reads
__device__ __forceinline__ int count_up(int* counter) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}

// The list cut into W nearly equal shares: the first `more` of them have q + 1 units, the others q.
struct KaShares {
  uint32_t W, q, more;
  // least: units of a share at least, for few tokens
  __device__ __forceinline__ KaShares(uint32_t total, uint32_t grid, uint32_t least) {
    W = (total + least - 1) / least;
    W = W < grid ? W : grid;
    q = total / W;
    more = total - q * W;
  }
  __device__ __forceinline__ uint32_t first(uint32_t c) const { return c * q + (c < more ? c : more); }
  __device__ __forceinline__ uint32_t owner(uint32_t u) const {
    const uint32_t big = more * (q + 1);
    return u < big ? u / (q + 1) : more + (u - big) / q;
  }
};

template <bool V>
struct KaFlag {
  static constexpr bool value = V;
};

// One sequence's place in the list of units.
struct KaSeq {
  int n, j0, t0;   // tokens, the first that is seen, and that one's block
  uint32_t units;  // per (head, row tile): X for the pair itself, then its tokens' (one at least: an empty sequence's
                   // output is written too)
};
template <int TB, int X>
__device__ __forceinline__ KaSeq ka_seq(const KvAttnArgs& a, int64_t b) {
  KaSeq s;
  int64_t n = a.lens[b];
  n = n < 0 ? 0 : (n > a.most ? a.most : n);
  const int64_t j0 = a.window > 0 && n > a.window ? n - a.window : 0;
  s.n = (int)n;
  s.j0 = (int)j0;
  s.t0 = s.j0 & ~(KV_BLOCK - 1);
  const uint32_t u = (uint32_t)(s.n - s.t0 + 16 * TB - 1) / (16 * TB);
  s.units = X + (u > 0 ? u : 1);
  return s;
}

// A walk over a CTA's share, one (sequence, head, row tile) after another.
template <int TB, int X>
struct KaWalk {
  uint32_t u, hi;  // position in the list, end of the share
  uint32_t seg0;   // the pair's first unit in the list
  int b;
  int hr;          // head * tiles + tile
  KaSeq s;
  __device__ __forceinline__ bool done() const { return u >= hi; }
  __device__ __forceinline__ uint32_t stop() const { return seg0 + s.units < hi ? seg0 + s.units : hi; }
  // the share's part of the pair: whether there are tokens' units in it, and all of them; the tokens
  __device__ __forceinline__ bool any() const { return stop() > seg0 + X; }
  __device__ __forceinline__ bool whole() const { return u <= seg0 + X && stop() == seg0 + s.units; }
  __device__ __forceinline__ int from() const { return s.t0 + (u > seg0 + X ? (int)((u - seg0 - X) * (16 * TB)) : 0); }
  __device__ __forceinline__ int to() const {
    const int t = s.t0 + (any() ? (int)((stop() - seg0 - X) * (16 * TB)) : 0);
    return t < s.n ? t : s.n;
  }
  __device__ __forceinline__ void next(const KvAttnArgs& a, int hrs) {
    u = stop();
    if (u >= hi) return;
    seg0 = u;
    if (++hr == hrs) {
      hr = 0;
      s = ka_seq<TB, X>(a, ++b);
    }
  }
};

// s -> cap tanh(s / cap).  Near zero tanh's Taylor series up to t^9, so that a score far below the cap keeps its relative
// error: 1 - 2 / (1 + e^2t) there is a difference of two numbers near 1, off by cap 2^-23 (a cap of 1e5: scores off by
// 0.01).  The series' remainder is under 2^-26 of t where the two meet.
__device__ __forceinline__ void ka_cap(float& s, float cap, float per_cap) {
  const float t = s * per_cap, t2 = t * t, y = t * 2.8853900817779268f;  // 2 log2 e
  const float p = fmaf(t2, fmaf(t2, fmaf(t2, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f), -1.0f / 3.0f);
  const float far = cap * (1.0f - __fdividef(2.0f, 1.0f + ex2(y > 80.0f ? 80.0f : y)));
  s = fabsf(t) < 0.25f ? fmaf(s * t2, p, s) : far;
}

// One row's result: 4 dims of o (over: its maximum over m), and lse
template <bool OD>
__device__ __forceinline__ void ka_store(const KvAttnArgs& a, int64_t q, int D, int d, float4 y, float over, float m,
                                         float sum, float gain) {
  const float inv = sum == 0.0f ? 0.0f : gain / sum;  // a NaN stays one
  y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
  if constexpr (OD) {  // by 2^over in two steps: half of it is never out of range
    const float h = ex2(0.5f * over);
    y.x = y.x * h * h, y.y = y.y * h * h, y.z = y.z * h * h, y.w = y.w * h * h;
  }
  *reinterpret_cast<uint2*>(a.out + q * D + d) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  if (d == 0 && a.lse) a.lse[q] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

// Joins at most 32 parts of a split pair in order: slot `first`, then slots others + k apart.  The result goes to the
// pair's rows, or, as one part, to slot `first` again.  Bound by latency: a thread's 16 to 32 loads of o are in flight
// while a warp per head finds the factors 2^(m - top), a part per lane.
template <int KIND, int D, int NT>
__device__ __forceinline__ void ka_join(const KvAttnArgs& a, float* slots, uint32_t first, uint32_t others,
                                        uint32_t apart, int parts, bool to_part, int64_t q0, int rows, float vg,
                                        float* merge, float* mls) {
  using C = KaCfg<KIND, D, NT>;
  constexpr int MINE = 8 * NT * (D / 4) / KA_THREADS, AHEAD = MINE >= 4 ? 4 : 16 / MINE, HEADS = 8 * NT / KA_WARPS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto part_at = [&](int k) { return slots + (k ? others + k * apart : first) * C::PART; };
  float* factor = merge;  // [head][32]
  float* tops = mls;      // [head][ML]: top, sum, o's top over it
  float4 v[AHEAD][MINE], y[MINE];
  auto take = [&](int k0) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int e = 4 * (threadIdx.x + i * KA_THREADS);
        v[k][i] = k0 + k < parts && e < rows * D ? __ldcg(reinterpret_cast<const float4*>(part_at(k0 + k) + e))
                                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
  };
  take(0);
  float2 ml[HEADS];
  float over[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int r = warp + i * KA_WARPS;
    ml[i] = lane < parts && r < rows ? __ldcg(reinterpret_cast<const float2*>(part_at(lane) + 8 * NT * D + 2 * r))
                                     : make_float2(KA_NONE, 0.0f);
    over[i] = C::OD && lane < parts && r < rows ? __ldcg(part_at(lane) + 8 * NT * (D + 2) + r) : KA_NONE;
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int r = warp + i * KA_WARPS;
    float top = ml[i].x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float f = ex2(ml[i].x - top), sum = f * ml[i].y, otop = KA_NONE;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (C::OD) {
      const float y = ml[i].x - top + over[i];
      otop = fmaxf(otop, y);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) otop = fmaxf(otop, __shfl_xor_sync(0xffffffffu, otop, o));
      f = ex2(y - otop);
    }
    factor[r * 32 + lane] = f;
    if (lane == 0) {
      tops[C::ML * r] = top, tops[C::ML * r + 1] = sum;
      if constexpr (C::OD) tops[C::ML * r + 2] = otop;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MINE; ++i) y[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int k0 = 0;;) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int r = 4 * (threadIdx.x + i * KA_THREADS) / D;
        const float f = k0 + k < parts ? factor[r * 32 + k0 + k] : 0.0f;
        y[i].x = fmaf(f, v[k][i].x, y[i].x), y[i].y = fmaf(f, v[k][i].y, y[i].y);
        y[i].z = fmaf(f, v[k][i].z, y[i].z), y[i].w = fmaf(f, v[k][i].w, y[i].w);
      }
    k0 += AHEAD;
    if (k0 >= parts) break;
    take(k0);
  }
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    const int e = 4 * (threadIdx.x + i * KA_THREADS), r = e / D, d = e % D;
    if (r >= rows) continue;
    const float top = tops[C::ML * r], sum = tops[C::ML * r + 1], otop = C::OD ? tops[C::ML * r + 2] : 0.0f;
    if (!to_part) {
      ka_store<C::OD>(a, q0 + r, D, d, y[i], otop, top, sum, vg);
    } else {  // (all (m, l) have been read, and o's dims are this thread's alone)
      __stcg(reinterpret_cast<float4*>(part_at(0) + e), y[i]);
      if (d == 0) {
        __stcg(reinterpret_cast<float2*>(part_at(0) + 8 * NT * D + 2 * r), make_float2(top, sum));
        if constexpr (C::OD) __stcg(part_at(0) + 8 * NT * (D + 2) + r, otop);
      }
    }
  }
  __syncthreads();  // the next pair's join writes where this one's was read
}

// A split pair whose part this CTA has written: the last CTA to arrive joins the parts, first to last; of many, the last
// of every KA_GROUP CTAs joins theirs first.  The pair's units are seg0 .. end - 1 of the list.  A function of its own,
// so that its registers are not the main loop's.
template <int KIND, int D, int NT>
__device__ __noinline__ void ka_split(const KvAttnArgs& a, const KaShares sh, uint32_t seg0, uint32_t end, int64_t pair,
                                      float* slots, int* groups, int* counters, int* last_one, int64_t q0, int rows,
                                      float vg, float* merge, float* mls) {
  const uint32_t c0 = sh.owner(seg0 + KaCfg<KIND, D, NT>::EXTRA), c1 = sh.owner(end - 1);
  const uint32_t s0 = 2 * c0 + (sh.first(c0) >= seg0 ? 0 : 1);  // the first part's slot; others' first pair is this
  auto last_of = [&](int* counter, uint32_t n) {  // whether this CTA is; its part is written
    __syncthreads();  // the counter's release and acquire order it and the others' parts
    if (threadIdx.x == 0) {
      *last_one = count_up(counter) == (int)(n - 1);
      if (*last_one) *counter = 0;
    }
    __syncthreads();
    return *last_one != 0;
  };
  uint32_t parts = c1 - c0 + 1, others = 2 * c0, apart = 2;
  if (parts > KA_MANY) {
    const uint32_t gr = blockIdx.x / KA_GROUP, from = c0 > gr * KA_GROUP ? c0 : gr * KA_GROUP;
    const uint32_t n = (c1 < gr * KA_GROUP + KA_GROUP - 1 ? c1 : gr * KA_GROUP + KA_GROUP - 1) - from + 1;
    if (n > 1) {  // two counters: a pair that comes from the group before, one that begins in this group and leaves it
      if (!last_of(groups + 2 * gr + (c0 < gr * KA_GROUP ? 0 : 1), n)) return;
      ka_join<KIND, D, NT>(a, slots, from == c0 ? s0 : 2 * from, 2 * from, 2, n, true, q0, rows, vg, merge, mls);
    }
    parts = c1 / KA_GROUP - c0 / KA_GROUP + 1;
    others = 2 * (c0 / KA_GROUP * KA_GROUP);
    apart = 2 * KA_GROUP;
  }
  if (last_of(counters + pair, parts))
    ka_join<KIND, D, NT>(a, slots, s0, others, apart, parts, false, q0, rows, vg, merge, mls);
}

template <int KIND, int D, int NT>
__global__ void __launch_bounds__(KA_THREADS, KaCfg<KIND, D, NT>::CTAS)
    kv_attention_kernel(const KvAttnArgs a, float* slots, int* groups, int* counters) {
  using C = KaCfg<KIND, D, NT>;
  constexpr bool BF = KIND == HQ_KV_BF16, F8 = KIND == HQ_KV_E4M3;
  constexpr int KS = D / 16, TB = C::TB, STRIDE = 16 * TB * KA_WARPS;
  constexpr uint32_t FULL = TB == 1 ? 0xFFFFu : 0xFFFFFFFFu;
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem);
  uint32_t* qsm = reinterpret_cast<uint32_t*>(smem + C::MERGE);
  int* found = reinterpret_cast<int*>(smem + C::MERGE + C::QBYTES);  // 2 words
  int* last_one = found + 2;
  float* mls = reinterpret_cast<float*>(smem + C::MERGE + C::QBYTES + 128);  // [warp][8 heads][ML]
  int64_t* scan = reinterpret_cast<int64_t*>(mls);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + C::FIXED + warp * C::DEPTH * C::STEP;
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + C::FIXED + KA_WARPS * C::DEPTH * C::STEP) + warp * C::DEPTH;
  const uint32_t ring_at = smem_u32(ring);
  pdl_trigger();
  // While the previous kernel ends, the lengths and the page table move to L2 (a hint: nothing is read before the wait).
  ka_prefetch(a.lens, a.B * 4, (int64_t)blockIdx.x * KA_THREADS + threadIdx.x);
  ka_prefetch(a.page_table, a.B * a.table_stride * 4, (int64_t)(gridDim.x - 1 - blockIdx.x) * KA_THREADS + threadIdx.x);
  pdl_wait();

  // ---- this CTA's share of the units
  const int G = a.group, tiles = (G + KA_ROWS - 1) / KA_ROWS, H = a.kv.heads, hrs = H * tiles;
  const int64_t per = (a.B + KA_THREADS - 1) / KA_THREADS;
  const int64_t b0 = per * threadIdx.x < a.B ? per * threadIdx.x : a.B, b1 = b0 + per < a.B ? b0 + per : a.B;
  int64_t mine = 0;
  for (int64_t b = b0; b < b1; ++b) {
    mine += ka_seq<TB, C::EXTRA>(a, b).units;
    if (blockIdx.x == 0 && (a.lens[b] < 0 || a.lens[b] > a.most)) kv_report(a.status);
  }
  int64_t before = mine;  // inclusive sum over the warp's lanes, then exclusive over the CTA
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  if (lane == 31) scan[warp] = before;
  before -= mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < KA_WARPS; ++w) {
    const int64_t y = scan[w];
    if (w < warp) before += y;
    total += y;
  }
  total *= hrs;
  if (total > INT32_MAX) {  // the list is counted in 32 bits
    if (threadIdx.x == 0) kv_report(a.status);
    return;
  }
  const KaShares sh((uint32_t)total, gridDim.x, 4 + C::EXTRA);
  if (blockIdx.x >= sh.W) return;
  const uint32_t lo = sh.first(blockIdx.x), start = (uint32_t)before * hrs;
  if (lo >= start && lo < start + (uint32_t)mine * hrs) {
    uint32_t p = start;
    for (int64_t b = b0; b < b1; ++b) {
      const uint32_t n = (b1 - b0 == 1 ? (uint32_t)mine : ka_seq<TB, C::EXTRA>(a, b).units) * hrs;
      if (lo < p + n) {
        found[0] = (int)b;
        found[1] = (int)p;
        break;
      }
      p += n;
    }
  }
  __syncthreads();
  KaWalk<TB, C::EXTRA> at;
  at.u = lo;
  at.hi = sh.first(blockIdx.x + 1);
  at.b = found[0];
  at.s = ka_seq<TB, C::EXTRA>(a, at.b);
  const uint32_t in = lo - (uint32_t)found[1];
  at.hr = (int)(in / at.s.units);
  at.seg0 = lo - (in - at.hr * at.s.units);

  // ---- the ring's front: this warp's chunks of the share, keys and values alternating
  KaWalk<TB, C::EXTRA> ahead = at;
  int next_tok = ahead.from() + 16 * TB * warp, next_end = ahead.to();
  int place = -1;       // lane i: the place in the pools (in blocks) of the warp's i-th block since the last table look
  int used = 32;        // blocks of it that are used up
  bool more = true;     // false: all of the share has been asked for
  int put = 0, get = 0;
  bool values = false;  // the side that is next (one side a step)
  uint32_t word = 0;    // tokens of the chunk that are seen
  int base[TB];         // its blocks' places
  auto next_chunk = [&]() {
    while (next_tok >= next_end) {  // the share's next pair
      ahead.next(a, hrs);
      more = !ahead.done();
      if (!more) return;
      next_tok = ahead.from() + 16 * TB * warp, next_end = ahead.to(), used = 32;
    }
    if (used == 32) {
      const int64_t tok = (int64_t)next_tok + STRIDE * (lane / TB) + 16 * (lane % TB);
      place = -1;
      if (tok < next_end) {
        const int col = (int)((uint32_t)tok / (uint32_t)a.kv.page_size);
        const int64_t page = a.page_table[(int64_t)ahead.b * a.table_stride + col];
        if (page >= 0 && page < a.kv.num_pages)
          place = (int)(((page * H + ahead.hr / tiles) * a.kv.page_size + ((int)tok - col * a.kv.page_size)) / KV_BLOCK);
        else
          kv_report(a.status);
      }
      used = 0;
    }
    const int first = ahead.s.j0 - next_tok, last = ahead.s.n - next_tok;
    word = FULL;
    if (first > 0) word &= FULL << first;
    if (last < 16 * TB) word &= FULL >> (16 * TB - last);
#pragma unroll
    for (int i = 0; i < TB; ++i) {
      base[i] = __shfl_sync(0xffffffffu, place, used + i);
      if (base[i] < 0) word &= ~(0xFFFFu << (16 * i)), base[i] = 0;
    }
    used += TB;
    next_tok += STRIDE;
  };
  // one side of the chunk; rows that are not seen are zero: whatever they hold meets a weight of zero, and may be NaN
  auto copy_side = [&](const uint8_t* pool, const uint8_t* scale_pool, uint32_t to, auto whole) {
    constexpr bool all = decltype(whole)::value;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const uint8_t* codes = pool + (uint64_t)(uint32_t)base[t] * (16 * C::RB) + lane * 16;
      const uint32_t w = word >> (16 * t);
#pragma unroll
      for (int i = 0; i < C::RB / 32; ++i) {
        const int r = (lane + 32 * i) / C::UPR;
        const uint32_t at = to + t * C::BLOCK + C::at(r, (lane + 32 * i) % C::UPR);
        if constexpr (all) copy16(at, codes + 512 * i);
        else copy16_or_zero(at, codes + 512 * i, (w >> r) & 1u ? 16u : 0u);
      }
    }
    if constexpr (C::SB > 0) {  // SB lanes a block
      constexpr int ONCE = TB * C::SB <= 32 ? TB : 1;
#pragma unroll
      for (int t = 0; t < TB; t += ONCE) {
        if (lane < ONCE * C::SB) {
          const int k = ONCE > 1 && lane >= C::SB ? 1 : 0, l = lane - k * C::SB;
          const uint8_t* scales = scale_pool + (uint64_t)(uint32_t)(k ? base[TB - 1] : base[t]) * (16 * C::SB) + 16 * l;
          const uint32_t at = to + (t + k) * C::BLOCK + 16 * C::RB + 16 * l;
          if constexpr (all) copy16(at, scales);
          else copy16_or_zero(at, scales, (word >> (16 * (t + k))) & 0xFFFFu ? 16u : 0u);
        }
      }
    }
  };
  auto issue = [&]() {  // one ring step
    if ((C::PAIR || !values) && more) next_chunk();
    if (more) {
      const uint32_t to = ring_at + put * C::STEP;
      auto copy = [&](auto whole) {
        if constexpr (C::PAIR) {
          copy_side(a.kv.k, a.kv.k_scale, to, whole);
          copy_side(a.kv.v, a.kv.v_scale, to + C::SIDE, whole);
        } else {
          copy_side(values ? a.kv.v : a.kv.k, nullptr, to, whole);
        }
      };
      if (word == FULL) copy(KaFlag<true>());
      else copy(KaFlag<false>());
      if (lane == 0) masks[put] = word;
    }
    cp_async_commit();
    put = put + 1 == C::DEPTH ? 0 : put + 1;
    values = !values;
  };
#pragma unroll 1
  for (int i = 0; i < C::DEPTH - 1; ++i) issue();

  float kg = 1.0f, vg = 1.0f;
  if constexpr (KIND == HQ_KV_NVFP4) {
    kg = *a.kv.k_global;
    vg = *a.kv.v_global;
  }
  const float cap = a.softcap * 1.4426950408889634f;
  const float per_cap = fminf(1.0f / cap, 3.4e38f);  // (a subnormal cap's is infinite)

  // ---- one pair after another
  for (; !at.done(); at.next(a, hrs)) {
    if (!at.any()) continue;  // the share ends before the pair's first token
    const int h = at.hr / tiles, r0 = (at.hr - h * tiles) * KA_ROWS, rows = G - r0 < KA_ROWS ? G - r0 : KA_ROWS;
    const int64_t q0 = ((int64_t)at.b * H + h) * G + r0;  // the tile's first query head
    uint32_t qb[C::QS ? 1 : KS][NT][2];  // B fragments: head 8 x + g, two pairs of dims of each 16-dim step
    float qscale[NT][2];                 // of heads 8 x + 2 c and the next
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      uint32_t raw[KS][2];
      const bool live = 8 * x + g < rows;
      const uint16_t* p = a.q + (q0 + 8 * x + g) * D;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int d0 = BF ? 16 * s + 2 * c : (F8 ? 16 * s + 4 * c : 32 * (s / 2) + 8 * c + 4 * (s & 1));
        const int d1 = BF ? d0 + 8 : d0 + 2;
        raw[s][0] = live ? *reinterpret_cast<const uint32_t*>(p + d0) : 0u;
        raw[s][1] = live ? *reinterpret_cast<const uint32_t*>(p + d1) : 0u;
      }
      float back = 1.0f;
      if constexpr (!BF) {
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(raw[s][i])), fabsf(bf16_hi(raw[s][i]))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = (int)(__float_as_uint(top) >> 23) - 127 - 14;  // the largest magnitude goes to [2^14, 2^15)
        e = top == 0.0f ? 0 : (e < -126 ? -126 : (e > 113 ? 113 : e));  // (both powers are normal numbers; 128: infinite)
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
        back = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i) raw[s][i] = pack_f16x2(bf16_lo(raw[s][i]) * f, bf16_hi(raw[s][i]) * f);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        qscale[x][k] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + k)) * kg * a.scale * 1.4426950408889634f;
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if constexpr (C::QS) {
          if (warp == 0)
            *reinterpret_cast<uint2*>(qsm + ((s * NT + x) * 32 + lane) * 2) = make_uint2(raw[s][0], raw[s][1]);
        } else {
          qb[s][x][0] = raw[s][0];
          qb[s][x][1] = raw[s][1];
        }
      }
    }
    if constexpr (C::QS) __syncthreads();
    auto qfrag = [&](int s, int x, uint32_t (&f)[2]) {
      if constexpr (C::QS) {
        const uint2 v = *reinterpret_cast<const uint2*>(qsm + ((s * NT + x) * 32 + lane) * 2);
        f[0] = v.x, f[1] = v.y;
      } else {
        f[0] = qb[s][x][0], f[1] = qb[s][x][1];
      }
    };
    float o[KS][NT][4];  // o^T: 16 dims by 8 heads
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][x][i] = 0.0f;
    float m[NT][2], l[NT][2], od[C::OD ? NT : 1][2];  // od: o's maximum over m
#pragma unroll
    for (int x = 0; x < NT; ++x) m[x][0] = m[x][1] = KA_NONE, l[x][0] = l[x][1] = 0.0f;
#pragma unroll
    for (int x = 0; x < (C::OD ? NT : 1); ++x) od[x][0] = od[x][1] = KA_NONE;

    const int end = at.to();
#pragma unroll 1
    for (int tok = at.from() + 16 * TB * warp; tok < end; tok += STRIDE) {
      // ---- keys: s^T = K q^T
      cp_async_wait_group<C::DEPTH - 2>();
      __syncwarp();
      issue();
      const uint32_t kslot = ring_at + get * C::STEP;
      uint8_t* kslot_p = ring + get * C::STEP;
      const uint32_t seen = masks[get];
      get = get + 1 == C::DEPTH ? 0 : get + 1;
      const int lr = lane & 15, lu = lane >> 4;  // ldmatrix: 16 tokens by two units
      float s[TB][NT][4];
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const uint32_t kb = kslot + t * C::BLOCK;
        const uint8_t* kscale = kslot_p + t * C::BLOCK + 16 * C::RB;
        float s2[C::SUMS][NT][4];
#pragma unroll
        for (int i = 0; i < C::SUMS * NT * 4; ++i) (&s2[0][0][0])[i] = 0.0f;
        if constexpr (BF) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t r[4], f[2];
            ldsm_x4(kb + C::at(lr, 2 * k + lu), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              qfrag(k, x, f);
              mma16<true>(s2[k & 1][x], r[0], r[1], r[2], r[3], f[0], f[1]);
            }
          }
        } else if constexpr (F8) {
#pragma unroll
          for (int k = 0; k < KS; k += 2) {  // a unit is 16 dims: one step
            uint32_t r[4], f[2];
            ldsm_x4(kb + C::at(lr, k + lu), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t a0 = e4m3x2_to_f16x2(r[2 * i]), a1 = e4m3x2_to_f16x2(r[2 * i + 1]),
                             a2 = e4m3x2_to_f16x2(r[2 * i] >> 16), a3 = e4m3x2_to_f16x2(r[2 * i + 1] >> 16);
#pragma unroll
              for (int x = 0; x < NT; ++x) {
                qfrag(k + i, x, f);
                mma16<false>(s2[0][x], a0, a1, a2, a3, f[0], f[1]);
              }
            }
          }
        } else {
          // a unit is 32 dims: two steps, two block scales; lanes c = 0, 1 hold the first block's dims
          uint32_t sc[2][D / 64];  // of tokens g and g + 8, two units' each
          const uint32_t ksel = c < 2 ? 0x6420 : 0x7531;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint8_t* from = kscale + (g + 8 * i) * C::SB;
            if constexpr (D == 64) {
              sc[i][0] = e4m3x2_to_f16x2(__byte_perm(*reinterpret_cast<const uint32_t*>(from), 0, ksel));
            } else {
#pragma unroll
              for (int w = 0; w < D / 128; ++w) {
                const uint2 x = *reinterpret_cast<const uint2*>(from + 8 * w);
                const uint32_t y = __byte_perm(x.x, x.y, ksel);
                sc[i][2 * w] = e4m3x2_to_f16x2(y);
                sc[i][2 * w + 1] = e4m3x2_to_f16x2(y >> 16);
              }
            }
          }
#pragma unroll
          for (int u = 0; u < D / 32; u += 2) {
            uint32_t r[4], f[2];
            ldsm_x4(kb + C::at(lr, u + lu), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t s0 = i ? dup16<1>(sc[0][u / 2]) : dup16<0>(sc[0][u / 2]),
                             s1 = i ? dup16<1>(sc[1][u / 2]) : dup16<0>(sc[1][u / 2]);
              uint32_t y[4], z[4];
              e2m1x8_to_f16x2(r[2 * i], y);
              e2m1x8_to_f16x2(r[2 * i + 1], z);
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const uint32_t a0 = hmul2(y[2 * p], s0), a1 = hmul2(z[2 * p], s1), a2 = hmul2(y[2 * p + 1], s0),
                               a3 = hmul2(z[2 * p + 1], s1);
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                  qfrag(2 * (u + i) + p, x, f);
                  mma16<false>(s2[0][x], a0, a1, a2, a3, f[0], f[1]);
                }
              }
            }
          }
        }
        // ---- scores: tokens g (+ 8: i >> 1), heads 2 c (+ 1: i & 1)
        float ks[2] = {1.0f, 1.0f};
        if constexpr (F8) {
          ks[0] = *reinterpret_cast<const float*>(kscale + 4 * g);
          ks[1] = *reinterpret_cast<const float*>(kscale + 4 * g + 32);
        }
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[t][x][i] = (C::SUMS == 2 ? s2[0][x][i] + s2[C::SUMS - 1][x][i] : s2[0][x][i]) *
                         (F8 ? qscale[x][i & 1] * ks[i >> 1] : qscale[x][i & 1]);
      }
      if (a.softcap > 0.0f) {
#pragma unroll
        for (int i = 0; i < TB * NT * 4; ++i) ka_cap((&s[0][0][0])[i], cap, per_cap);
      }
      if (seen != FULL) {
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((seen >> (16 * t + g + 8 * (i >> 1))) & 1u)) s[t][x][i] = -INFINITY;
      }

      // ---- values
      uint32_t vslot = kslot + C::SIDE;
      uint8_t* vslot_p = kslot_p + C::SIDE;
      if constexpr (!C::PAIR) {
        cp_async_wait_group<C::DEPTH - 2>();
        __syncwarp();
        issue();
        vslot = ring_at + get * C::STEP;
        get = get + 1 == C::DEPTH ? 0 : get + 1;
      }
      float vl[TB][2];  // log2 of the value scales of tokens g and g + 8
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        vl[t][0] = vl[t][1] = 0.0f;
        if constexpr (F8) {  // (a scale under 2^-126 counts as zero)
          const uint8_t* vscale = vslot_p + t * C::BLOCK + 16 * C::RB;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            vl[t][i] = lg2(*reinterpret_cast<const float*>(vscale + 4 * g + 32 * i));
            if (seen != FULL && !((seen >> (16 * t + g + 8 * i)) & 1u)) vl[t][i] = 0.0f;  // whatever is there
          }
        }
      }
      if constexpr (KIND == HQ_KV_NVFP4) {
        if (seen != FULL) {  // scales of tokens that are not seen: zero codes times them must be zero
          if (lane < 16 * TB && !((seen >> lane) & 1u)) {
            uint8_t* z = vslot_p + (lane / 16) * C::BLOCK + 16 * C::RB + (lane % 16) * C::SB;
#pragma unroll
            for (int w = 0; w < C::SB / 4; ++w) *reinterpret_cast<uint32_t*>(z + 4 * w) = 0u;
          }
          __syncwarp();
        }
      }
      // ---- weights: the running maximum of s, and of s - m + log2 of the value scale
      auto largest = [&](int x, int k) {
        float y = -INFINITY;
#pragma unroll
        for (int t = 0; t < TB; ++t) y = fmaxf(y, fmaxf(s[t][x][k], s[t][x][k + 2]));
        return y;
      };
      auto largest_scaled = [&](int x, int k) {
        float y = KA_NONE;
#pragma unroll
        for (int t = 0; t < TB; ++t)
          y = fmaxf(y, fmaxf(s[t][x][k] - m[x][k] + vl[t][0], s[t][x][k + 2] - m[x][k] + vl[t][1]));
        return y;
      };
      auto all_largest = [&](float y) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, i));
        return y;
      };
      bool over = false;
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          over |= largest(x, k) > m[x][k] + (KA_LAZY + C::LEAD);
          if constexpr (C::OD) over |= largest_scaled(x, k) > od[x][k] + (KA_LAZY + KA_LEAD);
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float y = all_largest(fmaxf(m[x][k], largest(x, k) - C::LEAD)), down = m[x][k] - y;
            float f = ex2(down);
            m[x][k] = y;
            l[x][k] *= f;
            if constexpr (C::OD) {  // (KA_NONE at least, so that differences stay numbers)
              const float z = all_largest(fmaxf(od[x][k] + down, largest_scaled(x, k) - KA_LEAD));
              f = ex2(od[x][k] - z + down);
              od[x][k] = z;
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) o[j][x][k] *= f, o[j][x][k + 2] *= f;
          }
      }
      uint32_t pb[TB][NT][2], pr[BF ? TB : 1][BF ? NT : 1][2];  // pr: the weights' second part
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float y = s[t][x][2 * i + k] - m[x][k], e = ex2(y);
              l[x][k] += e;
              w[k] = C::OD ? ex2(y + (vl[t][i] - od[C::OD ? x : 0][k])) : e;
            }
            // bf16's first part is of a weight 2^-8 smaller, and so below it: the rest is positive, between 2^-16 and
            // 2^-7 of the weight, and an infinite value stays that
            const uint32_t p = BF ? pack_bf16x2(w[0] * 0.99609375f, w[1] * 0.99609375f) : pack_f16x2(w[0], w[1]);
            pb[t][x][i] = turn8x8(p);
            if constexpr (BF) pr[t][x][i] = turn8x8(pack_bf16x2(w[0] - bf16_lo(p), w[1] - bf16_hi(p)));
          }
      // ---- o^T += V^T p^T
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const uint32_t vb = vslot + t * C::BLOCK;
        const uint8_t* vscale = vslot_p + t * C::BLOCK + 16 * C::RB;
        if constexpr (BF) {
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            uint32_t r[4];
            ldsm_x4_t(vb + C::at(lr, 2 * j + lu), r);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              mma16<true>(o[j][x], r[0], r[2], r[1], r[3], pb[t][x][0], pb[t][x][1]);
              mma16<true>(o[j][x], r[0], r[2], r[1], r[3], pr[t][x][0], pr[t][x][1]);
            }
          }
        } else if constexpr (F8) {
          // a unit is 16 dims: a lane gets dims 2 g, 2 g + 1 of two tokens; even dims are rows 0-7, odd ones 8-15
#pragma unroll
          for (int u = 0; u < KS; u += 2) {
            uint32_t r[4];
            ldsm_x4_t(vb + C::at(lr, u + lu), r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t y = __byte_perm(r[2 * i], 0, 0x3120), z = __byte_perm(r[2 * i + 1], 0, 0x3120);
              const uint32_t a0 = e4m3x2_to_f16x2(y), a1 = e4m3x2_to_f16x2(y >> 16), a2 = e4m3x2_to_f16x2(z),
                             a3 = e4m3x2_to_f16x2(z >> 16);
#pragma unroll
              for (int x = 0; x < NT; ++x) mma16<false>(o[u + i][x], a0, a1, a2, a3, pb[t][x][0], pb[t][x][1]);
            }
          }
        } else {
          // a unit is 32 dims: a lane gets dims 4 g .. 4 g + 3 of two tokens; two tiles of two of them each
          uint32_t sc[2][D / 32];  // of tokens 2 c, 2 c + 1, and 8 on
          const uint32_t vsel = g < 4 ? 0x6240 : 0x7351;  // the first or second block of each of two units
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint8_t* from = vscale + (8 * i + 2 * c) * C::SB;
            uint32_t x[D / 64], y[D / 64];
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
              if constexpr (D == 128) {
                if (w == 0) {
                  const uint4 v = *reinterpret_cast<const uint4*>(from);
                  x[0] = v.x, x[1] = v.y, y[0] = v.z, y[1] = v.w;
                }
              } else {
                x[w] = *reinterpret_cast<const uint32_t*>(from + 4 * w);
                y[w] = *reinterpret_cast<const uint32_t*>(from + C::SB + 4 * w);
              }
              const uint32_t z = __byte_perm(x[w], y[w], vsel);
              sc[i][2 * w] = e4m3x2_to_f16x2(z);
              sc[i][2 * w + 1] = e4m3x2_to_f16x2(z >> 16);
            }
          }
#pragma unroll
          for (int u = 0; u < D / 32; u += 2) {
            uint32_t r[4];
            ldsm_x4_t(vb + C::at(lr, u + lu), r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // the lane's word: dims 4 g .. 4 g + 3 of token 2 c, then of token 2 c + 1
              uint32_t y[4], z[4];
              e2m1x8_to_f16x2(r[2 * i], y);
              e2m1x8_to_f16x2(r[2 * i + 1], z);
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const uint32_t a0 = hmul2(__byte_perm(y[n], y[n + 2], 0x5410), sc[0][u + i]),
                               a1 = hmul2(__byte_perm(y[n], y[n + 2], 0x7632), sc[0][u + i]),
                               a2 = hmul2(__byte_perm(z[n], z[n + 2], 0x5410), sc[1][u + i]),
                               a3 = hmul2(__byte_perm(z[n], z[n + 2], 0x7632), sc[1][u + i]);
#pragma unroll
                for (int x = 0; x < NT; ++x)
                  mma16<false>(o[2 * (u + i) + n][x], a0, a1, a2, a3, pb[t][x][0], pb[t][x][1]);
              }
            }
          }
        }
      }
    }

    // ---- join the four warps, C::JOIN heads at a time, and write the pair's result or its part
    const bool whole = at.whole();
    float* part = slots + (2 * (int64_t)blockIdx.x + (at.u == lo ? 0 : 1)) * C::PART;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      if (8 * x >= rows) break;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) l[x][k] += __shfl_xor_sync(0xffffffffu, l[x][k], i);
        if (g == 0) {
          float* to = mls + (warp * 8 + 2 * c + k) * C::ML;
          to[0] = m[x][k];
          to[1] = l[x][k];
          if constexpr (C::OD) to[2] = od[C::OD ? x : 0][k];
        }
      }
#pragma unroll 1
      for (int j0 = 0; j0 < 8 && 8 * x + j0 < rows; j0 += C::JOIN) {
        if (C::JOIN == 8 || (2 * c >= j0 && 2 * c < j0 + C::JOIN)) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float* to = merge + (warp * C::JOIN + 2 * c + k - j0) * (D + C::PAD);
            if constexpr (BF) {
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                to[16 * j + g] = o[j][x][k];
                to[16 * j + 8 + g] = o[j][x][k + 2];
              }
            } else if constexpr (F8) {
#pragma unroll
              for (int j = 0; j < KS; ++j)
                *reinterpret_cast<float2*>(to + 16 * j + 2 * g) = make_float2(o[j][x][k], o[j][x][k + 2]);
            } else {
#pragma unroll
              for (int j = 0; j < KS; j += 2)
                *reinterpret_cast<float4*>(to + 16 * j + 4 * g) =
                    make_float4(o[j][x][k], o[j][x][k + 2], o[j + 1][x][k], o[j + 1][x][k + 2]);
            }
          }
        }
        __syncthreads();
        const int left = rows - 8 * x - j0, some = left < C::JOIN ? left : C::JOIN;
        for (int e = threadIdx.x; e < some * (D / 4); e += KA_THREADS) {
          const int n = e / (D / 4), r = j0 + n, d = 4 * (e % (D / 4));
          const float* ml = mls + r * C::ML;  // the first warp's
          constexpr int W = 8 * C::ML;
          float top = KA_NONE, otop = KA_NONE, sum = 0.0f;
#pragma unroll
          for (int w = 0; w < KA_WARPS; ++w) top = fmaxf(top, ml[w * W]);
          if constexpr (C::OD) {
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w) otop = fmaxf(otop, ml[w * W] - top + ml[w * W + C::ML - 1]);
          }
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < KA_WARPS; ++w) {
            float f = ex2(ml[w * W] - top);
            const float4 v = *reinterpret_cast<const float4*>(merge + (w * C::JOIN + n) * (D + C::PAD) + d);
            sum = fmaf(f, ml[w * W + 1], sum);
            if constexpr (C::OD) f = ex2(ml[w * W] - top + ml[w * W + C::ML - 1] - otop);
            y.x = fmaf(f, v.x, y.x), y.y = fmaf(f, v.y, y.y), y.z = fmaf(f, v.z, y.z), y.w = fmaf(f, v.w, y.w);
          }
          if (whole) {
            ka_store<C::OD>(a, q0 + 8 * x + r, D, d, y, otop, top, sum, vg);
          } else {
            __stcg(reinterpret_cast<float4*>(part + (8 * x + r) * D + d), y);
            if (d == 0) {
              __stcg(reinterpret_cast<float2*>(part + 8 * NT * D + 2 * (8 * x + r)), make_float2(top, sum));
              if constexpr (C::OD) __stcg(part + 8 * NT * (D + 2) + 8 * x + r, otop);
            }
          }
        }
        __syncthreads();
      }
    }
    if (whole) continue;

    ka_split<KIND, D, NT>(a, sh, at.seg0, at.seg0 + at.s.units, (int64_t)at.b * hrs + at.hr, slots, groups, counters,
                          last_one, q0, rows, vg, merge, mls);
  }
  cp_async_wait_all();
}

template <int KIND, int D, int NT>
cudaError_t launch_ka(const KvAttnArgs& a, int sms, int64_t tokens, uint8_t* workspace, cudaStream_t stream) {
  using C = KaCfg<KIND, D, NT>;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel has its shared memory (a bit each)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(allowed.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kv_attention_kernel<KIND, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or((uint64_t)1 << dev, std::memory_order_release);
  }
  // no more CTAs than the longest lengths make shares
  const int64_t per = (tokens + 16 * C::TB - 1) / (16 * C::TB);
  const int64_t pairs = a.B * a.kv.heads * ((a.group + KA_ROWS - 1) / KA_ROWS);
  const int64_t want = (pairs * (C::EXTRA + (per > 0 ? per : 1)) + C::EXTRA + 3) / (C::EXTRA + 4);
  const int64_t all = C::CTAS * sms < KA_MOST ? C::CTAS * sms : KA_MOST;
  return launch_kernel(kv_attention_kernel<KIND, D, NT>, dim3((unsigned)(want < all ? want : all)), dim3(KA_THREADS),
                       C::SMEM, stream, a, reinterpret_cast<float*>(workspace + KV_HEADER_BYTES),
                       reinterpret_cast<int*>(workspace + ka_group_counters_at(sms)),
                       reinterpret_cast<int*>(workspace + ka_counters_at(sms)));
}

template <int KIND>
cudaError_t launch_ka_dim(int dim, const KvAttnArgs& a, int sms, int64_t tokens, uint8_t* workspace,
                          cudaStream_t stream) {
  if (a.group <= 8)
    return dim == 64 ? launch_ka<KIND, 64, 1>(a, sms, tokens, workspace, stream)
                     : (dim == 128 ? launch_ka<KIND, 128, 1>(a, sms, tokens, workspace, stream)
                                   : launch_ka<KIND, 256, 1>(a, sms, tokens, workspace, stream));
  return dim == 64 ? launch_ka<KIND, 64, 2>(a, sms, tokens, workspace, stream)
                   : (dim == 128 ? launch_ka<KIND, 128, 2>(a, sms, tokens, workspace, stream)
                                 : launch_ka<KIND, 256, 2>(a, sms, tokens, workspace, stream));
}

#endif  // __CUDACC__

}  // namespace hq
