// Attention of one new token per sequence over a paged cache, split over the cache's length and joined.
//
//   s_j = scale (q . k_j);   m = max_j s_j;   l = sum_j exp(s_j - m);   o = (1 / l) sum_j exp(s_j - m) v_j
//
// in one pass over the cache: a part of the tokens keeps its own m, l and unnormalised o, and parts (m1, l1, o1),
// (m2, l2, o2) join to m = max(m1, m2), l = l1 e^(m1 - m) + l2 e^(m2 - m), o alike.  Everything is in powers of two
// (scores are multiplied by log2 e once), in fp32.
//
// What bounds it: the cache is read once and 4 G operations are done per key-value pair of elements for the G query
// heads that share a head, so up to G = 16 the kernel is bound by memory.  The work is laid out for that:
//  - The tokens of all (sequence, head) pairs form one list of 64-token units, cut into equal shares for a fixed number
//    of CTAs (two per SM), whatever the lengths are.  A pair inside one share is finished there; one that crosses
//    shares leaves fp32 partial results in the workspace, and the last CTA to arrive joins them in order.  The lengths
//    are read on the device, so a captured call follows them.
//  - The four warps of a CTA each stream every fourth 16-token block through a ring of their own in shared memory
//    (cp.async, 16 bytes a lane, one slot per block and side); no barrier but the warp's own between them until a
//    pair's parts are joined.  The ring runs ahead across pairs.
//  - Products run on mma.sync m16n8k16 with the G heads as the 16 rows.  A tcgen05 tile has at least 64 rows, of which
//    G would be used, and its operands would have to be decoded through shared memory; the legacy unit's rate is
//    several times what memory feeds here (see the table of measurements at the launch).
//  - 8- and 4-bit codes go from shared memory through ldmatrix to registers and become f16 there, exactly.  The
//    fragments' dims are permuted so that a lane's bytes are its own: the dot product does not care about the order of
//    dims if q follows it, and the output's order is undone when it is stored.
//  - e4m3: a token's key scale multiplies its score.  Its value scale v multiplies its weight, and a weight must fit
//    f16: the running maximum is taken over s_j + log2 v_j, so that the largest weight times its scale is about one
//    whatever the scales' range, while l sums exp2(s_j - m) in fp32 beside it.
//  - nvfp4: code * block scale is exact in f16 (2 + 4 significant bits); the global scales go to q's scale and o.
//  - Queries of the f16 kinds are scaled by a power of two per row, so that no bf16 query leaves f16's range.
//  - The running maximum only moves when a score exceeds it by 8 (powers of two): o is seldom rescaled, and weights up
//    to 2^8 fit the 16-bit types.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../hq_launch.h"
#include "../hq_ptx.cuh"
#include "hq_kv.h"
#include "hq_kv_codec.cuh"

namespace hq {

constexpr int KA_WARPS = 4;
constexpr int KA_THREADS = 32 * KA_WARPS;
constexpr int KA_ROWS = 16;        // query heads of one tile (the matrix instruction's rows)
constexpr float KA_LAZY = 8.0f;    // the running maximum lags by at most this (log2)

template <int KIND, int D>
struct KaCfg {
  static constexpr int RB = kv_row_bytes(KIND, D), SB = kv_scale_bytes(KIND, D);
  static constexpr int TOK = 16;                     // tokens of one ring slot
  static constexpr int SLOT = TOK * (RB + SB);       // bytes of one slot: codes, then scales, of one side
  static constexpr int PAD = KIND == HQ_KV_BF16 ? 8 : (KIND == HQ_KV_E4M3 ? 16 : 4);  // floats: no bank conflicts
  static constexpr int MERGE = KA_WARPS * 8 * (D + PAD) * 4;  // eight rows of every warp
  static constexpr bool QS = D == 256;               // q's fragments in shared memory instead of registers
  static constexpr int QBYTES = QS ? D / 16 * 512 : 0;
  static constexpr int FIXED = MERGE + QBYTES + 512;
  static constexpr int LIMIT = (228 * 1024) / 2 - 1024;  // shared memory of one of two CTAs on an SM
  static constexpr int FIT = (LIMIT - FIXED) / (KA_WARPS * (SLOT + 4));
  static constexpr int SLOTS = FIT < 2 ? 2 : (FIT > 12 ? 12 : FIT);
  static constexpr int SMEM = FIXED + KA_WARPS * SLOTS * (SLOT + 4);
  // 16-byte units: unit u of row r sits at u ^ swz(r), so that eight rows' equal units lie in different banks
  static constexpr int UPR = RB / 16;
  static constexpr int RPL = UPR >= 8 ? 1 : 8 / UPR;  // rows of a 128-byte line
  static constexpr int XM = (UPR >= 8 ? 8 : UPR) - 1;
  static __device__ __forceinline__ uint32_t at(int r, int u) { return (uint32_t)(r * RB + ((u ^ ((r / RPL) & XM)) << 4)); }
};

// Workspace of a call, for the host (sizes) and the device: the status, then two slots per CTA for the parts of split
// pairs, then a counter per (sequence, head, row tile).  A slot has room for any format's part, so that the counters,
// which have to be zero between calls, are at one place whatever the calls' shapes are.
constexpr size_t KA_SLOT_FLOATS = KA_ROWS * (256 + 2);  // o, then (m, l) of each row
constexpr size_t ka_counters_at(int ctas) {
  return KV_HEADER_BYTES + 2 * (size_t)ctas * KA_SLOT_FLOATS * sizeof(float);
}

#ifdef __CUDACC__

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
// the two values of one e2m1 byte
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t b) {
  uint32_t h;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(b));
  return h;
}
// nibble i of both halves of x -> f16x2 of value * 2^-14 (unpack_e2m1x8's placement of the bits)
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t x, int i) {
  const uint32_t y = x << (12 - 4 * i);
  return (y & 0x80008000u) | ((y >> 3) & 0x0E000E00u);
}

// One sequence's share of the list of units.
struct KaSeq {
  int n, j0, t0;     // tokens, the first that is seen, and that one's block
  int64_t units;     // per (head, row tile), at least one: an empty sequence's output is written too
};
__device__ __forceinline__ KaSeq ka_seq(const KvAttnArgs& a, int64_t b) {
  KaSeq s;
  int64_t n = a.lens[b];
  n = n < 0 ? 0 : (n > a.most ? a.most : n);
  const int64_t j0 = a.window > 0 && n > a.window ? n - a.window : 0;
  s.n = (int)n;
  s.j0 = (int)j0;
  s.t0 = (int)(j0 & ~(int64_t)(KV_BLOCK - 1));
  const int64_t u = (n - s.t0 + 63) >> 6;
  s.units = u > 0 ? u : 1;
  return s;
}

// A walk over a CTA's share, one (sequence, head, row tile) after another.
struct KaWalk {
  int64_t u, hi;   // position in the list, end of the share
  int64_t seg0;    // the pair's first unit in the list
  int64_t b;
  int hr;          // head * tiles + tile
  KaSeq s;
  __device__ __forceinline__ bool done() const { return u >= hi; }
  __device__ __forceinline__ int64_t stop() const { return seg0 + s.units < hi ? seg0 + s.units : hi; }
  // tokens of the share's part of the pair
  __device__ __forceinline__ int from() const { return s.t0 + (int)((u - seg0) << 6); }
  __device__ __forceinline__ int to() const {
    const int64_t t = s.t0 + ((stop() - seg0) << 6);
    return t < s.n ? (int)t : s.n;
  }
  __device__ __forceinline__ void next(const KvAttnArgs& a, int hrs) {
    u = stop();
    if (u >= hi) return;
    seg0 = u;
    if (++hr == hrs) {
      hr = 0;
      s = ka_seq(a, ++b);
    }
  }
};

template <int KIND, int D>
__global__ void __launch_bounds__(KA_THREADS, 2) kv_attention_kernel(const KvAttnArgs a, float* slots, int* counters) {
  using C = KaCfg<KIND, D>;
  constexpr bool BF = KIND == HQ_KV_BF16;
  constexpr int KS = D / 16, NT = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem);
  uint32_t* qsm = reinterpret_cast<uint32_t*>(smem + C::MERGE);
  int64_t* found = reinterpret_cast<int64_t*>(smem + C::MERGE + C::QBYTES);  // 3 words; then the warps' m and l
  float* mls = reinterpret_cast<float*>(smem + C::MERGE + C::QBYTES + 64);   // [warp][8 rows][2]
  uint32_t* scan = reinterpret_cast<uint32_t*>(smem + C::MERGE + C::QBYTES + 64);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + C::FIXED + warp * C::SLOTS * C::SLOT;
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + C::FIXED + KA_WARPS * C::SLOTS * C::SLOT) + warp * C::SLOTS;
  const uint32_t ring_at = smem_u32(ring);
  pdl_trigger();
  pdl_wait();

  // ---- this CTA's share of the units
  const int G = a.group, tiles = (G + KA_ROWS - 1) / KA_ROWS, H = a.kv.heads, hrs = H * tiles;
  const int part_rows = G < KA_ROWS ? G : KA_ROWS;
  const int64_t per = (a.B + KA_THREADS - 1) / KA_THREADS;
  const int64_t b0 = per * threadIdx.x < a.B ? per * threadIdx.x : a.B, b1 = b0 + per < a.B ? b0 + per : a.B;
  int64_t mine = 0;
  for (int64_t b = b0; b < b1; ++b) {
    mine += ka_seq(a, b).units;
    if (blockIdx.x == 0 && (a.lens[b] < 0 || a.lens[b] > a.most)) kv_report(a.status);
  }
  int64_t before = mine;  // inclusive sum over the warp's lanes, then exclusive over the CTA
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  if (lane == 31) reinterpret_cast<int64_t*>(scan)[warp] = before;
  before -= mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < KA_WARPS; ++w) {
    const int64_t y = reinterpret_cast<int64_t*>(scan)[w];
    if (w < warp) before += y;
    total += y;
  }
  total *= hrs;
  const int64_t W = total < gridDim.x ? total : gridDim.x;  // every CTA that works has a unit at least
  if (blockIdx.x >= W) return;
  const int64_t lo = total * blockIdx.x / W, hi = total * (blockIdx.x + 1) / W;
  if (lo >= before * hrs && lo < (before + mine) * hrs) {
    int64_t p = before;
    for (int64_t b = b0; b < b1; ++b) {
      const int64_t n = ka_seq(a, b).units;
      if (lo < (p + n) * hrs) {
        found[0] = b;
        found[1] = p;
        break;
      }
      p += n;
    }
  }
  __syncthreads();
  KaWalk at;
  at.u = lo;
  at.hi = hi;
  at.b = found[0];
  at.s = ka_seq(a, at.b);
  const int64_t in = lo - found[1] * hrs;
  at.hr = (int)(in / at.s.units);
  at.seg0 = lo - in % at.s.units;

  // ---- the ring's front: this warp's 16-token blocks of the share, keys and values alternating
  KaWalk ahead = at;
  int next_tok = ahead.from() + KV_BLOCK * warp, next_end = ahead.to();
  int page = 0, off = 0, have = 0, used = 0;  // lane i: the page and offset of the warp's i-th block from here
  bool more = true;
  int put = 0, side = 0;
  uint32_t word = 0;
  int64_t base = 0;
  auto issue = [&]() {
    if (side == 0) {
      while (more && next_tok >= next_end) {  // the share's next pair
        ahead.next(a, hrs);
        more = !ahead.done();
        if (more) next_tok = ahead.from() + KV_BLOCK * warp, next_end = ahead.to(), have = used = 0;
      }
      if (more) {
        if (used == have) {
          const int64_t tok = (int64_t)next_tok + KV_BLOCK * KA_WARPS * lane;
          page = -1;
          off = 0;
          if (tok < next_end) {
            const int col = (int)((uint32_t)tok / (uint32_t)a.kv.page_size);
            page = a.page_table[ahead.b * a.table_stride + col];
            off = (int)tok - col * a.kv.page_size;
            if (page < 0 || page >= a.kv.num_pages) {
              kv_report(a.status);
              page = -1;
            }
          }
          have = 32;
          used = 0;
        }
        const int p = __shfl_sync(0xffffffffu, page, used), o = __shfl_sync(0xffffffffu, off, used);
        ++used;
        const int first = ahead.s.j0 - next_tok, last = ahead.s.n - next_tok;  // tokens of the block that are seen
        word = 0xFFFFu;
        if (first > 0) word &= 0xFFFFu << first;
        if (last < 16) word &= 0xFFFFu >> (16 - last);
        if (p < 0) word = 0;
        base = ((int64_t)(p < 0 ? 0 : p) * H + ahead.hr / tiles) * a.kv.page_size + o;
        next_tok += KV_BLOCK * KA_WARPS;
      } else {
        word = 0;
      }
    }
    if (more) {
      const uint8_t* codes = (side ? a.kv.v : a.kv.k) + base * C::RB;
      uint8_t* slot = ring + put * C::SLOT;
#pragma unroll
      for (int i = 0; i < C::RB / 32; ++i) {
        const int e = lane + 32 * i, r = e / C::UPR, u = e % C::UPR;
        cp_async_16(slot + C::at(r, u), codes + e * 16, (word >> r) & 1u ? 16u : 0u);
      }
      if constexpr (C::SB > 0) {
        const uint8_t* scales = (side ? a.kv.v_scale : a.kv.k_scale) + base * C::SB;
        if (lane < C::SB) cp_async_16(slot + 16 * C::RB + 16 * lane, scales + 16 * lane, word ? 16u : 0u);
      }
      if (lane == 0) masks[put] = word;
    }
    cp_async_commit();
    put = put + 1 == C::SLOTS ? 0 : put + 1;
    side ^= 1;
  };
#pragma unroll 1
  for (int i = 0; i < C::SLOTS - 1; ++i) issue();
  int get = 0;

  float kg = 1.0f, vg = 1.0f;
  if constexpr (KIND == HQ_KV_NVFP4) {
    kg = *a.kv.k_global;
    vg = *a.kv.v_global * 128.0f;  // the values' f16 are 2^-7 of them
  }

  // ---- one pair after another
  for (; !at.done(); at.next(a, hrs)) {
    const int h = at.hr / tiles, r0 = (at.hr - h * tiles) * KA_ROWS, rows = G - r0 < KA_ROWS ? G - r0 : KA_ROWS;
    const uint16_t* qrow = a.q + ((at.b * H + h) * G + r0) * (int64_t)D;
    uint32_t qa[C::QS ? 1 : KS][4];
    float qscale[2];
    {
      // the lane's dims of rows g and g + 8: two pairs of each 16-dim step
      uint32_t raw[KS][4];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int d0 = BF ? 16 * s + 2 * c : (KIND == HQ_KV_E4M3 ? 16 * s + 4 * c : 32 * (s / 2) + 8 * c + 4 * (s & 1));
        const int d1 = BF ? d0 + 8 : d0 + 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool live = g + 8 * i < rows;
          const uint16_t* p = qrow + (int64_t)(g + 8 * i) * D;
          raw[s][i] = live ? *reinterpret_cast<const uint32_t*>(p + d0) : 0u;
          raw[s][2 + i] = live ? *reinterpret_cast<const uint32_t*>(p + d1) : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qscale[i] = a.scale;
        if constexpr (!BF) {
          float top = 0.0f;
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            top = fmaxf(top, fmaxf(fabsf(bf16_lo(raw[s][i])), fabsf(bf16_hi(raw[s][i]))));
            top = fmaxf(top, fmaxf(fabsf(bf16_lo(raw[s][2 + i])), fabsf(bf16_hi(raw[s][2 + i]))));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          int e = (int)(__float_as_uint(top) >> 23) - 127;  // the largest magnitude goes to [1, 2)
          e = top == 0.0f ? 0 : (e < -100 ? -100 : (e > 100 ? 100 : e));
          const float f = __uint_as_float((uint32_t)(127 - e) << 23);
          qscale[i] *= kg * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            raw[s][i] = pack_f16x2(bf16_lo(raw[s][i]) * f, bf16_hi(raw[s][i]) * f);
            raw[s][2 + i] = pack_f16x2(bf16_lo(raw[s][2 + i]) * f, bf16_hi(raw[s][2 + i]) * f);
          }
        }
        qscale[i] *= a.softcap > 0.0f ? 2.0f * 1.4426950408889634f / a.softcap : 1.4426950408889634f;
      }
      if constexpr (C::QS) {
        if (warp == 0) {
#pragma unroll
          for (int s = 0; s < KS; ++s)
            *reinterpret_cast<uint4*>(qsm + (s * 32 + lane) * 4) =
                make_uint4(raw[s][0], raw[s][1], raw[s][2], raw[s][3]);
        }
        __syncthreads();
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) qa[s][i] = raw[s][i];
      }
    }
    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    const int end = at.to();
#pragma unroll 1
    for (int tok = at.from() + KV_BLOCK * warp; tok < end; tok += KV_BLOCK * KA_WARPS) {
      // ---- keys
      cp_async_wait_group<C::SLOTS - 2>();
      __syncwarp();
      issue();
      const uint32_t kslot = ring_at + get * C::SLOT;
      const uint8_t* kscale = ring + get * C::SLOT + 16 * C::RB;
      const uint32_t seen = masks[get];
      get = get + 1 == C::SLOTS ? 0 : get + 1;
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] = 0.0f;
      const int lr = (lane & 7) + ((lane >> 4) << 3), lu = (lane >> 3) & 1;  // ldmatrix: tokens by two units
      auto qfrag = [&](int k, uint32_t (&f)[4]) {
        if constexpr (C::QS) {
          const uint4 v = *reinterpret_cast<const uint4*>(qsm + (k * 32 + lane) * 4);
          f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = qa[k][i];
        }
      };
      if constexpr (BF) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b[4], f[4];
          ldsm_x4(kslot + C::at(lr, 2 * k + lu), b[0], b[1], b[2], b[3]);
          qfrag(k, f);
          mma16<true>(s[0], f, b[0], b[1]);
          mma16<true>(s[1], f, b[2], b[3]);
        }
      } else if constexpr (KIND == HQ_KV_E4M3) {
#pragma unroll
        for (int k = 0; k < KS; k += 2) {  // a unit is 16 dims: one step
          uint32_t b[4], f[4];
          ldsm_x4(kslot + C::at(lr, k + lu), b[0], b[1], b[2], b[3]);
          qfrag(k, f);
          mma16<false>(s[0], f, e4m3x2_to_f16x2(b[0]), e4m3x2_to_f16x2(b[0] >> 16));
          mma16<false>(s[1], f, e4m3x2_to_f16x2(b[2]), e4m3x2_to_f16x2(b[2] >> 16));
          qfrag(k + 1, f);
          mma16<false>(s[0], f, e4m3x2_to_f16x2(b[1]), e4m3x2_to_f16x2(b[1] >> 16));
          mma16<false>(s[1], f, e4m3x2_to_f16x2(b[3]), e4m3x2_to_f16x2(b[3] >> 16));
        }
      } else {
        // a unit is 32 dims: two steps, two block scales; lanes c = 0, 1 hold the first block's dims
        uint32_t f16s[2][D / 32];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(kscale + (g + 8 * t) * C::SB + 4 * w);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t y = c < 2 ? __byte_perm(x, 0, i ? 0x22 : 0x00) : __byte_perm(x, 0, i ? 0x33 : 0x11);
              f16s[t][2 * w + i] = e4m3x2_to_f16x2(y);
            }
          }
#pragma unroll
        for (int u = 0; u < D / 32; u += 2) {
          uint32_t b[4], f[4];
          ldsm_x4(kslot + C::at(lr, u + lu), b[0], b[1], b[2], b[3]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              qfrag(2 * (u + i) + p, f);
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const uint32_t x = b[2 * t + i] >> (16 * p);
                mma16<false>(s[t], f, hmul2(e2m1x2_to_f16x2(x & 0xFFu), f16s[t][u + i]),
                             hmul2(e2m1x2_to_f16x2((x >> 8) & 0xFFu), f16s[t][u + i]));
              }
            }
          }
        }
      }

      // ---- scores: rows g and g + 8 (i >> 1), tokens 8 t + 2 c + (i & 1)
      float vl[2][2];  // e4m3: log2 of the value scales
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float2 ks = make_float2(1.0f, 1.0f);
        if constexpr (KIND == HQ_KV_E4M3) ks = *reinterpret_cast<const float2*>(kscale + 4 * (8 * t + 2 * c));
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] *= qscale[i >> 1] * ((i & 1) ? ks.y : ks.x);
      }
      if (a.softcap > 0.0f) {  // cap * tanh(x) = cap * (1 - 2 / (1 + e^2x)); the scores hold 2 x log2 e
        const float cap = a.softcap * 1.4426950408889634f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[t][i] = cap * (1.0f - __fdividef(2.0f, 1.0f + ex2(fminf(s[t][i], 80.0f))));
      }
      if (seen != 0xFFFFu) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((seen >> (8 * t + 2 * c + (i & 1))) & 1u)) s[t][i] = -INFINITY;
      }

      // ---- values
      cp_async_wait_group<C::SLOTS - 2>();
      __syncwarp();
      issue();
      const uint32_t vslot = ring_at + get * C::SLOT;
      uint8_t* vscale = ring + get * C::SLOT + 16 * C::RB;
      get = get + 1 == C::SLOTS ? 0 : get + 1;
      if constexpr (KIND == HQ_KV_E4M3) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float2 v = *reinterpret_cast<const float2*>(vscale + 4 * (8 * t + 2 * c));
          vl[t][0] = lg2(fmaxf(v.x, 7.8886091e-31f));  // 2^-100: a smaller scale's values are all but zero
          vl[t][1] = lg2(fmaxf(v.y, 7.8886091e-31f));
        }
      }
      if constexpr (KIND == HQ_KV_NVFP4) {
        if (seen != 0xFFFFu) {  // scales of tokens that are not seen: zero codes times them must be zero
          if (lane < 16 && !((seen >> lane) & 1u)) {
#pragma unroll
            for (int w = 0; w < C::SB / 4; ++w) *reinterpret_cast<uint32_t*>(vscale + lane * C::SB + 4 * w) = 0u;
          }
          __syncwarp();
        }
      }
      // running maximum: of s, or of s + log2 of the value scale
      float f[2] = {1.0f, 1.0f};
      bool moved = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float y = KIND == HQ_KV_E4M3 ? s[t][2 * i + k] + vl[t][k] : s[t][2 * i + k];
            x = fmaxf(x, y);
          }
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        if (x > m[i] + KA_LAZY || (m[i] == -INFINITY && x > m[i])) {
          f[i] = ex2(m[i] - x);
          m[i] = x;
          moved = true;
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] *= f[i >> 1];
        l[0] *= f[0];
        l[1] *= f[1];
      }
      uint32_t p[4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mm = m[i] == -INFINITY ? 0.0f : m[i];
          float w[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float e = ex2(s[t][2 * i + k] - mm);
            l[i] += e;
            w[k] = KIND == HQ_KV_E4M3 ? ex2(s[t][2 * i + k] + vl[t][k] - mm) : e;
          }
          p[2 * t + i] = BF ? pack_bf16x2(w[0], w[1]) : pack_f16x2(w[0], w[1]);
        }
      const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vu = lane >> 4;
      if constexpr (BF) {
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t b[4];
          ldsm4t(b, vslot + C::at(vr, j + vu));
          mma16<true>(o[j], p, b[0], b[1]);
          mma16<true>(o[j + 1], p, b[2], b[3]);
        }
      } else if constexpr (KIND == HQ_KV_E4M3) {
        // a unit is 16 dims: a lane gets dims 2g, 2g + 1 of tokens 2c, 2c + 1; tiles of the even and of the odd dims
#pragma unroll
        for (int u = 0; u < D / 16; u += 2) {
          uint32_t b[4];
          ldsm4t(b, vslot + C::at(vr, u + vu));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = __byte_perm(b[2 * i], 0, 0x3120), y = __byte_perm(b[2 * i + 1], 0, 0x3120);
            mma16<false>(o[2 * (u + i)], p, e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y));
            mma16<false>(o[2 * (u + i) + 1], p, e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y >> 16));
          }
        }
      } else {
        // a unit is 32 dims: a lane gets dims 4g .. 4g + 3 of tokens 2c, 2c + 1; four tiles, dims 4n + i each
        uint32_t vs[2][D / 32];  // f16x2 of the two tokens' scales * 2^7
        const uint32_t sel = g < 4 ? 0x0040u : 0x0051u;  // the first or second block's byte of each token
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(vscale + (8 * t + 2 * c) * C::SB + 4 * w);
            const uint32_t y = *reinterpret_cast<const uint32_t*>(vscale + (8 * t + 2 * c + 1) * C::SB + 4 * w);
            vs[t][2 * w] = hmul2(e4m3x2_to_f16x2(__byte_perm(x, y, sel)), 0x58005800u);
            vs[t][2 * w + 1] = hmul2(e4m3x2_to_f16x2(__byte_perm(x, y, sel + 0x0022u)), 0x58005800u);
          }
#pragma unroll
        for (int u = 0; u < D / 32; u += 2) {
          uint32_t b[4];
          ldsm4t(b, vslot + C::at(vr, u + vu));
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n)
              mma16<false>(o[4 * (u + i) + n], p, hmul2(e2m1_pair(b[2 * i], n), vs[0][u + i]),
                           hmul2(e2m1_pair(b[2 * i + 1], n), vs[1][u + i]));
        }
      }
    }

    // ---- join the four warps, eight rows at a time, and write the pair's result or its part
    const bool whole = at.u == at.seg0 && at.stop() == at.seg0 + at.s.units;
    const int64_t pair = at.b * hrs + at.hr;
    const int64_t my_slot = 2 * (int64_t)blockIdx.x + (at.u == lo ? 0 : 1);
    float* part = slots + my_slot * KA_SLOT_FLOATS;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (8 * i >= rows) break;
      if (c == 0) {
        mls[(warp * 8 + g) * 2] = m[i];
        mls[(warp * 8 + g) * 2 + 1] = l[i];
      }
      float* to = merge + (warp * 8 + g) * (D + C::PAD);
      if constexpr (BF) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          *reinterpret_cast<float2*>(to + 8 * j + 2 * c) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
      } else if constexpr (KIND == HQ_KV_E4M3) {
#pragma unroll
        for (int j = 0; j < NT; j += 2)
          *reinterpret_cast<float4*>(to + 8 * j + 4 * c) =
              make_float4(o[j][2 * i], o[j + 1][2 * i], o[j][2 * i + 1], o[j + 1][2 * i + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < NT; j += 4)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float4*>(to + 8 * j + 8 * c + 4 * k) =
                make_float4(o[j][2 * i + k], o[j + 1][2 * i + k], o[j + 2][2 * i + k], o[j + 3][2 * i + k]);
      }
      __syncthreads();
      const int some = rows - 8 * i < 8 ? rows - 8 * i : 8;
      for (int e = threadIdx.x; e < some * (D / 4); e += KA_THREADS) {
        const int r = e / (D / 4), d = 4 * (e % (D / 4));
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < KA_WARPS; ++w) top = fmaxf(top, mls[(w * 8 + r) * 2]);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < KA_WARPS; ++w) {
          const float mw = mls[(w * 8 + r) * 2], x = mw == -INFINITY ? 0.0f : ex2(mw - top);
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * 8 + r) * (D + C::PAD) + d);
          sum = fmaf(x, mls[(w * 8 + r) * 2 + 1], sum);
          y.x = fmaf(x, v.x, y.x), y.y = fmaf(x, v.y, y.y), y.z = fmaf(x, v.z, y.z), y.w = fmaf(x, v.w, y.w);
        }
        const int row = 8 * i + r;
        if (whole) {
          const float inv = sum > 0.0f ? vg / sum : 0.0f;
          const int64_t q = (at.b * H + h) * G + r0 + row;
          *reinterpret_cast<uint2*>(a.out + q * D + d) =
              make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
          if (d == 0 && a.lse) a.lse[q] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
        } else {
          __stcg(reinterpret_cast<float4*>(part + row * D + d), y);
          if (d == 0) __stcg(reinterpret_cast<float2*>(part + part_rows * D + 2 * row), make_float2(top, sum));
        }
      }
      __syncthreads();
    }
    if (whole) continue;

    // ---- split pair: the last CTA to arrive joins the parts, first to last
    const int64_t c0 = ((at.seg0 + 1) * W - 1) / total, c1 = ((at.seg0 + at.s.units) * W - 1) / total;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) found[2] = atomicAdd(counters + pair, 1) == (int)(c1 - c0);
    __syncthreads();
    if (!found[2]) continue;
    __threadfence();
    const int parts = (int)(c1 - c0) + 1;
    const int64_t s0 = 2 * c0 + (total * c0 / W == at.seg0 ? 0 : 1);  // the others' first pair is this one
    for (int e = threadIdx.x; e < rows * (D / 4); e += KA_THREADS) {
      const int row = e / (D / 4), d = 4 * (e % (D / 4));
      float top = -INFINITY, sum = 0.0f;
      for (int k = 0; k < parts; ++k) {
        const float* x = slots + (k ? 2 * (c0 + k) : s0) * KA_SLOT_FLOATS;
        top = fmaxf(top, __ldcg(x + part_rows * D + 2 * row));
      }
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k = 0; k < parts; ++k) {
        const float* x = slots + (k ? 2 * (c0 + k) : s0) * KA_SLOT_FLOATS;
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(x + part_rows * D + 2 * row));
        const float4 v = __ldcg(reinterpret_cast<const float4*>(x + row * D + d));
        const float w = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
        sum = fmaf(w, ml.y, sum);
        y.x = fmaf(w, v.x, y.x), y.y = fmaf(w, v.y, y.y), y.z = fmaf(w, v.z, y.z), y.w = fmaf(w, v.w, y.w);
      }
      const float inv = sum > 0.0f ? vg / sum : 0.0f;
      const int64_t q = (at.b * H + h) * G + r0 + row;
      *reinterpret_cast<uint2*>(a.out + q * D + d) =
          make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
      if (d == 0 && a.lse) a.lse[q] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
    if (threadIdx.x == 0) counters[pair] = 0;
  }
  cp_async_wait_all();
}

template <int KIND, int D>
cudaError_t launch_ka(const KvAttnArgs& a, int ctas, float* slots, int* counters, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<KIND, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             KaCfg<KIND, D>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv_attention_kernel<KIND, D>, dim3((unsigned)ctas), dim3(KA_THREADS), KaCfg<KIND, D>::SMEM,
                       stream, a, slots, counters);
}

#endif  // __CUDACC__

}  // namespace hq
