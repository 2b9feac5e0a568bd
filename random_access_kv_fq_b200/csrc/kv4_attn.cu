// Attention over the 4-bit paged cache.
//
// The rows (query token, query head) that share a kv head are taken 8 or 16 at a time; such a row
// block with the tokens that it may see is an item.  All items' tokens form one line that is cut
// into equal ranges, a range to a warp: long contexts are split over many warps, short ones
// share a warp, whatever the lengths.  A warp streams its units (16 tokens, keys and values
// together: one bulk copy each) through a ring of its own in shared memory and waits for no other
// warp.  Per unit, with codes c, steps s and zeros z:
//   scores   S^T = sum_g s_g (C_g Q_g^T) + Z qsum^T    (16 tokens x 8 rows per product)
//            4-bit codes are fp16 numbers as they stand: 0x000c is c 2^-24, a subnormal, and
//            0x00c0 is 16 c 2^-24, so unpacking is one AND per pair; the 16 is taken out of q.
//            Steps multiply in fp32 after the products, zeros enter as one more product with the
//            groups' sums of q (in two fp16 parts), so scores carry no 16-bit rounding: q itself
//            is scaled to fp16 by a power of two per row.
//   softmax  base 2, against a running maximum that moves only when a score passes it by 8 (kLow, kLag).
//   values   O^T += V^T P^T with V = fp16(c s + z), which the product takes 16 bits of, off by at most
//            2^-11.  P is fp16 too, for fp16 outputs in two parts, so that V's is the one rounding beside
//            the output's own of 2^-11; beside bf16's of 2^-8 one part does.
// A warp's unfinished ranges are joined in shared memory, a block's by the last block to leave a part
// of the item.
//
// mma.sync and not tcgen05: the products of decode are 8 to 16 rows wide, operands come out of
// registers, and the tensor pipe has three quarters of its time left at the HBM bound.
//
// Measured: 64 sequences of 1 to 8,191 tokens, 32 query and 8 kv heads of 128, bf16, 342 MB: 71 us, 4,800
// GB/s, 0.73 of a copy's; issue slots 61 % busy, of the rest ~10,000 cycles are the way to the first unit
// and ~12,000 the joins.  16 sequences of 32K tokens, 4 kv heads of 64, fp16, 168 MB: 49 us, 3,420 GB/s, 0.52;
// neither memory (39 % busy) nor issue (62 %, 231 warp instructions a unit of 1,280 bytes) binds it but the
// results that a warp waits for: of 7.5 cycles an instruction 1.7 are a fixed latency, 0.8 the matrix pipe, 0.5
// barriers.  24 sequences of up to 12K tokens behind a window of 4,096, up to 42 rows a kv head: 41 us; each 16
// rows unpack the units again.
#include <atomic>
#include <cfloat>

#include "fq_internal.h"
#include "kv4_attn.cuh"

namespace fq {
namespace kv4 {
namespace {

__device__ unsigned int g_kv4_wait_timeouts = 0;  // blocks whose bounded waits gave up

constexpr int kChunk = 2;        // units of a stage of a warp's ring: one wait for 32 tokens
constexpr int kItemUnits = 3;    // an item's fixed cost, in units (its queries and its end)

// warps of a block, by the registers that their accumulators leave
template <int NT, int D>
constexpr int kWarpsOf = NT == 1 ? 16 : D == 64 ? 12 : 8;
// stages of a ring: ~10 KB a warp, 160 KB of an SM's copies in flight or in use
template <int D>
constexpr int kStagesOf = D == 64 ? 4 : 2;

template <int NT, int D>
struct Part {
  float4 o[NT * D / 16 * 32];  // accumulators in fragment order
  float m[8 * NT], l[8 * NT];
};

// The cost of each of its row blocks: the units of the most tokens that one may see, and what is fixed.
struct CostedSeq : Seq {
  int cost;
};
template <int NB>
__device__ __forceinline__ CostedSeq load_costed(const AttnArgs& a, int b, int r) {
  CostedSeq s;
  static_cast<Seq&>(s) = load_seq<NB>(a, b, r);
  const int most = a.window > 0 ? min(s.n, a.window + NB + kUnit) : s.n;
  s.cost = (most + kUnit - 1) / kUnit + kItemUnits;
  return s;
}

// What a warp says of a part that it leaves.
struct PartHeader {
  int state;               // 0: none, 1: the item goes on, 3: its last part
  int q0, rows, head, rb;  // where its rows are
  int cost;                // of the whole item,
  int64_t start;           // and where it begins on the line
};

// Blocks that have left a part of the item begun in block c, at the workspace's start: the call's tag
// and the number.  The workspace needs no preparation: a word without the call's tag counts as none.
// The last block leaves the tag with 0, for a replay of the same call.
constexpr int kCountBits = 8;
static_assert(kCtas < 1 << kCountBits, "");
constexpr size_t kCounters = (kCtas * sizeof(uint64_t) + 15) / 16 * 16;

// ------------------------------------------------------------------------------ items

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same, and the k = 8 form, with nothing to add to
__device__ __forceinline__ void mma16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma8_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
      "{%7,%7,%7,%7};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// ------------------------------------------------------------------------------ one warp's state

template <typename T, int D, int G, int NT>
struct Warp {
  static constexpr int NG = D / G, KB = D / 32, MT = D / 16, UB = kUnit * D + 128 * NG;
  static constexpr bool kTwoParts = __is_same(T, __half);
  uint32_t q[NT][KB][4];     // query fragments; odd ones over 16
  uint32_t qz[NT];           // sums of q over the groups, in two parts
  float kappa[NT][2];        // score scale of rows 2 t, 2 t + 1 of the tile
  int hi[NT][2], lo[NT][2];  // tokens that the rows see: [lo, hi)
  float o[NT][MT][4], m[NT][2], l[NT][2];  // m: kLow below the scores' maximum

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.f;
      m[nt][0] = m[nt][1] = -FLT_MAX;
      l[nt][0] = l[nt][1] = 0.f;
    }
  }

  // Queries of row block rb of (sequence, kv head): row r is query token r / R, head r % R.  Asked
  // for before the first unit is, used while it is on its way.
  __device__ __forceinline__ void fetch_queries(const AttnArgs& a, const Seq& s, int head, int rb, uint32_t r, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t row = rb * 8 * NT + nt * 8 + g;
      const bool in = row < (uint32_t)s.rows;
      const uint32_t tok = in ? row / r : 0, hh = in ? row - tok * r : 0;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(s.q0 + tok) * a.q_tok +
                            (int64_t)(head * r + hh) * a.q_head + 8 * t;
      const bool wide = in && reinterpret_cast<uintptr_t>(src) % 16 == 0;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (wide) {
          w = __ldg(reinterpret_cast<const uint4*>(src + 32 * kb));
        } else if (in) {
          const uint16_t* p = src + 32 * kb;
          w.x = __ldg(p) | (uint32_t)__ldg(p + 1) << 16;
          w.y = __ldg(p + 2) | (uint32_t)__ldg(p + 3) << 16;
          w.z = __ldg(p + 4) | (uint32_t)__ldg(p + 5) << 16;
          w.w = __ldg(p + 6) | (uint32_t)__ldg(p + 7) << 16;
        }
        q[nt][kb][0] = w.x;
        q[nt][kb][1] = w.y;
        q[nt][kb][2] = w.z;
        q[nt][kb][3] = w.w;
      }
    }
  }

  __device__ __forceinline__ void convert_queries(const AttnArgs& a, const Seq& s, int rb, uint32_t r, int lane) {
    const int t = lane & 3;
    const int past = s.n - s.m + 1;
    float kap[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[KB][8];
      float top = 0.f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[kb][e] = q_float<T>((uint16_t)(q[nt][kb][e / 2] >> (16 * (e & 1))));
          top = fmaxf(top, fabsf(x[kb][e]));
        }
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      // the row times 2^-e lies within +-2^8: exact in fp16 but for what is 2^-28 of the largest
      int e = top > 0.f ? (int)(__float_as_uint(top) >> 23) - 127 - 7 : 0;
      e = max(e, -126);
      const float down = __uint_as_float((uint32_t)(127 - max(e, -126)) << 23);
      kap[nt] = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
      float sum[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) sum[i] = 0.f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        __half y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = __float2half_rn(x[kb][i] * down);
          sum[32 * kb / G] += __half2float(y[i]);
        }
        const __half2 over = __floats2half2_rn(0.0625f, 0.0625f);
        q[nt][kb][0] = u32(__halves2half2(y[0], y[4]));
        q[nt][kb][1] = u32(__hmul2(__halves2half2(y[1], y[5]), over));
        q[nt][kb][2] = u32(__halves2half2(y[2], y[6]));
        q[nt][kb][3] = u32(__hmul2(__halves2half2(y[3], y[7]), over));
      }
      __half part[2][NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        sum[i] += __shfl_xor_sync(~0u, sum[i], 1);
        sum[i] += __shfl_xor_sync(~0u, sum[i], 2);
        part[0][i] = __float2half_rn(sum[i]);
        part[1][i] = __float2half_rn(sum[i] - __half2float(part[0][i]));
      }
      // zero words of a token: (z0 z1) (z2 z3) for NG = 4, (z0 z1) for 2, (s0 z0) for 1
      const __half none = __ushort_as_half(0);
      uint32_t w = 0;
      if constexpr (NG == 4) {
        const int p = t >> 1;
        w = t & 1 ? u32(__halves2half2(part[p][2], part[p][3])) : u32(__halves2half2(part[p][0], part[p][1]));
      } else if constexpr (NG == 2) {
        if (t < 2) w = u32(__halves2half2(part[t][0], part[t][1]));
      } else {
        if (t < 2) w = u32(__halves2half2(none, part[t][0]));
      }
      qz[nt] = w;
    }
    // the accumulators' columns are rows 2 t, 2 t + 1: their scale sits in lanes 8 t, 8 t + 4
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        kappa[nt][c] = __shfl_sync(~0u, kap[nt], 8 * t + 4 * c);
        const uint32_t row = min(rb * 8 * NT + nt * 8 + 2 * t + c, s.rows - 1);
        hi[nt][c] = past + (int)(row / r);
        lo[nt][c] = a.window > 0 ? hi[nt][c] - a.window : 0;
      }
  }

  // Where in a unit this lane reads: its key codes, key steps, value codes, value steps.
  struct Place {
    uint32_t k, ks, v, vs;
  };
  static __device__ __forceinline__ Place place(uint32_t u, int lane) {
    const int g = lane >> 2, t = lane & 3;
    Place p{u + lane * (D / 8), u + off_ks(D) + g * 4 * NG,
            u + off_v(D) + t * (D / 2) + (D == 128 ? ((2 * g) ^ ((t & 2) << 2)) * 4 : 4 * g),
            u + off_vs(D, G) + t * 4 * NG + (g * (D / 8) / G) * 4};
    // kept in registers: made again for every unit they would cost a twelfth of its instructions
    asm volatile("" : "+r"(p.k), "+r"(p.ks), "+r"(p.v), "+r"(p.vs));
    return p;
  }

  // One unit at `u`, whose first token is at position pos0.  MASK: some row may not see all of it;
  // [first, end) is what any row sees.
  template <bool MASK>
  __device__ __forceinline__ void unit(const Place& u, int pos0, int first, int end, int lane) {
    uint32_t k0[KB], k1[KB];
    lds<D / 8>(u.k, k0);
    lds<D / 8>(u.k + 4 * D, k1);
    // steps and zeros of token rows g and g + 8: 2 NG numbers each, of which lane t feeds the product
    // with the zeros of groups 2 (t & 1) and 2 (t & 1) + 1
    uint32_t s0[NG], s1[NG];
    lds<4 * NG>(u.ks, s0);
    lds<4 * NG>(u.ks + 32 * NG, s1);
    const uint32_t z0 = NG == 4 ? (lane & 1 ? s0[NG - 1] : s0[NG / 2]) : s0[NG - 1];
    const uint32_t z1 = NG == 4 ? (lane & 1 ? s1[NG - 1] : s1[NG / 2]) : s1[NG - 1];
    float x[NT][4];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      float acc[NT][4];
#pragma unroll
      for (int kb = gr * G / 32; kb < (gr + 1) * G / 32; ++kb) {
        const uint32_t lowm = 0x000F000Fu, highm = 0x00F000F0u;
        const uint32_t a = k0[kb] >> 8, b = k1[kb] >> 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (kb == gr * G / 32)
            mma16_first(acc[nt], k0[kb] & lowm, k1[kb] & lowm, k0[kb] & highm, k1[kb] & highm, q[nt][kb][0], q[nt][kb][1]);
          else
            mma16(acc[nt], k0[kb] & lowm, k1[kb] & lowm, k0[kb] & highm, k1[kb] & highm, q[nt][kb][0], q[nt][kb][1]);
          mma16(acc[nt], a & lowm, b & lowm, a & highm, b & highm, q[nt][kb][2], q[nt][kb][3]);
        }
      }
      const __half2 p0 = h2(s0[gr / 2]), p1 = h2(s1[gr / 2]);
      const float f0 = gr % 2 ? __high2float(p0) : __low2float(p0);
      const float f1 = gr % 2 ? __high2float(p1) : __low2float(p1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[nt][i] = gr == 0 ? acc[nt][i] * (i < 2 ? f0 : f1) : fmaf(acc[nt][i], i < 2 ? f0 : f1, x[nt][i]);
    }
    // x: scores over kappa; y: base-2 logarithms of the weights
    float y[NT][4];
    float high = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float acc[4];
      mma8_first(acc, z0, z1, qz[nt]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[nt][i] = fmaf(x[nt][i], 16777216.f, acc[i]);
        y[nt][i] = fmaf(x[nt][i], kappa[nt][i & 1], -m[nt][i & 1]);
        if (MASK) {
          // rows of the product are tokens (g >> 1) + 4 (g & 1), and 8 further
          const int pos = pos0 + (lane >> 3) + (lane & 4) + 4 * (i & 2);
          if (pos >= hi[nt][i & 1] || pos < lo[nt][i & 1]) y[nt][i] = -INFINITY;
        }
        high = fmaxf(high, y[nt][i]);
      }
    }
    if (__any_sync(~0u, high > kLow + kLag)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float xa = y[nt][c] == -INFINITY ? -INFINITY : x[nt][c] * kappa[nt][c];
          const float xb = y[nt][c + 2] == -INFINITY ? -INFINITY : x[nt][c + 2] * kappa[nt][c];
          float top = fmaxf(xa, xb);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
          top = fmaxf(top - kLow, m[nt][c]);
          const float f = ex2(m[nt][c] - top);
          y[nt][c] = xa - top;
          y[nt][c + 2] = xb - top;
          m[nt][c] = top;
          l[nt][c] *= f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            o[nt][mt][c] *= f;
            o[nt][mt][c + 2] *= f;
          }
        }
    }
    uint32_t p[NT][2], pl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[nt][i] = ex2(y[nt][i]);
      l[nt][0] += x[nt][0] + x[nt][2];
      l[nt][1] += x[nt][1] + x[nt][3];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2 v = __floats2half2_rn(x[nt][2 * i], x[nt][2 * i + 1]);
        p[nt][i] = transpose8(u32(v));
        if (kTwoParts) {
          const float2 f = __half22float2(v);
          pl[nt][i] = transpose8(u32(__floats2half2_rn(x[nt][2 * i] - f.x, x[nt][2 * i + 1] - f.y)));
        }
      }
    }
    // values: this lane's tokens are t + 4 i, its coordinates g D/8 .. + D/8 (all of one group)
    uint32_t w[4][D / 64], sz[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lds<D / 16>(u.v + 4 * i * (D / 2), w[i]);
      lds<4>(u.vs + 16 * i * NG, &sz[i]);
      if (MASK) {
        const int pos = pos0 + (lane & 3) + 4 * i;
        if (pos < first || pos >= end) sz[i] = 0;  // a token that nobody sees: its value becomes 0
      }
    }
    const __half2 st[2] = {h2(__byte_perm(sz[0], sz[1], 0x5410)), h2(__byte_perm(sz[2], sz[3], 0x5410))};
    const __half2 ze[2] = {h2(__byte_perm(sz[0], sz[1], 0x7632)), h2(__byte_perm(sz[2], sz[3], 0x7632))};
    const __half2 bias = h2(0xE400E400u), sixteenth = h2(0x2C002C00u), bias16 = h2(0xD400D400u);
#pragma unroll
    for (int wi = 0; wi < D / 64; ++wi)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t v[2][4];  // [token pair][coordinate]
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t y = __byte_perm(w[2 * j][wi], w[2 * j + 1][wi], half ? 0x7632 : 0x5410);
          const uint32_t y8 = y >> 8;
          // 0x6400 + c is 1024 + c, 0x6400 + 16 c is 1024 + 16 c: back to c without rounding
          const __half2 c0 = __hadd2(h2(and_or<0x000F000Fu>(y, 0x64006400u)), bias);
          const __half2 c1 = __hfma2(h2(and_or<0x00F000F0u>(y, 0x64006400u)), sixteenth, bias16);
          const __half2 c2 = __hadd2(h2(and_or<0x000F000Fu>(y8, 0x64006400u)), bias);
          const __half2 c3 = __hfma2(h2(and_or<0x00F000F0u>(y8, 0x64006400u)), sixteenth, bias16);
          v[j][0] = u32(__hfma2(c0, st[j], ze[j]));
          v[j][1] = u32(__hfma2(c1, st[j], ze[j]));
          v[j][2] = u32(__hfma2(c2, st[j], ze[j]));
          v[j][3] = u32(__hfma2(c3, st[j], ze[j]));
        }
        const int mt = wi * 4 + half * 2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16(o[nt][mt], v[0][0], v[0][1], v[1][0], v[1][1], p[nt][0], p[nt][1]);
          mma16(o[nt][mt + 1], v[0][2], v[0][3], v[1][2], v[1][3], p[nt][0], p[nt][1]);
          if (kTwoParts) {
            mma16(o[nt][mt], v[0][0], v[0][1], v[1][0], v[1][1], pl[nt][0], pl[nt][1]);
            mma16(o[nt][mt + 1], v[0][2], v[0][3], v[1][2], v[1][3], pl[nt][0], pl[nt][1]);
          }
        }
      }
  }

  __device__ __forceinline__ void finish_sums() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][c] += __shfl_xor_sync(~0u, l[nt][c], d);
  }

  __device__ __forceinline__ void write_part(Part<NT, D>* part, int lane) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        part->o[(nt * MT + mt) * 32 + lane] = make_float4(o[nt][mt][0], o[nt][mt][1], o[nt][mt][2], o[nt][mt][3]);
      if (lane < 4) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          part->m[nt * 8 + 2 * lane + c] = m[nt][c];
          part->l[nt * 8 + 2 * lane + c] = l[nt][c];
        }
      }
    }
  }

  __device__ __forceinline__ void write_out(const AttnArgs& a, const Seq& s, int head, int rb, uint32_t r, int lane) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t row = rb * 8 * NT + nt * 8 + 2 * t + c;
        if (row >= (uint32_t)s.rows) continue;
        const uint32_t tok = row / r;
        const float inv = l[nt][c] > 0.f ? 1.0f / l[nt][c] : 0.f;
        T* dst = static_cast<T*>(a.out) + ((int64_t)(s.q0 + tok) * a.hq + head * r + row - tok * r) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < MT / 4; ++i) {
          uint4 v;
          v.x = pack_out<T>(o[nt][4 * i][c] * inv, o[nt][4 * i][c + 2] * inv);
          v.y = pack_out<T>(o[nt][4 * i + 1][c] * inv, o[nt][4 * i + 1][c + 2] * inv);
          v.z = pack_out<T>(o[nt][4 * i + 2][c] * inv, o[nt][4 * i + 2][c + 2] * inv);
          v.w = pack_out<T>(o[nt][4 * i + 3][c] * inv, o[nt][4 * i + 3][c + 2] * inv);
          reinterpret_cast<uint4*>(dst)[i] = v;
        }
      }
  }
};

// N fragment words of an item's rows nt * 8 + 2 t and + 1: two coordinates each, all of one row adjacent.
// A warp's piece of a join.
template <int NT, int D>
struct Words {
  static constexpr int N = D / 32, kPieces = NT * D / 16 / N;
  float4 o[N];
  float2 l;

  static __device__ __forceinline__ int row(int piece, int lane) { return piece * N / (D / 16) * 8 + 2 * (lane & 3); }

  // Sums the parts at(0) .. at(n - 1) of this block.  The maxima come first, so that the numbers wait
  // only for their own weights.
  template <typename At>
  __device__ __forceinline__ float2 join(int piece, int lane, int n, const At& at) {
    const int r0 = row(piece, lane);
    float2 top = make_float2(-FLT_MAX, -FLT_MAX);
#pragma unroll 4
    for (int c = 0; c < n; ++c) {
      const float2 m = *reinterpret_cast<const float2*>(&at(c)->m[r0]);
      top.x = fmaxf(top.x, m.x);
      top.y = fmaxf(top.y, m.y);
    }
    clear();
#pragma unroll 2
    for (int c = 0; c < n; ++c) {
      const Part<NT, D>* p = at(c);
      const float2 m = *reinterpret_cast<const float2*>(&p->m[r0]);
      add(p->o + piece * N * 32 + lane, *reinterpret_cast<const float2*>(&p->l[r0]), ex2(m.x - top.x), ex2(m.y - top.y));
    }
    return top;
  }

  // The same for parts of other blocks: everything of a part is asked for at once, against a running
  // maximum.
  template <typename At>
  __device__ __forceinline__ float2 join_far(int piece, int lane, int n, const At& at) {
    const int r0 = row(piece, lane);
    float2 top = make_float2(-FLT_MAX, -FLT_MAX);
    clear();
#pragma unroll 2
    for (int c = 0; c < n; ++c) {
      const Part<NT, D>* p = at(c);
      const float2 m = __ldcg(reinterpret_cast<const float2*>(&p->m[r0])), s = __ldcg(reinterpret_cast<const float2*>(&p->l[r0]));
      float4 y[N];
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = __ldcg(p->o + (piece * N + i) * 32 + lane);
      const float2 up = make_float2(fmaxf(top.x, m.x), fmaxf(top.y, m.y));
      const float f0 = ex2(top.x - up.x), f1 = ex2(top.y - up.y);
      l.x *= f0;
      l.y *= f1;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = make_float4(o[i].x * f0, o[i].y * f1, o[i].z * f0, o[i].w * f1);
      top = up;
      add<1>(y, s, ex2(m.x - up.x), ex2(m.y - up.y));
    }
    return top;
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    l = make_float2(0.f, 0.f);
  }

  template <int STEP = 32>
  __device__ __forceinline__ void add(const float4* y, float2 s, float w0, float w1) {
    l.x = fmaf(s.x, w0, l.x);
    l.y = fmaf(s.y, w1, l.y);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 v = y[i * STEP];
      o[i] = make_float4(fmaf(v.x, w0, o[i].x), fmaf(v.y, w1, o[i].y), fmaf(v.z, w0, o[i].z), fmaf(v.w, w1, o[i].w));
    }
  }

  __device__ __forceinline__ void leave(Part<NT, D>* dst, int piece, int lane, float2 top) const {
#pragma unroll
    for (int i = 0; i < N; ++i) dst->o[(piece * N + i) * 32 + lane] = o[i];
    if (piece * N % (D / 16) == 0 && lane < 4) {
      const int r0 = row(piece, lane);
      *reinterpret_cast<float2*>(&dst->m[r0]) = top;
      *reinterpret_cast<float2*>(&dst->l[r0]) = l;
    }
  }

  template <typename T>
  __device__ __forceinline__ void write(const AttnArgs& a, const PartHeader& h, int piece, int lane) const {
    const uint32_t r = a.hq / a.hkv;
    const int word = piece * N % (D / 16);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t at = h.rb * 8 * NT + row(piece, lane) + c;
      if (at >= (uint32_t)h.rows) continue;
      const uint32_t tok = at / r;
      const float sum = c ? l.y : l.x, inv = sum > 0.f ? 1.0f / sum : 0.f;
      T* dst = static_cast<T*>(a.out) + ((int64_t)(h.q0 + tok) * a.hq + h.head * r + at - tok * r) * D + (lane >> 2) * (D / 8) + 2 * word;
      uint32_t v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = pack_out<T>((c ? o[i].y : o[i].x) * inv, (c ? o[i].w : o[i].z) * inv);
      if constexpr (N == 4) *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
      else *reinterpret_cast<uint2*>(dst) = make_uint2(v[0], v[1]);
    }
  }
};

template <typename T, int D, int G, int NT>
__global__ void __launch_bounds__(32 * kWarpsOf<NT, D>, 1) attn_kernel(AttnArgs a, int page_shift, int own_blocks, uint64_t tag) {
  using W_ = Warp<T, D, G, NT>;
  using P = Part<NT, D>;
  constexpr int W = kWarpsOf<NT, D>, NB = 8 * NT, UB = W_::UB, kStages = kStagesOf<D>;
  constexpr size_t kRing = kStages * kChunk * UB, kSlot = kRing > sizeof(P) ? kRing : sizeof(P);
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* rings = smem;                                          // [W][kSlot]
  P* heads = reinterpret_cast<P*>(smem + W * kSlot);              // [W]
  __shared__ uint64_t bars[W][kStages];
  __shared__ PartHeader hdr[W][2];
  __shared__ int64_t scan[W];
  __shared__ int64_t range_end[W];
  __shared__ int4 closing[2];
  __shared__ uint32_t groups[2 * W];  // an item's first slot, its parts << 8, whether others join it << 16
  __shared__ int gave_up;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = a.hq / a.hkv;

  if (tid == 0) gave_up = 0;
  if (lane < kStages) ptx::mbar_init(&bars[warp][lane], kChunk);
  if (lane < 2) hdr[warp][lane].state = 0;
  ptx::fence_mbar_init();
  __syncwarp();  // a warp uses its own barriers only

  W_ st;
  uint8_t* ring = rings + warp * kSlot;
  const typename W_::Place place = W_::place(ptx::smem_u32(ring), lane);
  uint32_t count = 0;  // chunks so far: the ring's stage and its barrier's parity
  bool ok = true;
  // What is left of this warp's range of the line, where it begins in its first item, and that item:
  // number `block` of the row blocks of (sequence b, kv head).
  int64_t left = 0, span = 1;
  int from = 0, b = 0, head = 0, block = 0;
  CostedSeq s = {};
  if (own_blocks > 0) {
    // short contexts: a block to an item, shared out to its warps
    block = blockIdx.x % own_blocks;
    head = blockIdx.x / own_blocks % a.hkv;
    b = blockIdx.x / own_blocks / a.hkv;
    s = load_costed<NB>(a, b, r);
    if (block < s.blocks) {
      s.cost = kItemUnits + W;  // a W-th of the units each, whatever their number
      from = warp == 0 ? 0 : kItemUnits + warp;
      left = warp == 0 ? kItemUnits + 1 : 1;
    }
  } else {
    // The line of all items' costs: running sums over groups of `per` sequences, in shared memory where
    // the rings will be, in which each warp looks up its range's start.
    const int per = (a.B + 32 * W - 1) / (32 * W), b0 = tid * per, b1 = min(a.B, b0 + per);
    int64_t* sums = reinterpret_cast<int64_t*>(smem);
    int64_t x = 0;
    for (int i = b0; i < b1; ++i) {
      s = load_costed<NB>(a, i, r);
      x += (int64_t)(a.hkv * s.blocks) * s.cost;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    // the sums of the warps, by every warp
    int64_t all = lane < W ? scan[lane] : 0;
#pragma unroll
    for (int d = 1; d < W; d <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, all, d);
      if (lane >= d) all += y;
    }
    const int64_t total = __shfl_sync(~0u, all, W - 1), before = __shfl_sync(~0u, all, warp > 0 ? warp - 1 : 0);
    sums[tid] = x + (warp > 0 ? before : 0);
    ptx::fence_proxy_async_smem();  // copies will write where the sums are
    __syncthreads();
    span = max((int64_t)(total * (1.0 / (kCtas * W))) + 1, (int64_t)kChunk);
    const int64_t x0 = (int64_t)(blockIdx.x * W + warp) * span;
    left = min(span, total - x0);
    range_end[warp] = x0 + left;
    if (left > 0) {
      // the first group whose sum is past x0, 32 places at a time
      int lo = 0, n = 32 * W;
      while (n > 1) {
        const int step = (n + 31) / 32, i = min(lo + (lane + 1) * step, lo + n) - 1;
        lo += (__ffs(__ballot_sync(~0u, sums[i] > x0)) - 1) * step;
        n = step;
      }
      int64_t in_seq = x0 - (lo > 0 ? sums[lo - 1] : 0);
      for (b = lo * per;; ++b) {
        s = load_costed<NB>(a, b, r);
        const int64_t cost = (int64_t)(a.hkv * s.blocks) * s.cost;
        if (in_seq < cost) break;
        in_seq -= cost;
      }
      const int item = item_of(in_seq, s.cost);  // which of the sequence's items
      from = (int)(in_seq - (int64_t)item * s.cost);
      head = s.blocks == 1 ? item : item / s.blocks;
      block = item - head * s.blocks;
    }
    __syncthreads();  // the sums are read
  }
  // after a wait that gave up the rest of the range counts as empty, so that each item gets its parts
  while (left > 0) {
    const int to = (int)min((int64_t)s.cost, from + left);
    left -= to - from;
    // Row blocks from both ends in turn: later ones see more tokens, two neighbours about as many as
    // any two.
    const int rb = block & 1 ? s.blocks - 1 - (block >> 1) : block >> 1;
    // tokens that any row of the block sees, in units; the part of them in this range
    const int past = s.n - s.m + 1;
    const uint32_t row0 = rb * NB, row1 = min(rb * NB + NB, s.rows) - 1;
    const int tok0 = row0 / (uint32_t)r, tok1 = row1 / (uint32_t)r;
    const int end = max(0, past + tok1);
    const int first = a.window > 0 ? max(0, past + tok0 - a.window) : 0;
    const int base_u = first / kUnit, units = end > first ? (end + kUnit - 1) / kUnit - base_u : 0;
    const int full = s.cost - kItemUnits;
    const float ratio = (float)units / (float)full;
    const auto share = [&](int x) {
      x -= kItemUnits;
      return x <= 0 ? 0 : x >= full ? units : units == full ? x : min(units, (int)(x * ratio));
    };
    const int u0 = share(from), u1 = share(to);

    st.reset();
    if (u0 < u1 && ok) {
      // Copies run up to kStages chunks ahead.  Lane i issues units i, i + 32, ... of the range, from
      // the table entry that it holds; a unit behind the range or on a page outside the pool only
      // counts as arrived, and `gone` has its bit.
      const int32_t* table = a.tables + (int64_t)b * a.max_blocks;
      const int n_units = u1 - u0, chunks = (n_units + kChunk - 1) / kChunk;
      const int shift = page_shift - 4;
      auto entry = [&](int i) { return i < n_units ? __ldg(table + ((base_u + u0 + i) >> shift)) : -1; };
      const uint8_t* src = nullptr;
      int id_next = entry(lane);
      uint32_t gone = 0, gone_next = 0;  // of the 32 units that are being used, and being issued
      auto issue = [&](int j) {
        const int who = (j * kChunk) & 31;
        if (who == 0) {
          const int id = id_next, i = j * kChunk + lane;
          id_next = entry(i + 32);
          src = nullptr;
          if (id >= 0 && id < a.n_blocks)
            src = a.cache + ((((int64_t)id * a.hkv + head) << shift) + ((base_u + u0 + i) & ((1 << shift) - 1))) * UB;
          gone_next = __ballot_sync(~0u, src == nullptr);
        }
        if ((unsigned)(lane - who) < kChunk) {
          const uint32_t at_stage = (count + j) % kStages;
          uint64_t* bar = &bars[warp][at_stage];
          if (src) {
            ptx::mbar_arrive_expect_tx(bar, UB);
            ptx::bulk_load(ring + (at_stage * kChunk + lane - who) * UB, src, UB, bar);
          } else {
            ptx::mbar_arrive(bar);
          }
        }
      };
      st.fetch_queries(a, s, head, rb, r, lane);
      for (int j = 0; j < chunks && j < kStages; ++j) issue(j);
      st.convert_queries(a, s, rb, r, lane);
      // a few units go through the code that checks each token: less code to fetch
      const bool clean = chunks > 2;
      const int all_end = past + tok0, all_first = a.window > 0 ? past + tok1 - a.window : 0;
      // a wait that gives up ends the loop once the copies in flight had the time of another wait each to land
      int landing = chunks;
      for (int j = 0; j < landing; ++j) {
        if (((j * kChunk) & 31) == 0) gone = gone_next;
        const uint32_t at_stage = (count + j) % kStages, parity = (count + j) / kStages & 1;
        if (!__all_sync(~0u, ptx::mbar_try(&bars[warp][at_stage], parity)) &&
            !__all_sync(~0u, ptx::mbar_wait(&bars[warp][at_stage], parity)) && ok) {
          ok = false;
          landing = min(chunks, j + kStages);
          --j;  // this one too
          continue;
        }
        if (ok) {
          const uint32_t skip = gone >> ((j * kChunk) & 31) & ((1u << kChunk) - 1);
          const int pos0 = (base_u + u0 + j * kChunk) * kUnit;
          typename W_::Place u = place;
          const uint32_t off = at_stage * kChunk * UB;
          u.k += off;
          u.ks += off;
          u.v += off;
          u.vs += off;
          if (clean && pos0 >= all_first && pos0 + kChunk * kUnit <= all_end && skip == 0) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
              st.template unit<false>(typename W_::Place{u.k + i * UB, u.ks + i * UB, u.v + i * UB, u.vs + i * UB}, 0, 0, 0, lane);
          } else {
#pragma unroll 1
            for (int i = 0; i < kChunk; ++i) {
              if (!((skip >> i) & 1)) st.template unit<true>(u, pos0 + i * kUnit, first, end, lane);
              u.k += UB;
              u.ks += UB;
              u.v += UB;
              u.vs += UB;
            }
          }
          __syncwarp();
          if (j + kStages < chunks) issue(j + kStages);
        }
      }
      count += chunks;
      st.finish_sums();
    }
    if (from == 0 && to == s.cost) {
      st.write_out(a, s, head, rb, r, lane);
    } else {
      // an item begun before this range leaves its part beside the ring, one that goes on in it
      const int k = from > 0 ? 0 : 1;
      st.write_part(k == 0 ? heads + warp : reinterpret_cast<P*>(ring), lane);
      if (lane == 0) {
        const int64_t start = own_blocks > 0 ? 0 : range_end[warp] - left - to;
        hdr[warp][k] = PartHeader{to == s.cost ? 3 : 1, s.q0, s.rows, head, rb, s.cost, start};
      }
    }
    // the next item of the line
    from = 0;
    if (left > 0 && ++block == s.blocks) {
      block = 0;
      if (++head == a.hkv) {
        head = 0;
        do s = load_costed<NB>(a, ++b, r); while (s.blocks == 0);
      }
    }
  }
  if (!ok) gave_up = 1;
  __syncthreads();
  if (tid == 0 && gave_up) atomicAdd(&g_kv4_wait_timeouts, 1u);

  // Join the parts of each item; what begins before or ends behind the block goes to the workspace.
  // Slot 2 w + k holds part k of warp w.  An item's parts are a part 1 (or, if begun before the
  // block, warp 0's part 0) and the next warps' parts 0 up to its last one.
  uint64_t* counters = static_cast<uint64_t*>(a.workspace);
  P* out_part = reinterpret_cast<P*>(static_cast<uint8_t*>(a.workspace) + kCounters);  // [kCtas][2]
  const int state = lane < 2 * W ? hdr[lane >> 1][lane & 1].state : 0;
  const uint32_t has = __ballot_sync(~0u, state != 0), ends = __ballot_sync(~0u, state == 3) & 0x55555555u;
  const bool begins = state != 0 && ((lane & 1) || lane == 0);
  const uint32_t starts = __ballot_sync(~0u, begins);
  bool leaves = false;
  int c0 = 0, blocks = 0;  // of the item that a lane of warp 0 has a part of to leave
  uint64_t seen = 0;
  if (warp == 0) {
    // the next warps' parts 0, up to one that ends the item or is missing
    const int next = (lane | 1) + 1;
    const uint32_t stop = next < 32 ? (ends | (~has & 0x55555555u)) >> next : 0;
    const int steps = stop ? (__ffs(stop) - 1) / 2 : (2 * W - next) / 2;
    const bool last = state == 3 || (next < 32 && ((ends >> next) >> (2 * steps)) & 1);
    const int parts = state == 3 ? 1 : 1 + steps + last;
    leaves = begins && own_blocks == 0 && !((lane & 1) && last);
    if (begins) groups[__popc(starts & ((1u << lane) - 1))] = lane | parts << 8 | (leaves ? 1u << 16 : 0u);
    if (lane < 2) closing[lane].y = 0;
    if (leaves) {
      const PartHeader& h = hdr[lane >> 1][lane & 1];
      c0 = (int)(h.start / (span * W));
      blocks = (int)((h.start + h.cost - 1) / (span * W)) - c0 + 1;
      seen = *reinterpret_cast<volatile uint64_t*>(counters + c0);
    }
  }
  __syncthreads();
  using J = Words<NT, D>;
  J join;
  for (int i = warp; i < __popc(starts) * J::kPieces; i += W) {
    const uint32_t gr = groups[i / J::kPieces];
    const int piece = i % J::kPieces, k = gr & 1, w0 = (gr & 0xff) >> 1;
    const P* first = k ? reinterpret_cast<const P*>(rings + w0 * kSlot) : heads + w0;
    const float2 top = join.join(piece, lane, gr >> 8 & 0xff, [&](int c) { return c == 0 ? first : heads + w0 + c; });
    if (gr >> 16) join.leave(out_part + blockIdx.x * 2 + k, piece, lane, top);
    else join.template write<T>(a, hdr[w0][k], piece, lane);
  }
  if (own_blocks > 0) return;

  // The last block to leave a part of an item joins them.
  __threadfence();
  __syncthreads();
  if (leaves) {
    unsigned long long* at = reinterpret_cast<unsigned long long*>(counters + c0);
    while (seen >> kCountBits != tag >> kCountBits) {
      const uint64_t was = atomicCAS(at, seen, tag);
      seen = was == seen ? tag : was;  // only to the tag does anyone else change it
    }
    if ((int)(atomicAdd(at, 1ull) - tag) + 1 == blocks) {
      *at = tag;
      __threadfence();
      closing[lane & 1] = make_int4(c0, blocks, lane, 0);
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int4 cl = closing[k];
    if (cl.y == 0) continue;
    // warps take slices of the parts and a piece each, then a few of them join the slices
    constexpr int S = W / J::kPieces;
    static_assert(S >= 2, "");
    const int piece = warp % J::kPieces, slice = warp / J::kPieces, slices = min(S, cl.y);
    if (slice < slices) {
      const int n = (cl.y - slice + S - 1) / S;
      const float2 top = join.join_far(piece, lane, n, [&](int i) {
        const int c = slice + i * S;
        return out_part + (cl.x + c) * 2 + (c == 0);
      });
      join.leave(heads + slice, piece, lane, top);
    }
    __syncthreads();
    if (slice == 0) {
      join.join(piece, lane, slices, [&](int c) { return heads + c; });
      join.template write<T>(a, hdr[cl.z >> 1][cl.z & 1], piece, lane);
    }
    __syncthreads();
  }
}

// Row blocks of a sequence where every item gets a block of its own, or 0.  That is so where the items
// fit the SMs at once and a warp's share is at most 8 units: no parts leave a block, and the line, the joins
// between blocks and the workspace fall away (one sequence of 517 tokens, 8 kv heads: 9.2 us against 13.3; 8
// of up to 1,024, 12 kv heads: 9.4 against 11.9; with long contexts ranges over all SMs win).
int own_blocks(int B, int hkv, int max_q, int r, int64_t capacity, int nt, int warps) {
  const int64_t blocks = ((int64_t)max_q * r + 8 * nt - 1) / (8 * nt);
  return (int64_t)B * hkv * blocks <= kCtas && capacity <= 8 * kUnit * warps ? (int)blocks : 0;
}

// Of every call another, and none that memory holds by chance: an odd multiple of the call's number.
uint64_t next_tag() {
  static std::atomic<uint64_t> calls{0};
  return (calls.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9E3779B97F4A7C15ull << kCountBits;
}

template <typename T, int D, int G, int NT>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  using P = Part<NT, D>;
  constexpr int W = kWarpsOf<NT, D>;
  constexpr size_t ring = kStagesOf<D> * kChunk * unit_bytes(D, G), slot = ring > sizeof(P) ? ring : sizeof(P);
  constexpr size_t bytes = W * (slot + sizeof(P));
  static_assert(bytes + 2048 <= 227 * 1024, "shared memory of a block, static included");
  static_assert(slot % 16 == 0 && sizeof(P) % 16 == 0, "parts are read in 16 bytes");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may have this much shared memory
  if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(attn_kernel<T, D, G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  int shift = 4;
  while ((1 << shift) < a.page) ++shift;
  const int r = a.hq / a.hkv, own = own_blocks(a.B, a.hkv, a.max_q, r, (int64_t)a.max_blocks * a.page, NT, W);
  attn_kernel<T, D, G, NT><<<own ? (unsigned)(a.B * a.hkv * own) : kCtas, 32 * W, bytes, st>>>(a, shift, own, next_tag());
  return cudaGetLastError();
}

template <typename T, int D, int G>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t st) {
  // 8 rows a block while a kv head has no more: half the products and registers of 16
  return (int64_t)a.max_q * (a.hq / a.hkv) <= 8 ? launch<T, D, G, 1>(a, st) : launch<T, D, G, 2>(a, st);
}

template <typename T>
cudaError_t launch_shape(const AttnArgs& a, cudaStream_t st) {
  if (a.d == 64) return a.group == 32 ? launch_rows<T, 64, 32>(a, st) : launch_rows<T, 64, 64>(a, st);
  if (a.group == 32) return launch_rows<T, 128, 32>(a, st);
  return a.group == 64 ? launch_rows<T, 128, 64>(a, st) : launch_rows<T, 128, 128>(a, st);
}

}  // namespace

size_t attn_workspace_bytes(int B, int hq, int hkv, int d, int max_q, int64_t capacity) {
  const int64_t rows = (int64_t)max_q * (hq / hkv);
  if (rows > kFewRows) return attn_rows_workspace_bytes(d);
  const int nt = rows <= 8 ? 1 : 2, warps = nt == 1 ? kWarpsOf<1, 64> : d == 64 ? kWarpsOf<2, 64> : kWarpsOf<2, 128>;
  if (own_blocks(B, hkv, max_q, hq / hkv, capacity, nt, warps)) return 0;
  return kCounters + 2 * kCtas * (d == 64 ? sizeof(Part<2, 64>) : sizeof(Part<2, 128>));
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st) {
  if ((int64_t)a.max_q * (a.hq / a.hkv) > kFewRows) return launch_attn_rows(a, st);
  return a.type == FQ_F16 ? launch_shape<__half>(a, st) : launch_shape<__nv_bfloat16>(a, st);
}

cudaError_t wait_timeouts_kv4(bool clear, unsigned* count) {
  return read_wait_counter(g_kv4_wait_timeouts, clear, count);
}

}  // namespace kv4
}  // namespace fq
