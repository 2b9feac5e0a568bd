// Attention over the 4-bit paged cache for many rows of a kv head (chunks of a prompt, drafted
// tokens): 128 rows (query token, query head) at a time on the fifth-generation tensor cores.
//
// One block per SM, its warps in roles that meet in mbarriers, over tiles of 128 tokens:
//   loaders  one warp copies the units' keys, one their values (bulk copies), into a ring each, 64 tokens
//            a stage;
//   unpack   4 warps turn keys and 4 turn values into fp16 operands in shared memory, two tiles deep;
//   products one thread issues S = Q K^T into one of two buffers of tensor memory, the next tile's under
//            this tile's softmax, one issues O += P V with P in tensor memory;
//   softmax  8 warps, two threads to a row: S out of tensor memory, weights P back into its place.
// q is scaled to fp16 by a power of two per row.  Values are V = fp16(c s + z), at most half a step (2^-11) off.
// For bf16 outputs, whose own rounding is 2^-8, keys and weights are fp16 numbers likewise.  For fp16
// outputs neither may add to it:  s is split into its leading 7 bits and the rest, so that s_hi c and
// s_lo c are fp16 numbers exactly, and
//   S = Q (s_hi C)^T + Q (s_lo C)^T + qsum Z^T,
// the last one a 16-wide product of the groups' sums of q (in two parts) with the zeros; weights are in
// two parts, O = P_hi V + P_lo V.  The softmax runs to base 2 against a maximum that moves only when a
// score passes it by 8 (kLow, kLag); moving it rescales O in tensor memory.
//
// A product of 128 x 128 x 16 takes 64 cycles (of 128 x 64 x 16: 50 to 57, so tiles are 128 tokens), so
// a tile of d = 128 needs 1,024 cycles of the tensor pipe for bf16 and 2,112 for fp16.  Of a call's time a tile
// takes about 3,300 and 3,800 (3 chunks of up to 1,024 queries over up to 8K tokens, 32 query and 8 kv heads: 206
// to 220 us, from run to run, and 249; 600 to 640 and 530 TFLOP/s): 9,200 warp instructions of unpacking and
// softmax a tile (fp16), which keep the issue slots 68 % and the tensor pipe 50 % busy.  A change of item takes
// 10,000 to 15,000 cycles, so ranges are cut by tokens and parts of one tile are not made.
// Measured and not kept: 8 unpacking warps more, 16 softmax warps, softmax groups on
// alternate tiles, asynchronous copies by the unpacking warps.
#include <atomic>
#include <cfloat>

#include "fq_internal.h"
#include "kv4_attn.cuh"

namespace fq {
namespace kv4 {
namespace {

// What a block leaves for the kernel that joins: [kCtas][2] parts, part 0 of an item begun before the
// block's range, part 1 of an item begun in it that goes on behind it.
struct PartHeader {
  int state;             // 0: none, 1: goes on, 3: the item's last part
  int q0, rows, head, rb;  // where its rows are
};
static_assert(2 * kCtas * sizeof(PartHeader) % 16 == 0, "parts behind the headers are read in 16 bytes");

// The block that holds the last part of the item begun in block c0.  All lanes of a warp call it.
__device__ __forceinline__ int last_part(const PartHeader* hdr, int c0) {
  const int lane = threadIdx.x & 31;
  for (int c = c0 + 1; c < kCtas; c += 32) {
    const uint32_t last = __ballot_sync(~0u, c + lane < kCtas && hdr[(c + lane) * 2].state == 3);
    if (last) return c + __ffs(last) - 1;
  }
  return kCtas - 1;
}

__device__ unsigned int g_kv4_rows_wait_timeouts = 0;  // blocks whose bounded waits gave up

constexpr int kRows = 128;      // rows of a block's item
constexpr int kTile = 128;      // tokens of a tile
constexpr int kTileUnits = kTile / kUnit;
constexpr int kItemTiles = 6;   // an item's fixed cost, in tiles: its queries, its end, the first tile's way
constexpr int kSoftmaxWarps = 8;  // warps w and w + 4 share 32 rows, 64 columns each
constexpr int kKeyWarps = 4, kValueWarps = 4, kUnpackWarps = kKeyWarps + kValueWarps;
constexpr int kWarps = kSoftmaxWarps + kUnpackWarps + 4;  // two for the products, two loaders
// units of a stage of a ring: a loader's step takes ~700 cycles and ~85 more for each copy
constexpr int kChunkUnits = 4;
// registers a thread: 96 at launch, 20 warps x 96 >= 8 x 128 + 12 x 72; nothing is spilled
constexpr int kSoftmaxRegs = 128, kOtherRegs = 72;

constexpr int kItemBytes = 96;  // of a warp's Items

template <int D>
struct RowsPart {
  float4 o[D / 4][kRows];  // 32 rows' pieces lie together
  float m[kRows], l[kRows];
};

template <int D, int G, bool EXACT>
struct Shape {
  static constexpr int NG = D / G, UB = unit_bytes(D, G), KB = D / 32, NA = D / 64;
  static constexpr int kOp = kTile * D * 2;          // bytes of one fp16 operand of a tile
  static constexpr int kZ = EXACT ? kTile * 32 : 0;  // zeros: 16 numbers a token
  static constexpr int kK = (EXACT ? 2 : 1) * kOp + kZ, kBuf = kK + kOp;
  static constexpr int kChunks = kTileUnits / kChunkUnits, kCodes = kUnit * D / 2, kScales = 64 * NG;
  // a stage of the keys' ring: codes of its units, then steps and zeros; of the values': codes, the keys'
  // steps and zeros, which lie between, and their own of a unit in one piece
  static constexpr int kKeys = kChunkUnits * (kCodes + kScales), kValue = kCodes + 2 * kScales, kValues = kChunkUnits * kValue;
  static constexpr int kRing = D == 64 ? 8 : EXACT ? 2 : 4;  // what shared memory leaves
  static constexpr size_t kControl = 1024;
  static constexpr size_t kItems = kControl + 2 * kBuf + kRing * (kKeys + kValues);
  static constexpr size_t kSmem = kItems + kWarps * kItemBytes;
  // tensor memory columns: [2] S, of which P takes the place (hi, then lo), O, Q and its sums
  static constexpr uint32_t S = 0, O = 256, Q = 384, QZ = 448;
};

struct Control {
  uint64_t ring_full[2][8], ring_empty[2][8];  // keys, values
  // scores may be computed: keys are there, and the weights in their place used up; are computed;
  // values and weights are there; are used up
  uint64_t s_ready[2], s_full[2], pv_ready[2], pv_done[2], q_full;
  uint64_t products_done[2];  // all that the scores' and the weighted values' thread issued
  uint32_t tmem;
  int gave_up;
  int gone[2][8];  // units of the last eight tiles that are not there (bits), by each loader
  int64_t sums[kWarps];
  int start_b;
  int64_t start_in;
};
static_assert(sizeof(Control) <= 1024, "in front of the operands");

// A bounded wait that the whole block gives up together: from then on every wait returns at once.  The
// loaders and the threads that issue products stop, the other roles run to their end on whatever is there.  No
// stage is filled again before its copies have landed, and copies and products in flight end before the block does.
__device__ __forceinline__ bool wait(Control* c, uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < ptx::kSpinLimit; ++i) {
    if (ptx::mbar_try(bar, parity & 1)) return true;
    if ((i & 15) == 15 && *(volatile int*)&c->gave_up) return false;
  }
  *(volatile int*)&c->gave_up = 1;
  return false;
}
// Waits, with a limit, for all products that this thread has issued: they read shared memory and write tensor
// memory that the block gives back at its end.  A barrier of its own, whose one phase nothing else completes.
__device__ __forceinline__ void products_end(uint64_t* bar) {
  ptx::umma_commit(bar);
  ptx::mbar_wait(bar, 0);
}
// Warps that wait for an mbarrier are woken, and poll, whenever any mbarrier of the block moves: with all
// of them doing so half of the issued instructions were polls.  So one softmax warp waits for the
// scores, and the others for it at a named barrier.
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
enum { kBarSoftmax = 1, kBarPair = 2 };

// A sequence's place on the line.  Row block i (from 1) of a head sees 128 / r tokens more than the one
// before, none while its rows lie before the first token, and no more than the window: in steps of
// 128 / r tokens clamp(base + i, 0, top).  Its cost is that and a fixed part; the sums are closed forms, so
// that ranges are equal in tokens though later rows of a prompt see more (a prompt of 2,048 tokens: the
// fullest block has 34 tiles where the mean is 30; with one cost for all row blocks of a sequence 56).
struct Line {
  int64_t base, top;
  int fixed;
  __device__ __forceinline__ Line(const AttnArgs& a, const Seq& s, int r)
      : base(((int64_t)s.past * r) >> 7),
        top(a.window > 0 ? (((int64_t)a.window * r) >> 7) + 2 : (int64_t)1 << 40), fixed(kItemTiles * r) {}
  __device__ __forceinline__ int64_t cost(int block) const {
    return fixed + min(max(base + block + 1, (int64_t)0), top);
  }
  // of a head's first k row blocks
  __device__ __forceinline__ int64_t sum(int k) const { return ramp(base, k) - ramp(base - top, k) + (int64_t)k * fixed; }

 private:
  // max(0, b + 1) + .. + max(0, b + k)
  static __device__ __forceinline__ int64_t ramp(int64_t b, int64_t k) {
    const int64_t i = max((int64_t)1, 1 - b), n = max((int64_t)0, k - i + 1);
    return n * b + (i + k) * n / 2;
  }
};

// The items of a block's range of the line, one at a time, the same in every role.  Each warp has its own
// in shared memory: in registers they would be spilled.
template <int D>
struct alignas(16) Items {
  int64_t left, from;
  int b, head, block;  // block: its row block
  Seq s;
  // of the current item
  int end, first, base_u, t0, t1;
  int64_t to, cost;
  __device__ __forceinline__ bool next(const AttnArgs& a, int r, bool begun) {
    __syncwarp();
    Items x = *this;
    __syncwarp();
    for (;; begun = true) {
      if (begun) {
        x.from = 0;
        if (x.left > 0 && ++x.block == x.s.blocks) {
          x.block = 0;
          if (++x.head == a.hkv) {
            x.head = 0;
            do x.s = load_seq<kRows>(a, ++x.b, r); while (x.s.blocks == 0);
          }
        }
      }
      if (x.left <= 0) return false;
      const Seq& s = x.s;
      const Line line(a, s, r);
      x.cost = line.cost(x.block);
      x.to = min(x.cost, x.from + x.left);
      x.left -= x.to - x.from;
      const uint32_t row0 = x.block * kRows, row1 = min(x.block * kRows + kRows, s.rows) - 1;
      x.end = max(0, s.past + (int)(row1 / (uint32_t)r));
      x.first = a.window > 0 ? max(0, s.past + (int)(row0 / (uint32_t)r) - a.window) : 0;
      x.base_u = x.first / kUnit;
      const int tiles = x.end > x.first ? (x.end - x.base_u * kUnit + kTile - 1) / kTile : 0;
      const int64_t full = x.cost - line.fixed;
      const float ratio = (float)tiles / (float)full;
      // Tiles before a place of the item.  No part has fewer than two: it would cost more than it takes over.
      // A place so near an end counts as that end, to the blocks on both sides of it.
      const auto share = [&](int64_t y) {
        if (y <= 0) return 0;
        if (y >= x.cost) return tiles;
        y -= line.fixed;
        const int n = y >= full ? tiles : y <= 0 ? 0 : min(tiles, (int)(y * ratio));
        return n > tiles - 2 ? tiles : n < 2 ? 0 : n;
      };
      x.t0 = share(x.from);
      x.t1 = share(x.to);
      if (x.from > 0) {
        if (x.t0 == tiles) continue;  // the block before ends it
        if (x.t0 == 0) x.from = 0;
      }
      if (x.to < x.cost) {
        if (x.t1 == tiles) x.to = x.cost;
        else if (x.t1 == 0) return false;  // the block behind begins it
      }
      break;
    }
    *this = x;  // every lane writes the same
    __syncwarp();
    return true;
  }
};

// ------------------------------------------------------------------------------ unpacking

__device__ __forceinline__ void sts16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The 8 codes of a word as exact fp16 numbers, in the order 0 4 | 1 5 | 2 6 | 3 7.
__device__ __forceinline__ void codes(uint32_t w, __half2 (&c)[4]) {
  const __half2 bias = h2(0xE400E400u), sixteenth = h2(0x2C002C00u), bias16 = h2(0xD400D400u);
  const uint32_t w8 = w >> 8;
  c[0] = __hadd2(h2(and_or<0x000F000Fu>(w, 0x64006400u)), bias);
  c[1] = __hfma2(h2(and_or<0x00F000F0u>(w, 0x64006400u)), sixteenth, bias16);
  c[2] = __hadd2(h2(and_or<0x000F000Fu>(w8, 0x64006400u)), bias);
  c[3] = __hfma2(h2(and_or<0x00F000F0u>(w8, 0x64006400u)), sixteenth, bias16);
}

// Eight tokens' keys (16 for d = 64), from row `row` of a tile on: 32 lanes, each a 16-byte chunk (4
// words) of a token.  Rows go K-major with the 128-byte swizzle; lanes are spread so that no eight of
// them meet in a bank.
template <int D, int G, bool EXACT>
__device__ __forceinline__ void unpack_keys(const uint32_t (&w)[4], const uint32_t (&sc)[D / G], uint32_t buf, int place, int ch, int row_unit) {
  using C = Shape<D, G, EXACT>;
  // packed row `place` holds token 0 4 1 5 2 6 3 7 (+ 8)
  const int n = row_unit + (place >> 1 & 3) + 4 * (place & 1) + (place & 8);
  const uint32_t krow = buf + n * 128;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int kb = j % C::KB, t = D == 128 ? ch : 2 * ch + (j >> 1), word = 4 * kb + t;
    const int g = 32 * kb / G;
    const uint32_t s = C::NG == 1 ? __byte_perm(sc[0], 0, 0x1010) : __byte_perm(sc[g / 2], 0, g & 1 ? 0x3232 : 0x1010);
    const uint32_t z = C::NG == 1 ? __byte_perm(sc[0], 0, 0x3232) : __byte_perm(sc[(C::NG + g) / 2], 0, g & 1 ? 0x3232 : 0x1010);
    __half2 c[4];
    codes(w[j], c);
    const uint32_t at = krow + (word >> 3) * (kTile * 128) + (((word & 7) ^ (n & 7)) << 4);
    if constexpr (EXACT) {
      const __half2 hi = h2(s & 0xFFF0FFF0u), lo = __hsub2(h2(s), hi);
      sts16(at, u32(__hmul2(c[0], hi)), u32(__hmul2(c[1], hi)), u32(__hmul2(c[2], hi)), u32(__hmul2(c[3], hi)));
      sts16(at + C::kOp, u32(__hmul2(c[0], lo)), u32(__hmul2(c[1], lo)), u32(__hmul2(c[2], lo)), u32(__hmul2(c[3], lo)));
    } else {
      sts16(at, u32(__hfma2(c[0], h2(s), h2(z))), u32(__hfma2(c[1], h2(s), h2(z))), u32(__hfma2(c[2], h2(s), h2(z))),
            u32(__hfma2(c[3], h2(s), h2(z))));
    }
  }
  if (EXACT && ch == 0) {
    // zeros twice (for the two parts of the sums of q), then nothing
    const uint32_t at = buf + 2 * C::kOp + ptx::noswz16_offset(n, 0);
    if constexpr (C::NG == 4) sts16(at, sc[2], sc[3], sc[2], sc[3]);
    else if constexpr (C::NG == 2) sts16(at, sc[1], sc[1], 0, 0);
    else sts16(at, __byte_perm(sc[0], 0, 0x3232), 0, 0, 0);
  }
}

// Which 32 coordinates a chunk of packed values holds.
template <int D>
__device__ __forceinline__ int value_group(int place, int ch) {
  return D == 128 ? ch ^ (place & 2) : ch;
}

// The same of values: rows go MN-major.  seen: somebody sees the token; its values are 0 otherwise.
template <int D, int G, bool EXACT>
__device__ __forceinline__ void unpack_values(uint32_t (&w)[4], uint32_t sz, uint32_t buf, int place, int ch, int row, bool seen) {
  using C = Shape<D, G, EXACT>;
  const int group = value_group<D>(place, ch);
  if (!seen) sz = 0;
  if (D == 128 && (group & 2)) {
    uint32_t x = w[0]; w[0] = w[2]; w[2] = x;
    x = w[1]; w[1] = w[3]; w[3] = x;
  }
  const __half2 st = h2(__byte_perm(sz, 0, 0x1010)), ze = h2(__byte_perm(sz, 0, 0x3232));
  const uint32_t vrow = buf + (row >> 3) * (C::NA * 1024) + (row & 7) * 128;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int word = 4 * group + (D == 128 ? j ^ (group & 2) : j);
    __half2 c[4];
    codes(w[j], c);
    sts16(vrow + (word >> 3) * 1024 + (((word & 7) ^ (row & 7)) << 4), u32(__hfma2(c[0], st, ze)), u32(__hfma2(c[1], st, ze)),
          u32(__hfma2(c[2], st, ze)), u32(__hfma2(c[3], st, ze)));
  }
}

// ------------------------------------------------------------------------------ the kernel

// An operand's descriptor `bytes` further on.  One addition: one thread issues a tile's products one
// after another, and whatever it computes between them is time of the tensor pipe's.
__device__ __forceinline__ uint64_t moved(uint64_t desc, uint32_t bytes) {
  uint64_t y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "r"((uint32_t)desc + bytes / 16), "r"((uint32_t)(desc >> 32)));
  return y;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(32 * kWarps, 1) rows_kernel(AttnArgs a, int page_shift) {
  constexpr bool kExact = __is_same(T, __half);
  using C = Shape<D, G, kExact>;
  constexpr int kRing = C::kRing;
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  __shared__ float shared_rows[2][2][kRows];  // numbers that the two threads of a row give each other
  Control& ctl = *reinterpret_cast<Control*>(raw_smem);
  uint8_t* smem = raw_smem + C::kControl;
  uint8_t* packed = smem + 2 * C::kBuf;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = a.hq / a.hkv;

  if (tid == 0) {
    ctl.gave_up = 0;
    for (int i = 0; i < kRing; ++i) {
      for (int k = 0; k < 2; ++k) {
        ptx::mbar_init(&ctl.ring_full[k][i], kChunkUnits);
        ptx::mbar_init(&ctl.ring_empty[k][i], 4);
      }
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl.s_ready[i], kKeyWarps + 1);
      ptx::mbar_arrive(&ctl.s_ready[i]);  // no weights before the first two tiles
      ptx::mbar_init(&ctl.s_full[i], 1);
      ptx::mbar_init(&ctl.pv_ready[i], kValueWarps + kSoftmaxWarps);
      ptx::mbar_init(&ctl.pv_done[i], 1);
    }
    ptx::mbar_init(&ctl.q_full, kSoftmaxWarps);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(&ctl.products_done[i], 1);
    ptx::fence_mbar_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc(&ctl.tmem, 512);
    ptx::tmem_relinquish();
  }
  // the upper half of the zeros' 16 numbers is never written again
  if (kExact)
    for (int i = tid; i < 2 * kTile; i += 32 * kWarps)
      sts16(ptx::smem_u32(smem) + (i / kTile) * C::kBuf + 2 * C::kOp + ptx::noswz16_offset(i % kTile, 8), 0, 0, 0, 0);
  ptx::fence_proxy_async_smem();

  // The line of all items' costs, cut into one range per block; the thread whose sequences hold the
  // range's start tells the block.
  static_assert(sizeof(Items<D>) == kItemBytes, "");
  Items<D>& it = reinterpret_cast<Items<D>*>(raw_smem + C::kItems)[warp];
  {
    Items<D> x = {};
    const int per = (a.B + 32 * kWarps - 1) / (32 * kWarps), b0 = tid * per, b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    for (int i = b0; i < b1; ++i) {
      x.s = load_seq<kRows>(a, i, r);
      mine += a.hkv * Line(a, x.s, r).sum(x.s.blocks);
    }
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, sum, d);
      if (lane >= d) sum += y;
    }
    if (lane == 31) ctl.sums[warp] = sum;
    __syncthreads();
    int64_t below = sum - mine, total = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) below += ctl.sums[w];
      total += ctl.sums[w];
    }
    const int64_t span = max((int64_t)(total * (1.0 / kCtas)) + 1, (int64_t)(kItemTiles + 1) * r);
    const int64_t x0 = blockIdx.x * span;
    for (int i = b0; i < b1 && below <= x0; ++i) {
      if (per > 1) {
        x.s = load_seq<kRows>(a, i, r);
        mine = a.hkv * Line(a, x.s, r).sum(x.s.blocks);
      }
      if (x0 < below + mine) {
        ctl.start_b = i;
        ctl.start_in = x0 - below;
      }
      below += mine;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    x.left = min(span, total - x0);
    x.from = x.b = x.head = x.block = 0;
    if (x.left > 0) {
      x.b = ctl.start_b;
      x.s = load_seq<kRows>(a, x.b, r);
      const Line line(a, x.s, r);
      const int64_t head = line.sum(x.s.blocks);
      x.head = (int)(ctl.start_in / head);
      x.from = ctl.start_in - x.head * head;
      // the last row block that begins at or before the place
      int lo = 0, hi = x.s.blocks;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (line.sum(mid) <= x.from) lo = mid; else hi = mid;
      }
      x.block = lo;
      x.from -= line.sum(lo);
    }
    it = x;
  }
  const uint32_t tmem = ctl.tmem;
  const uint32_t smem32 = ptx::smem_u32(smem), packed32 = smem32 + 2 * C::kBuf;
  uint32_t tile = 0;  // tiles so far, over all items: buffers and parities
  PartHeader* out_hdr = static_cast<PartHeader*>(a.workspace);

  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------------------------------------------------------- softmax
    RowsPart<D>* out_part = reinterpret_cast<RowsPart<D>*>(static_cast<uint8_t*>(a.workspace) + 2 * kCtas * sizeof(PartHeader));
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int half = warp >> 2, my_row = tid & (kRows - 1);
    int left_part[2] = {0, 0};
    uint32_t meets = 0;  // of the two warps that share rows
    // Gives the row's other thread a number and waits for its; both see what was done before.
    const auto meet = [&](float x) {
      shared_rows[meets & 1][half][my_row] = x;
      ptx::tc_fence_before();
      named_sync(kBarPair + (warp & 3), 64);
      ptx::tc_fence_after();
      ++meets;
    };
    const auto theirs = [&] { return shared_rows[(meets - 1) & 1][half ^ 1][my_row]; };
    // the whole role waits for an mbarrier
    const auto all_wait = [&](uint64_t* bar, uint32_t parity) {
      if (warp == 0) wait(&ctl, bar, parity);
      named_sync(kBarSoftmax, 32 * kSoftmaxWarps);
      ptx::tc_fence_after();
    };
    for (bool begun = false; it.next(a, r, begun); begun = true) {
      const uint32_t row = it.block * kRows + my_row;
      const bool in = row < (uint32_t)it.s.rows;
      const uint32_t tok = in ? row / r : 0, hh = in ? row - tok * r : 0;
      float m = -FLT_MAX, l = 0.f, kappa = 0.f;
      const uint32_t last_row = min(it.block * kRows + kRows, it.s.rows) - 1;
      const int hi = it.s.past + (int)(min(row, last_row) / (uint32_t)r), lo = a.window > 0 ? max(0, hi - a.window) : 0;
      if (it.t0 < it.t1) {
        // this thread's half row of q, by a power of two in fp16, its keys' order of coordinates
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(it.s.q0 + tok) * a.q_tok + (int64_t)(it.head * r + hh) * a.q_head + half * (D / 2);
        const bool wide = reinterpret_cast<uintptr_t>(src) % 16 == 0;
        uint32_t q[D / 4];
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {
          uint4 v = make_uint4(0, 0, 0, 0);
          const uint16_t* p = src + 8 * w;
          if (in && wide) {
            v = __ldg(reinterpret_cast<const uint4*>(p));
          } else if (in) {
            v.x = __ldg(p) | (uint32_t)__ldg(p + 1) << 16;
            v.y = __ldg(p + 2) | (uint32_t)__ldg(p + 3) << 16;
            v.z = __ldg(p + 4) | (uint32_t)__ldg(p + 5) << 16;
            v.w = __ldg(p + 6) | (uint32_t)__ldg(p + 7) << 16;
          }
          q[4 * w] = v.x;
          q[4 * w + 1] = v.y;
          q[4 * w + 2] = v.z;
          q[4 * w + 3] = v.w;
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
          top = fmaxf(top, fmaxf(fabsf(q_float<T>((uint16_t)q[i])), fabsf(q_float<T>((uint16_t)(q[i] >> 16)))));
        meet(top);
        top = fmaxf(top, theirs());
        const int e = top > 0.f ? max((int)(__float_as_uint(top) >> 23) - 134, -126) : 0;
        float down = __uint_as_float((uint32_t)(127 - e) << 23);
        kappa = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
        if (kappa < 0.f) {  // the largest score is the largest product
          kappa = -kappa;
          down = -down;
        }
        kappa = fmaxf(kappa, 1e-37f);  // so that -inf, a masked score, stays that
        constexpr int kSums = C::NG > 1 ? C::NG / 2 : 1;  // groups of half a row
        float sum[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) sum[i] = 0.f;
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {
          __half y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            y[k] = __float2half_rn(q_float<T>((uint16_t)(q[4 * w + k / 2] >> (16 * (k & 1)))) * down);
            if (kExact) sum[C::NG > 1 ? 8 * w / G : 0] += __half2float(y[k]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) q[4 * w + k] = u32(__halves2half2(y[k], y[k + 4]));
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < D / 4; c += 16) ptx::tmem_st16(lanes + C::Q + half * (D / 4) + c, *reinterpret_cast<uint32_t(*)[16]>(q + c));
        if (kExact) {
          float all[2 * kSums];
#pragma unroll
          for (int i = 0; i < kSums; ++i) {
            meet(sum[i]);
            all[i] = sum[i];
            all[kSums + i] = theirs();
          }
          if (half == 0) {
            if (C::NG == 1) all[0] += all[1];
            uint32_t qz[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            __half part[2][C::NG];
#pragma unroll
            for (int i = 0; i < C::NG; ++i) {
              part[0][i] = __float2half_rn(all[i]);
              part[1][i] = __float2half_rn(all[i] - __half2float(part[0][i]));
            }
            if constexpr (C::NG == 1) {
              qz[0] = u32(__halves2half2(part[0][0], part[1][0]));
            } else {
#pragma unroll
              for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < C::NG; i += 2) qz[(p * C::NG + i) / 2] = u32(__halves2half2(part[p][i], part[p][i + 1]));
            }
            ptx::tmem_st8(lanes + C::QZ, qz);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ctl.q_full);

        const int tiles = it.t1 - it.t0, pos = it.base_u * kUnit + it.t0 * kTile + 64 * half, see0 = lo - pos, see1 = hi - pos;
        for (int j = 0; j < tiles; ++j, ++tile) {
          const uint32_t buf = tile & 1, sp = lanes + C::S + 128 * buf + 64 * half;
          all_wait(&ctl.s_full[buf], tile >> 1);
          // what this row sees of these columns: [c0, c1), less units that are not there
          const int c0 = see0 - j * kTile, c1 = see1 - j * kTile, gone = *(volatile int*)&ctl.gone[0][tile & 7] >> (4 * half) & 15;
          const bool masked = __any_sync(~0u, c0 > 0 || c1 < 64 || gone != 0);
          // 32 columns at a time, read twice and not kept: what the loop saves in code the instruction
          // cache has for the other roles
          const auto scores = [&](int c, uint32_t (&s)[32]) {
            ptx::tmem_ld_cols<0, 32>(sp + c, s);
            ptx::tmem_wait_ld();
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c + i < c0 || c + i >= c1 || (gone >> ((c + i) / kUnit) & 1)) s[i] = 0xFF800000u;
            }
          };
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            uint32_t s[32];
            scores(c, s);
            float top4[4] = {top, top, top, top};
#pragma unroll
            for (int i = 0; i < 32; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                top4[k] = fmaxf(fmaxf(top4[k], __uint_as_float(s[i + k])), __uint_as_float(s[i + 4 + k]));
            top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
          }
          meet(top);
          top = fmaxf(top, theirs()) * kappa;
          if (__any_sync(~0u, top > m + (kLow + kLag))) {
            const float now = fmaxf(m, top - kLow), f = ex2(m - now);
            m = now;
            l *= f;
            if (j > 0) {
              // O is the softmax's once the tile before is in it; each warp takes half of the columns
              wait(&ctl, &ctl.pv_done[buf ^ 1], (tile - 1) >> 1);
              __syncwarp();
              ptx::tc_fence_after();
#pragma unroll 1
              for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                uint32_t o[16];
                ptx::tmem_ld16(lanes + C::O + c, o);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                ptx::tmem_st16(lanes + C::O + c, o);
              }
              ptx::tmem_wait_st();
            }
          }
          float sum4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            uint32_t s[32], p[16], pl[16];
            scores(c, s);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float s0 = __uint_as_float(s[2 * i]), s1 = __uint_as_float(s[2 * i + 1]);
              const float x = ex2(fmaf(s0, kappa, -m)), y = ex2(fmaf(s1, kappa, -m));
              sum4[i & 3] += x + y;
              const __half2 v = __floats2half2_rn(x, y);
              p[i] = u32(v);
              if (kExact) {
                const float2 back = __half22float2(v);
                pl[i] = u32(__floats2half2_rn(x - back.x, y - back.y));
              }
            }
            // in the place of their scores: 16 columns of weights, 16 of their second parts
            ptx::tmem_st16(sp + c, p);
            if (kExact) ptx::tmem_st16(sp + c + 16, pl);
          }
          l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&ctl.pv_ready[buf]);
        }
        all_wait(&ctl.pv_done[(tile - 1) & 1], (tile - 1) >> 1);
        meet(l);
        l += theirs();
        ptx::tc_fence_after();
      }
      const bool any = it.t0 < it.t1, whole = it.from == 0 && it.to == it.cost;
      const float inv = l > 0.f ? 1.0f / l : 0.f;
      const int k = it.from > 0 ? 0 : 1;
      RowsPart<D>* part = out_part + blockIdx.x * 2 + k;
      T* dst = static_cast<T*>(a.out) + ((int64_t)(it.s.q0 + tok) * a.hq + it.head * r + hh) * D;
#pragma unroll 1
      for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0;
        __syncwarp();
        if (any) {
          ptx::tmem_ld_cols<0, 32>(lanes + C::O + c, o);
          ptx::tmem_wait_ld();
        }
        if (!in) continue;
        float v[32];  // columns are coordinates 0 4 1 5 2 6 3 7 of each eight
#pragma unroll
        for (int i = 0; i < 32; ++i) v[(i & 24) + (i >> 1 & 3) + 4 * (i & 1)] = __uint_as_float(o[i]);
        if (whole) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(pack_out<T>(v[i] * inv, v[i + 1] * inv), pack_out<T>(v[i + 2] * inv, v[i + 3] * inv),
                                                                pack_out<T>(v[i + 4] * inv, v[i + 5] * inv), pack_out<T>(v[i + 6] * inv, v[i + 7] * inv));
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4) part->o[(c + i) / 4][my_row] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      }
      if (!whole) {
        if (in && half == 0) {
          part->m[my_row] = m;
          part->l[my_row] = l;
        }
        left_part[k] = 1;
        if (tid == 0) out_hdr[blockIdx.x * 2 + k] = PartHeader{it.to == it.cost ? 3 : 1, it.s.q0, it.s.rows, it.head, it.block};
      }
      // O is read before the next item's first product: its q comes after the warps met here
      if (any) meet(0.f);
    }
    if (tid == 0)
      for (int k = 0; k < 2; ++k)
        if (!left_part[k]) out_hdr[blockIdx.x * 2 + k].state = 0;
  } else if (warp < kSoftmaxWarps + kUnpackWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ---------------------------------------------------------------- unpack
    constexpr int kStep = 1024 / D;  // tokens of a warp's step
    const bool keys = warp < kSoftmaxWarps + kKeyWarps;
    const int ch = lane % (D / 32), row_lane = lane / (D / 32);
    uint32_t chunk = 0;
    for (bool begun = false; it.next(a, r, begun); begun = true) {
      const int tiles = it.t1 - it.t0, pos0 = it.base_u * kUnit + it.t0 * kTile, first = it.first - pos0, end = it.end - pos0;
      for (int j = 0; j < tiles; ++j, ++tile) {
        const uint32_t buf = tile & 1, base = smem32 + buf * C::kBuf;
        // keys are done with when their scores are, values when the products with the weights are
        if (tile >= 2) wait(&ctl, keys ? &ctl.s_full[buf] : &ctl.pv_done[buf], (tile - 2) >> 1);
#pragma unroll 1
        for (int c = 0; c < C::kChunks; ++c, ++chunk) {
          const uint32_t slot = chunk % kRing;
          wait(&ctl, &ctl.ring_full[!keys][slot], chunk / kRing);
          __syncwarp();
          const uint32_t at = packed32 + (keys ? slot * C::kKeys : kRing * C::kKeys + slot * C::kValues);
          constexpr int kSteps = kChunkUnits * kUnit / (4 * kStep);
          const int row0 = (warp & 3) * kStep + row_lane, place = row0 % kUnit;
          const int gone = keys ? 0 : *(volatile int*)&ctl.gone[1][tile & 7];
#pragma unroll 1
          for (int i = 0; i < kSteps; ++i) {
            const int unit = (4 * i * kStep + row0) / kUnit;
            const uint32_t codes_at = at + unit * (keys ? C::kCodes : C::kValue);
            uint32_t w[4], sc[C::NG];
            lds<16>(codes_at + place * (D / 2) + ch * 16, w);
            const int row = c * kChunkUnits * kUnit + 4 * i * kStep + row0;  // of the tile
            if (keys) {
              lds<4 * C::NG>(at + kChunkUnits * C::kCodes + unit * C::kScales + place * 4 * C::NG, sc);
              unpack_keys<D, G, kExact>(w, sc, base, place, ch, row & ~(kUnit - 1));
            } else {
              lds<4>(codes_at + C::kCodes + C::kScales + (place * C::NG + value_group<D>(place, ch) * 32 / G) * 4, sc);
              const int pos = j * kTile + row;
              unpack_values<D, G, kExact>(w, sc[0], base + C::kK, place, ch, row, pos >= first && pos < end && !(gone >> (row / kUnit) & 1));
            }
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&ctl.ring_empty[!keys][slot]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(keys ? &ctl.s_ready[buf] : &ctl.pv_ready[buf]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSoftmaxWarps + kUnpackWarps) {
      // ---------------------------------------------------------------- scores
      constexpr uint32_t idesc = ptx::idesc_f16_f32(128, kTile);
      bool ok = true, issued = false;
      uint32_t item = 0;
      for (bool begun = false; ok && it.next(a, r, begun); begun = true) {
        const int tiles = it.t1 - it.t0;
        if (tiles <= 0) continue;
        if (lane == 0) {
          ok = wait(&ctl, &ctl.q_full, item);
          for (uint32_t t = tile; t < tile + tiles && ok; ++t) {
            const uint32_t buf = t & 1, base = smem32 + buf * C::kBuf, d = tmem + C::S + 128 * buf;
            ok = wait(&ctl, &ctl.s_ready[buf], t >> 1);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint64_t keys = ptx::sdesc_kmajor_sw128(base);
#pragma unroll
            for (int part = 0; part < (kExact ? 2 : 1); ++part)
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                ptx::umma_f16_ts(d, tmem + C::Q + 8 * ks, moved(keys, part * C::kOp + (ks >> 2) * (kTile * 128) + (ks & 3) * 32), idesc,
                                 part > 0 || ks > 0 ? 1u : 0u);
            if (kExact) ptx::umma_f16_ts(d, tmem + C::QZ, ptx::sdesc_kmajor_noswz(base + 2 * C::kOp, 128, 256), idesc, 1u);
            ptx::umma_commit(&ctl.s_full[buf]);
            issued = true;
          }
        }
        ok = __shfl_sync(~0u, (int)ok, 0);
        tile += tiles;
        ++item;
      }
      if (issued) products_end(&ctl.products_done[0]);
    } else if (warp == kSoftmaxWarps + kUnpackWarps + 1) {
      // ---------------------------------------------------------------- weighted values
      constexpr uint32_t idesc = ptx::idesc_f16_f32(128, D) | (1u << 16);
      bool ok = true, issued = false;
      for (bool begun = false; ok && it.next(a, r, begun); begun = true) {
        const int tiles = it.t1 - it.t0;
        if (lane == 0)
          for (uint32_t t = tile; t < tile + tiles; ++t) {
            const uint32_t buf = t & 1, weights = tmem + C::S + 128 * buf;
            ok = wait(&ctl, &ctl.pv_ready[buf], t >> 1);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint64_t values = ptx::sdesc_mnmajor_sw128(smem32 + buf * C::kBuf + C::kK, 1024, C::NA * 1024);
#pragma unroll
            for (int part = 0; part < (kExact ? 2 : 1); ++part)
#pragma unroll
              for (int ks = 0; ks < kTile / 16; ++ks)
                ptx::umma_f16_ts(tmem + C::O, weights + 32 * (ks >> 1) + 8 * (ks & 1) + 16 * part, moved(values, ks * 2 * C::NA * 1024), idesc,
                                 t > tile || part > 0 || ks > 0 ? 1u : 0u);
            ptx::umma_commit(&ctl.pv_done[buf]);
            ptx::umma_commit(&ctl.s_ready[buf]);
            issued = true;
          }
        ok = __shfl_sync(~0u, (int)ok, 0);
        tile += max(tiles, 0);
      }
      if (issued) products_end(&ctl.products_done[1]);
    } else {
      // ---------------------------------------------------------------- loaders
      const bool keys = warp == kSoftmaxWarps + kUnpackWarps + 2;
      const int ring = keys ? 0 : 1, stage = keys ? C::kKeys : C::kValues;
      const uint8_t* cache = a.cache + (keys ? 0 : C::kCodes);
      // where lane i's unit of a stage goes: lanes at .. at + 3 copy its four units
      uint8_t* dst = packed + (keys ? (lane % kChunkUnits) * C::kCodes : kRing * C::kKeys + (lane % kChunkUnits) * C::kValue);
      bool ok = true;
      const int shift = page_shift - 4;
      uint32_t chunk = 0;
      for (bool begun = false; ok && it.next(a, r, begun); begun = true) {
        const int32_t* table = a.tables + (int64_t)it.b * a.max_blocks;
        const int u_begin = it.base_u + it.t0 * kTileUnits, u_end = min(it.base_u + it.t1 * kTileUnits, (it.end + kUnit - 1) / kUnit);
        auto entry = [&](int u) { return u < u_end ? __ldg(table + (u >> shift)) : -1; };
        // lane i holds the table entry of units i, i + 32, ... of the part; the next 32 are on their way
        int id_next = it.t0 < it.t1 ? entry(u_begin + lane) : -1;
        const uint8_t* src = nullptr;
        uint32_t there = 0;
        const int chunks = (it.t1 - it.t0) * C::kChunks, head = it.head;
        for (int j = 0; j < chunks; ++j, ++chunk) {
          const int at = (j * kChunkUnits) & 31;
          if (at == 0) {
            const int id = id_next, u = u_begin + j * kChunkUnits + lane;
            id_next = entry(u + 32);
            there = __ballot_sync(~0u, id >= 0 && id < a.n_blocks);
            src = cache + ((((int64_t)id * a.hkv + head) << shift) + (u & ((1 << shift) - 1))) * C::UB;
          }
          const uint32_t slot = chunk % kRing;
          // a warp whose wait gave up has said that the stage is empty all the same: its copies may be on their way
          if (chunk >= kRing) ok = __all_sync(~0u, wait(&ctl, &ctl.ring_empty[ring][slot], chunk / kRing - 1) && !*(volatile int*)&ctl.gave_up);
          if (!ok) break;
          if (lane / kChunkUnits == at / kChunkUnits) {
            uint64_t* bar = &ctl.ring_full[ring][slot];
            // A tile's first chunk brings its mask.  The place is free: a ring holds four tiles at most, the keys
            // of the tile four back are unpacked when the scores of the one six back are done, and these come
            // after the weighted values of the one eight back.
            if (j % C::kChunks == 0 && lane == at)
              *(volatile int*)&ctl.gone[ring][(chunk / C::kChunks) & 7] = ~(there >> (at & ~(kTileUnits - 1))) & ((1 << kTileUnits) - 1);
            if (there >> lane & 1) {
              ptx::mbar_arrive_expect_tx(bar, keys ? C::kCodes + C::kScales : C::kValue);
              ptx::bulk_load(dst + slot * stage, src, keys ? C::kCodes : C::kValue, bar);
              if (keys)
                ptx::bulk_load(packed + slot * stage + kChunkUnits * C::kCodes + (lane % kChunkUnits) * C::kScales, src + 2 * C::kCodes, C::kScales, bar);
            } else {
              ptx::mbar_arrive(bar);
            }
          }
          __syncwarp();
        }
      }
      // whoever's wait it was that gave up; where none did they have landed
      drain(chunk > kRing ? chunk - kRing : 0, chunk, kRing, [&](uint32_t slot, uint32_t parity) { ptx::mbar_wait(&ctl.ring_full[ring][slot], parity); });
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (ctl.gave_up && tid == 0) atomicAdd(&g_kv4_rows_wait_timeouts, 1u);
  if (warp == 0) ptx::tmem_dealloc(tmem, 512);
  asm volatile("griddepcontrol.launch_dependents;");
}

// Joins the parts of the items that span blocks: blocks (c, i) rows 16 i .. of the item begun in block
// c of the first kernel.
template <typename T, int D>
__global__ void __launch_bounds__(128) rows_join_kernel(AttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PartHeader* hdr = static_cast<const PartHeader*>(a.workspace);
  const RowsPart<D>* part = reinterpret_cast<const RowsPart<D>*>(static_cast<const uint8_t*>(a.workspace) + 2 * kCtas * sizeof(PartHeader));
  const int c0 = blockIdx.x;
  const PartHeader h = hdr[c0 * 2 + 1];
  if (h.state != 1) return;
  const int rows = min(kRows, h.rows - h.rb * kRows);
  if ((int)blockIdx.y * 16 >= rows) return;
  const int end = last_part(hdr, c0);
  const uint32_t r = a.hq / a.hkv;
  for (int i = threadIdx.x; i < 16 * D / 4; i += 128) {
    const int row = blockIdx.y * 16 + i % 16, c = i / 16 * 4;
    if (row >= rows) continue;
    float m = -FLT_MAX, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = c0; p <= end; ++p) {
      const RowsPart<D>& x = part[p * 2 + (p == c0)];
      const float mx = x.m[row], now = fmaxf(m, mx), f0 = ex2(m - now), f1 = ex2(mx - now);
      const float4 y = x.o[c / 4][row];
      o.x = fmaf(y.x, f1, o.x * f0);
      o.y = fmaf(y.y, f1, o.y * f0);
      o.z = fmaf(y.z, f1, o.z * f0);
      o.w = fmaf(y.w, f1, o.w * f0);
      l = fmaf(x.l[row], f1, l * f0);
      m = now;
    }
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    const uint32_t at = h.rb * kRows + row, tok = at / r;
    T* dst = static_cast<T*>(a.out) + ((int64_t)(h.q0 + tok) * a.hq + h.head * r + at - tok * r) * D + c;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_out<T>(o.x * inv, o.y * inv), pack_out<T>(o.z * inv, o.w * inv));
  }
}

template <typename T, int D, int G>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  constexpr size_t bytes = Shape<D, G, __is_same(T, __half)>::kSmem;
  static_assert(bytes + 4 * 2 * 2 * kRows <= 227 * 1024, "shared memory of a block");
  static_assert(sizeof(RowsPart<D>) % 16 == 0, "parts are read in 16 bytes");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may have this much shared memory
  if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(rows_kernel<T, D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  int shift = 4;
  while ((1 << shift) < a.page) ++shift;
  rows_kernel<T, D, G><<<kCtas, 32 * kWarps, bytes, st>>>(a, shift);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas, kRows / 16);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, rows_join_kernel<T, D>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_shape(const AttnArgs& a, cudaStream_t st) {
  if (a.d == 64) return a.group == 32 ? launch<T, 64, 32>(a, st) : launch<T, 64, 64>(a, st);
  if (a.group == 32) return launch<T, 128, 32>(a, st);
  return a.group == 64 ? launch<T, 128, 64>(a, st) : launch<T, 128, 128>(a, st);
}

}  // namespace

size_t attn_rows_workspace_bytes(int d) {
  return 2 * kCtas * (sizeof(PartHeader) + (d == 64 ? sizeof(RowsPart<64>) : sizeof(RowsPart<128>)));
}

cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t st) {
  return a.type == FQ_F16 ? launch_shape<__half>(a, st) : launch_shape<__nv_bfloat16>(a, st);
}

cudaError_t wait_timeouts_kv4_rows(bool clear, unsigned* count) {
  return read_wait_counter(g_kv4_rows_wait_timeouts, clear, count);
}

}  // namespace kv4
}  // namespace fq
