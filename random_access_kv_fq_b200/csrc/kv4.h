// The 4-bit paged key/value cache: layout of a unit and the launchers of its kernels.
//
// A unit holds 16 consecutive tokens of one kv head, keys and values, as fq.h describes it.  Its
// parts and the order of their rows are those of the attention kernel's matrix fragments, so that
// a warp reads each part with full-width shared-memory loads and no bank conflicts; a token's
// codes and a token's steps and zeros are each contiguous, so that a write touches whole sectors.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "fq.h"

namespace fq {
namespace kv4 {

constexpr int kUnit = 16;            // tokens of a unit
constexpr int kMaxRequests = 8192;   // requests of one page step (their scans sit in shared memory)
constexpr int kMinPage = 16, kMaxPage = 1024;
constexpr int kMaxHeads = 1 << 20;  // query heads: what an item costs beside its tokens, kItemTiles of them, is an int
constexpr int kMaxWindow = 1 << 30;  // the longest sequence: wider ones are cut to it, so that a place less a window is an int

__host__ __device__ constexpr int unit_bytes(int d, int group) {
  return kUnit * d + 128 * (d / group);
}
// byte offsets of a unit's parts
__host__ __device__ constexpr int off_v(int d) { return kUnit * d / 2; }
__host__ __device__ constexpr int off_ks(int d) { return kUnit * d; }
__host__ __device__ constexpr int off_vs(int d, int group) { return kUnit * d + 64 * (d / group); }

// row of token t (0..15) in the key parts
__host__ __device__ constexpr int key_row(int t) { return 2 * (t & 3) + ((t >> 2) & 1) + (t & 8); }
// 32-bit word (8 coordinates) w of a key row sits at this word of the row ...
__host__ __device__ constexpr int key_word(int w, int d) { return (w & 3) * (d / 32) + (w >> 2); }
// ... and of token t's value row at this one
__host__ __device__ constexpr int value_word(int w, int t, int d) {
  return d == 128 ? w ^ (((t >> 1) & 1) << 3) : w;
}

// place / cost, for a quotient below 2^30.  A 64-bit division takes a warp some hundred cycles at the start of
// every call; this estimate is off by one at most below 2^22 items, and by 2^-22 of them above.
__host__ __device__ inline int item_of(int64_t place, int cost) {
  int item = (int)((float)place / (float)cost);
  while ((int64_t)item * cost > place) --item;
  while (place - (int64_t)item * cost >= cost) ++item;
  return item;
}

// Waits until the copies of steps first .. last - 1 of a ring have landed: step t fills stage t % ring for the
// (t / ring)th time.  wait(stage, parity) is a bounded wait for one phase.  A block whose waits gave up must
// not end, nor write where the ring is, before that: a copy still on its way would land in whatever is there.
template <typename Wait>
__host__ __device__ inline void drain(uint32_t first, uint32_t last, uint32_t ring, Wait wait) {
  for (uint32_t t = first; t < last; ++t) wait(t % ring, t / ring & 1);
}

struct WriteArgs {
  const void* k;
  const void* v;
  fq_dtype type;
  int64_t n;
  int hkv, d;
  int64_t k_tok, k_head, v_tok, v_head;  // strides in elements
  const int32_t* slots;
  uint8_t* cache;
  int64_t n_blocks;
  int page, group;
  void* k_values;
  void* v_values;
};

struct AttnArgs {
  const void* q;
  fq_dtype type;
  int64_t n_q;
  int hq, d;
  int64_t q_tok, q_head;  // strides in elements
  const int32_t* cu_q;
  int B, max_q;
  const uint8_t* cache;
  int64_t n_blocks;
  int hkv, page, group;
  const int32_t* tables;
  int max_blocks;
  const int32_t* kv_lens;
  int window;  // 0 .. kMaxWindow
  float scale;
  void* out;
  void* workspace;
};

struct PageArgs {
  const int32_t* lens;
  const int32_t* new_lens;
  int B;
  int32_t* tables;
  int max_blocks, page;
  int32_t* free_list;
  int n_blocks;
  const int32_t* free_count;
  int32_t* lens_out;
  int32_t* free_count_out;
  int32_t* cu_new;
  int32_t* slots;
  int n_slots;
  int32_t* refused;
};

cudaError_t launch_write(const WriteArgs& a, cudaStream_t st);
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_page_step(const PageArgs& a, cudaStream_t st);
size_t attn_workspace_bytes(int B, int hq, int hkv, int d, int max_q, int64_t capacity);
cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t st);  // many rows of a kv head
size_t attn_rows_workspace_bytes(int d);
cudaError_t wait_timeouts_kv4(bool clear, unsigned* count);  // as those in fq_internal.h
cudaError_t wait_timeouts_kv4_rows(bool clear, unsigned* count);

// Rows of a kv head, by a call's max_q, up to which the register-fed kernel runs: where the two meet for d = 128
// (24 sequences of 6,000 tokens, 4 kv heads, 1 to n drafted tokens: 32 rows 49 us against 75, 48 rows 61, 64
// rows 75).  For d = 64 they would meet later: 33 us against 68, 39, and 48 at 64 rows.
constexpr int64_t kFewRows = 64;

}  // namespace kv4
}  // namespace fq
