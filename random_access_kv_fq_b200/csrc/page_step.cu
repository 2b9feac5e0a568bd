// Block tables, slots and the free list of a paged cache, advanced by one serving step on the GPU.
//
// Exclusive sums over the requests give each its first new token, its first new page and its
// place among the released pages; the a-th new page of the step is the a-th from the top of the
// free stack, so every page, table entry and slot has a closed form and nothing is atomic.
//
// Bound by latency: at most a few bytes per request, page and slot.  One launch: every block of
// one cluster computes the sums itself (B values from L2, the sums in shared memory), so no block
// waits for another's sums; two cluster barriers order (1) all reads of lens and free_count before
// they may be overwritten in place and (2) released pages before they are handed out again.  The
// slots are written one thread each, the request found by bisection of the sums in shared memory.
#include <climits>

#include <cooperative_groups.h>

#include "kv4.h"

namespace fq {
namespace kv4 {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kCluster = 8;

__device__ __forceinline__ int sat(int64_t x) { return x > INT_MAX ? INT_MAX : (int)x; }

// Inclusive block-wide sum of one value per thread; `total` gets the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* part, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, x, m);
    if (lane >= m) x += y;
  }
  __syncthreads();  // `part` may still be read from the scan before
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int64_t below = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) below += part[i];
    total += part[i];
  }
  return x + below;
}

// the last of a[0..n) that is <= x (a ascending, a[0] <= x)
__device__ __forceinline__ int last_le(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_step_kernel(PageArgs a) {
  extern __shared__ int sums[];
  __shared__ int64_t part[kThreads / 32];
  int* cu = sums;              // [B + 1] first new token of a request
  int* off = cu + a.B + 1;     // [B]     first new page
  int* rel = off + a.B;        // [B]     first released page
  int* held = rel + a.B;       // [B]     tokens held before the step; ~held when it is refused
  const cg::cluster_group cluster = cg::this_cluster();
  const int n_thr = kThreads * cluster.num_blocks();
  const int me = cluster.block_rank() * kThreads + threadIdx.x;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  const int64_t room = (int64_t)a.max_blocks * a.page;
  const int count = min(max(__ldcg(a.free_count), 0), a.n_blocks);

  // this thread's requests: tokens to add and pages to release
  int64_t tokens = 0, released = 0, total_tokens, total_released, total_need, total_refused, total_taken;
  for (int b = b0; b < b1; ++b) {
    const int add = __ldcg(a.new_lens + b);
    const int h = (int)min((int64_t)max(__ldcg(a.lens + b), 0), room);
    held[b] = h;
    off[b] = add;
    if (add < 0) released += (h + (int64_t)a.page - 1) / a.page; else tokens += add;
  }
  int64_t at = block_scan(tokens, part, total_tokens) - tokens;
  int64_t gone = block_scan(released, part, total_released) - released;
  const int avail = (int)min((int64_t)a.n_blocks, count + total_released);
  int64_t need = 0;
  for (int b = b0; b < b1; ++b) {
    const int add = off[b];
    const int64_t h = held[b], pages = (h + a.page - 1) / a.page;
    cu[b] = sat(at);
    rel[b] = sat(gone);
    if (add < 0) { gone += pages; continue; }
    at += add;
    if (h + add <= room && at <= a.n_slots) need += (h + add + a.page - 1) / a.page - pages;
  }
  int64_t upto = block_scan(need, part, total_need) - need;
  int64_t refused = 0, taken = 0;
  // cu, rel of this thread's requests are final; off and held get their final meaning
  int64_t tok_end = at;
  at = tok_end - tokens;
  for (int b = b0; b < b1; ++b) {
    const int add = off[b];
    const int64_t h = held[b], pages = (h + a.page - 1) / a.page;
    off[b] = sat(upto);
    if (add < 0) continue;
    at += add;
    const bool fits = h + add <= room && at <= a.n_slots;
    const int64_t n = fits ? (h + add + a.page - 1) / a.page - pages : 0;
    upto += n;
    if (!fits || (n > 0 && upto > avail)) {
      held[b] = ~held[b];
      ++refused;
    } else if (n > 0) {
      taken += n;
    }
  }
  block_scan(refused, part, total_refused);
  block_scan(taken, part, total_taken);
  if (threadIdx.x == 0) cu[a.B] = sat(total_tokens);
  __syncthreads();
  cluster.sync();  // lens and free_count are read: they may be overwritten now

  for (int b = me; b < a.B; b += n_thr) {
    const int h = held[b], next = cu[b + 1] - cu[b];
    const bool out = a.new_lens[b] < 0;
    a.lens_out[b] = out ? 0 : h < 0 ? ~h : h + next;
  }
  for (int b = me; b <= a.B; b += n_thr) a.cu_new[b] = cu[b];
  if (me == 0) {
    *a.free_count_out = avail - (int)total_taken;
    *a.refused = (int)total_refused;
  }
  for (int r = me; r < avail - count; r += n_thr) {
    const int b = last_le(rel, a.B, r);
    a.free_list[count + r] = a.tables[(int64_t)b * a.max_blocks + (r - rel[b])];
  }
  cluster.sync();  // released pages are on the stack

  for (int p = me; p < (int)total_taken; p += n_thr) {
    const int b = last_le(off, a.B, p);
    const int pages = (held[b] + a.page - 1) / a.page;
    a.tables[(int64_t)b * a.max_blocks + pages + (p - off[b])] = __ldcg(a.free_list + (avail - 1 - p));
  }
  for (int i = me; i < a.n_slots; i += n_thr) {
    int slot = -1;
    if (i < cu[a.B]) {
      const int b = last_le(cu, a.B, i);
      const int h = held[b];
      if (h >= 0) {
        const int pos = h + (i - cu[b]), pg = pos / a.page, pages = (h + a.page - 1) / a.page;
        const int id = pg < pages ? a.tables[(int64_t)b * a.max_blocks + pg]
                                  : __ldcg(a.free_list + (avail - 1 - (off[b] + pg - pages)));
        if (id >= 0 && id < a.n_blocks) slot = id * a.page + pos % a.page;
      }
    }
    a.slots[i] = slot;
  }
}

}  // namespace

cudaError_t launch_page_step(const PageArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(int) * (4 * (size_t)a.B + 1);
  cudaError_t e = cudaFuncSetAttribute(page_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(sizeof(int) * (4 * kMaxRequests + 1)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // one block does a small step; a cluster shares the stores of a large one
  const unsigned blocks = (int64_t)a.n_slots + a.B <= 4 * kThreads ? 1 : kCluster;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, page_step_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kv4
}  // namespace fq
