// Block tables, slots and the free list of a paged cache, advanced by one serving step on the GPU.
//
// Exclusive sums over the requests give each its first new token, its first new page and its
// place among the released pages; the a-th new page of the step is the a-th from the top of the
// free stack, so every page, table entry and slot has a closed form and nothing is atomic.
//
// Bound by latency: a few bytes per request, page and slot, behind four dependent steps (lengths,
// sums, pages, slots).  One launch: every block of one cluster computes the sums itself (B values
// from L2, the sums in shared memory), so no block waits for another's sums; two cluster barriers
// order (1) all reads of lens and free_count before they may be overwritten in place and (2)
// released pages before they are handed out again.  A warp writes 32 or 256 slots at a time: it finds
// the requests of the first and the last by bisection and its lanes search only between them.
// Measured: 256 decodes 5.0 to 5.4 us; 2,048 requests with prompts, releases and 262,144 slots 15 us, on 16
// multiprocessors and with a second barrier of the cluster between released pages and new ones.
#include <atomic>
#include <climits>

#include <cooperative_groups.h>

#include "kv4.h"

namespace fq {
namespace kv4 {
namespace {

namespace cg = cooperative_groups;


__device__ __forceinline__ int sat(int64_t x) { return x > INT_MAX ? INT_MAX : (int)x; }

__device__ __forceinline__ int64_t warp_scan(int64_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// Exclusive block-wide sums of two values per thread; `total` gets the block's sums.
struct Two {
  int64_t a, b;
};
__device__ __forceinline__ Two block_scan(Two x, Two* part, Two& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const Two up{warp_scan(x.a), warp_scan(x.b)};
  __syncthreads();  // `part` may still be read from the scan before
  if (lane == 31) part[warp] = up;
  __syncthreads();
  Two w{0, 0};
  if (lane < warps) w = part[lane];
  const Two all{warp_scan(w.a), warp_scan(w.b)};
  total = Two{__shfl_sync(~0u, all.a, 31), __shfl_sync(~0u, all.b, 31)};
  return Two{__shfl_sync(~0u, all.a - w.a, warp) + up.a - x.a,
             __shfl_sync(~0u, all.b - w.b, warp) + up.b - x.b};
}

// the last of a[lo..hi) that is <= x (a ascending, a[lo] <= x)
__device__ __forceinline__ int last_le(const int* a, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The same by a whole warp, 32 places at a time.
__device__ __forceinline__ int warp_last_le(const int* a, int lo, int hi, int x) {
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const int stride = (hi - lo + 31) / 32, i = lo + lane * stride;
    lo += (__popc(__ballot_sync(~0u, i < hi && a[i] <= x)) - 1) * stride;
    hi = min(hi, lo + stride);
  }
  return lo;
}

template <bool ALONE>
__global__ void __launch_bounds__(1024) page_step_kernel(PageArgs a, int page_shift) {
  // slots of a lane at a time: in a large step their searches and table reads are in flight together
  constexpr int kSlots = ALONE ? 1 : 8;
  extern __shared__ int sums[];
  __shared__ Two part[32];
  __shared__ int taken, refused;
  int* cu = sums;              // [B + 1] first new token of a request
  int* off = cu + a.B + 1;     // [B]     first new page
  int* rel = off + a.B;        // [B]     first released page
  int* held = rel + a.B;       // [B]     tokens held before the step; ~held when it is refused
  const cg::cluster_group cluster = cg::this_cluster();
  const auto all_blocks = [&] {
    if (ALONE) __syncthreads(); else cluster.sync();
  };
  const int rank = ALONE ? 0 : (int)cluster.block_rank();
  const int threads = blockDim.x, n_thr = threads * (ALONE ? 1 : (int)cluster.num_blocks()), me = rank * threads + threadIdx.x;
  const int per = (a.B + threads - 1) / threads;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  const int64_t room = (int64_t)a.max_blocks << page_shift;
  const int count = min(max(__ldcg(a.free_count), 0), a.n_blocks);
  const auto pages_of = [&](int64_t tokens) { return (tokens + a.page - 1) >> page_shift; };

  if (threadIdx.x == 0) taken = refused = 0;
  // this thread's requests: tokens to add and pages to release
  Two mine{0, 0}, total;
  for (int b = b0; b < b1; ++b) {
    const int add = __ldcg(a.new_lens + b);
    const int h = (int)min((int64_t)max(__ldcg(a.lens + b), 0), room);
    held[b] = h;
    off[b] = add;
    if (add < 0) mine.b += pages_of(h); else mine.a += add;
  }
  const Two first = block_scan(mine, part, total);
  const int64_t total_tokens = total.a;
  const int avail = (int)min((int64_t)a.n_blocks, count + total.b);
  // the pages that they need, if they fit the table and the slots
  Two need{0, 0};
  int64_t at = first.a, gone = first.b;
  for (int b = b0; b < b1; ++b) {
    const int add = off[b];
    const int64_t h = held[b];
    cu[b] = sat(at);
    rel[b] = sat(gone);
    if (add < 0) {
      gone += pages_of(h);
    } else {
      at += add;
      if (h + add <= room && at <= a.n_slots) need.a += pages_of(h + add) - pages_of(h);
    }
  }
  int64_t upto = block_scan(need, part, total).a;
  // a request that fits is served while the pages needed up to it are there
  int last_page = 0, turned_away = 0;  // behind the last page handed out; requests refused
  at = first.a;
  for (int b = b0; b < b1; ++b) {
    const int add = off[b];
    const int64_t h = held[b];
    off[b] = sat(upto);
    if (add < 0) continue;
    at += add;
    const bool fits = h + add <= room && at <= a.n_slots;
    const int64_t n = fits ? pages_of(h + add) - pages_of(h) : 0;
    upto += n;
    if (!fits || (n > 0 && upto > avail)) {
      held[b] = ~held[b];
      ++turned_away;
    } else if (n > 0) {
      last_page = (int)upto;
    }
  }
  last_page = __reduce_max_sync(~0u, last_page);
  turned_away = __reduce_add_sync(~0u, turned_away);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&taken, last_page);
    atomicAdd(&refused, turned_away);
  }
  if (threadIdx.x == 0) cu[a.B] = sat(total_tokens);
  all_blocks();  // the sums are there; lens and free_count are read and may be overwritten

  for (int b = me; b < a.B; b += n_thr) {
    const int h = held[b], next = cu[b + 1] - cu[b];
    const bool out = __ldcg(a.new_lens + b) < 0;
    a.lens_out[b] = out ? 0 : h < 0 ? ~h : h + next;
  }
  for (int b = me; b <= a.B; b += n_thr) a.cu_new[b] = cu[b];
  if (me == 0) {
    *a.free_count_out = avail - taken;
    *a.refused = refused;
  }
  if (avail > count) {
    for (int r = me; r < avail - count; r += n_thr) {
      const int b = last_le(rel, 0, a.B, r);
      a.free_list[count + r] = a.tables[(int64_t)b * a.max_blocks + (r - rel[b])];
    }
    all_blocks();  // released pages are on the stack
  }

  for (int p = me; p < taken; p += n_thr) {
    const int b = last_le(off, 0, a.B, p);
    a.tables[(int64_t)b * a.max_blocks + (int)pages_of(held[b]) + (p - off[b])] = __ldcg(a.free_list + (avail - 1 - p));
  }
  const int lane = threadIdx.x & 31, written = min(a.n_slots, cu[a.B]);
  for (int i0 = (me >> 5) * 32 * kSlots; i0 < a.n_slots; i0 += n_thr * kSlots) {
    int lo = 0, hi = 1;
    if (i0 < written) {
      lo = warp_last_le(cu, 0, a.B, i0);
      const int last = min(i0 + 32 * kSlots, written) - 1;
      hi = cu[lo + 1] > last ? lo + 1 : warp_last_le(cu, lo, a.B, last) + 1;
    }
    if (!ALONE && hi - lo == 1 && i0 + 32 * kSlots <= written) {
      // all 256 of one request
      const int h = held[lo], pages = (int)pages_of(h), first_pos = h + (i0 + lane - cu[lo]);
      const int32_t* row = a.tables + (int64_t)lo * a.max_blocks;
      const int32_t* fresh = a.free_list + (avail - 1 - off[lo] + pages);  // page pg >= pages is fresh[-pg]
      int id[kSlots];
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        const int pg = (first_pos + 32 * k) >> page_shift;
        id[k] = h < 0 ? -1 : pg < pages ? row[pg] : __ldcg(fresh - pg);
      }
#pragma unroll
      for (int k = 0; k < kSlots; ++k)
        a.slots[i0 + 32 * k + lane] = (unsigned)id[k] < (unsigned)a.n_blocks ? (id[k] << page_shift) + ((first_pos + 32 * k) & (a.page - 1)) : -1;
      continue;
    }
    int at[kSlots], id[kSlots], in[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k) at[k] = lo;
    for (int step = hi - lo > 1 ? 1 << (31 - __clz(hi - lo)) : 0; step; step >>= 1) {
#pragma unroll
      for (int k = 0; k < kSlots; ++k)
        if (at[k] + step < hi && cu[at[k] + step] <= i0 + 32 * k + lane) at[k] += step;
    }
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const int i = i0 + 32 * k + lane, b = at[k];
      id[k] = -1;
      in[k] = 0;
      if (i < written) {
        const int h = held[b];
        if (h >= 0) {
          const int pos = h + (i - cu[b]), pg = pos >> page_shift, pages = (int)pages_of(h);
          in[k] = pos & (a.page - 1);
          id[k] = pg < pages ? a.tables[(int64_t)b * a.max_blocks + pg]
                             : __ldcg(a.free_list + (avail - 1 - (off[b] + pg - pages)));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const int i = i0 + 32 * k + lane;
      if (i < a.n_slots) a.slots[i] = id[k] >= 0 && id[k] < a.n_blocks ? (id[k] << page_shift) + in[k] : -1;
    }
  }
}

// Blocks of the cluster that a large step runs on: 16, or the 8 that are always to be had where the device
// cannot place 16 (2,048 requests, prompts, releases and 262,144 slots: 14.8 us with 16, 21.0 with 8).
cudaError_t cluster_blocks(cudaLaunchConfig_t& cfg, int* blocks) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *blocks = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*blocks > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(page_step_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  // asked for the largest step, so that the answer holds for every one
  cudaLaunchConfig_t most = cfg;
  most.blockDim = dim3(1024);
  most.dynamicSmemBytes = sizeof(int) * (4 * (size_t)kMaxRequests + 1);
  e = cudaFuncSetAttribute(page_step_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most.dynamicSmemBytes);
  if (e != cudaSuccess) return e;
  int fit = 0;
  most.gridDim = dim3(16);
  most.attrs[0].val.clusterDim.x = 16;
  e = cudaOccupancyMaxActiveClusters(&fit, page_step_kernel<false>, &most);
  if (e != cudaSuccess) cudaGetLastError();  // not a size that it knows
  *blocks = e == cudaSuccess && fit > 0 ? 16 : 8;
  if (dev < 64) known[dev].store(*blocks, std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_page_step(const PageArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(int) * (4 * (size_t)a.B + 1);
  // One block does a small step: its barriers cost less.  A cluster shares the searches and stores of a
  // large one.  In us, one block and the cluster: 256 decodes 5.0 and 6.8, with every 17th request
  // released 8.4 and 8.0; 1,024 such requests 14.1 and 10.9; 4,096 of them 36.2 and 15.7.
  // Few requests need few warps: their sums are sooner there.
  const bool alone = (int64_t)a.n_slots + a.B <= 1024;
  const auto kernel = alone ? page_step_kernel<true> : page_step_kernel<false>;
  int shift = 0;
  while ((1 << shift) < a.page) ++shift;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(a.B <= 256 && a.n_slots <= 2048 ? 256 : 1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = alone ? 0 : 1;
  if (!alone) {
    int blocks = 8;
    const cudaError_t e = cluster_blocks(cfg, &blocks);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(blocks);
    at[0].val.clusterDim.x = blocks;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, shift);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kv4
}  // namespace fq
