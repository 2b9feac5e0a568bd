// Attention over the 4-bit paged cache, in its plainest form: one block per (query token, query
// head) walks the tokens it may see, 128 at a time, with the running maximum and sum of a softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.h"

namespace fq {
namespace kv4 {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float load_q(const void* q, fq_dtype t, int64_t i) {
  return t == FQ_F16 ? __half2float(static_cast<const __half*>(q)[i])
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i]);
}

// The unit of token position `pos` of sequence b, or null when its page is not in the pool.
__device__ __forceinline__ const uint8_t* unit_of(const AttnArgs& a, int b, int head, int pos) {
  const int id = a.tables[(int64_t)b * a.max_blocks + pos / a.page];
  if (id < 0 || id >= a.n_blocks) return nullptr;
  return a.cache + (((int64_t)id * a.hkv + head) * (a.page / kUnit) + pos % a.page / kUnit) *
                       unit_bytes(a.d, a.group);
}

__device__ float block_reduce(float x, bool is_max, float* part) {
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    const float y = __shfl_xor_sync(~0u, x, m);
    x = is_max ? fmaxf(x, y) : x + y;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
  __syncthreads();
  x = part[0];
  for (int i = 1; i < kThreads / 32; ++i) x = is_max ? fmaxf(x, part[i]) : x + part[i];
  return x;
}

__global__ void __launch_bounds__(kThreads) attn_kernel(AttnArgs a) {
  __shared__ float q[128], p[kThreads], part[4];
  const int64_t row = blockIdx.x / a.hq;
  const int h = blockIdx.x % a.hq, head = h / (a.hq / a.hkv), tid = threadIdx.x;
  int b = (int)row, m = 1, i = 0;
  if (a.cu_q) {
    for (b = 0; b < a.B; ++b)
      if (row >= a.cu_q[b] && row < a.cu_q[b + 1]) break;
    if (b == a.B) return;  // a row behind the last sequence
    m = a.cu_q[b + 1] - a.cu_q[b];
    i = (int)(row - a.cu_q[b]);
  }
  const int64_t room = (int64_t)a.max_blocks * a.page;
  const int n = (int)min((int64_t)max(a.kv_lens[b], 0), room);
  const int end = min(n, n - m + i + 1), first = a.window > 0 ? max(0, end - a.window) : 0;
  for (int c = tid; c < a.d; c += kThreads) q[c] = load_q(a.q, a.type, row * a.q_tok + h * a.q_head + c);
  __syncthreads();
  const int ng = a.d / a.group;
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (int t0 = first; t0 < end; t0 += kThreads) {
    const int pos = t0 + tid, ut = pos % kUnit;
    float s = -INFINITY;
    const uint8_t* unit = pos < end ? unit_of(a, b, head, pos) : nullptr;
    if (unit) {
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(unit) + key_row(ut) * (a.d / 8);
      const __half* sz = reinterpret_cast<const __half*>(unit + off_ks(a.d)) + key_row(ut) * 2 * ng;
      s = 0.f;
      for (int w = 0; w < a.d / 8; ++w) {
        const uint32_t word = codes[key_word(w, a.d)];
        const int g = w * 8 / a.group;
        const float step = __half2float(sz[g]), zero = __half2float(sz[ng + g]);
        for (int e = 0; e < 8; ++e)
          s += q[8 * w + e] * fmaf((float)((word >> (4 * e)) & 15), step, zero);
      }
      s *= a.scale;
    }
    const float now = fmaxf(top, block_reduce(s, true, part));
    const float base = now == -INFINITY ? 0.f : now;
    const float keep = expf(top - base);
    p[tid] = expf(s - base);
    sum = sum * keep + block_reduce(p[tid], false, part);  // its barriers publish p
    acc *= keep;
    top = now;
    for (int j = 0; j < kThreads && t0 + j < end; ++j) {
      if (p[j] == 0.f || tid >= a.d) continue;  // a masked token's codes and steps may hold anything
      const uint8_t* u = unit_of(a, b, head, t0 + j);
      const int tt = (t0 + j) % kUnit;
      const uint32_t word = reinterpret_cast<const uint32_t*>(u + off_v(a.d))[tt * (a.d / 8) + value_word(tid / 8, tt, a.d)];
      const __half* sz = reinterpret_cast<const __half*>(u + off_vs(a.d, a.group)) + (tt * ng + tid / a.group) * 2;
      acc += p[j] * fmaf((float)((word >> (4 * (tid % 8))) & 15), __half2float(sz[0]), __half2float(sz[1]));
    }
    __syncthreads();
  }
  if (tid < a.d) {
    const float o = sum > 0.f ? acc / sum : 0.f;
    const int64_t at = (row * a.hq + h) * a.d + tid;
    if (a.type == FQ_F16) static_cast<__half*>(a.out)[at] = __float2half_rn(o);
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o);
  }
}

}  // namespace

size_t attn_workspace_bytes(int) { return 16; }

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st) {
  attn_kernel<<<(unsigned)(a.n_q * a.hq), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kv4
}  // namespace fq
