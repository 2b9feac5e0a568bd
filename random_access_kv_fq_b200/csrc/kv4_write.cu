// Quantised write of new keys and values into the 4-bit paged cache.
//
// Per (token, kv head, group of G coordinates), all in fp32:
//   z = fp16(min),  s = fp16((max - z) * fp32(1/15)),  c = clamp(rint((x - z) * (1 / s)), 0, 15)
// (c = 0 where s = 0); the cache then stands for c s + z.  The record keeps z and s in 16 bits, so
// the codes are taken against the rounded z and s: what is lost to their rounding is not lost twice.
//
// Bound by HBM: 2 d elements in, d + 8 d / G bytes out per (token, kv head), ~15 instructions per
// element.  One thread takes 8 coordinates (a 16-byte load and one 32-bit word of codes) of a
// token's key and of its value, a block the same kv head of 2048 / d consecutive tokens, whose
// rows share units: their 4-byte stores join to whole sectors in L2.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.h"

namespace fq {
namespace kv4 {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ float from_float(float x) { return x; }

template <typename T>
struct alignas(16) Pack {
  T x[8];
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (VEC) {
    Pack<T> v;
    uint4* w = reinterpret_cast<uint4*>(&v);
#pragma unroll
    for (int i = 0; i < (int)sizeof(v) / 16; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float(v.x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float(p[i]);
  }
}

// Quantises this thread's 8 coordinates with the other lanes of its group; returns the code word
// and, in `sz`, the group's s (low half) and z.
template <typename T, int G>
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t& sz, T* values) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int m = 1; m < G / 8; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(~0u, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, m));
  }
  const __half z16 = __float2half_rn(fminf(fmaxf(lo, -65504.f), 65504.f));
  const float z = __half2float(z16);
  const __half s16 = __float2half_rn(fminf(fmaxf((hi - z) * (1.0f / 15.0f), 0.f), 65504.f));
  const float s = __half2float(s16);
  const float inv = s > 0.f ? 1.0f / s : 0.f;
  sz = (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(z16) << 16);
  uint32_t word = 0;
  Pack<T> out;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = fminf(fmaxf(rintf((x[i] - z) * inv), 0.f), 15.f);
    word |= (uint32_t)c << (4 * i);
    out.x[i] = from_float<T>(fmaf(c, s, z));
  }
  if (values) {
    uint4* w = reinterpret_cast<uint4*>(&out);
#pragma unroll
    for (int i = 0; i < (int)sizeof(out) / 16; ++i) reinterpret_cast<uint4*>(values)[i] = w[i];
  }
  return word;
}

template <typename T, int D, int G, bool VEC>
__global__ void __launch_bounds__(kThreads) write_kernel(WriteArgs a) {
  constexpr int kLanes = D / 8, NG = D / G;
  const int head = blockIdx.x % a.hkv;
  const int64_t tok = (int64_t)(blockIdx.x / a.hkv) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int w = threadIdx.x % kLanes;  // this thread's word of 8 coordinates
  const bool in = tok < a.n;
  const int64_t t = in ? tok : a.n - 1;  // all lanes take part in the shuffles
  float kx[8], vx[8];
  load8<T, VEC>(static_cast<const T*>(a.k) + t * a.k_tok + head * a.k_head + 8 * w, kx);
  load8<T, VEC>(static_cast<const T*>(a.v) + t * a.v_tok + head * a.v_head + 8 * w, vx);
  const int64_t slot = a.slots[t];
  const int64_t dense = (t * a.hkv + head) * D + 8 * w;
  uint32_t ksz, vsz;
  const uint32_t kc = quantise<T, G>(kx, ksz, in && a.k_values ? static_cast<T*>(a.k_values) + dense : nullptr);
  const uint32_t vc = quantise<T, G>(vx, vsz, in && a.v_values ? static_cast<T*>(a.v_values) + dense : nullptr);
  if (!in || slot < 0 || slot >= a.n_blocks * a.page) return;
  const int64_t block = slot / a.page;
  const int at = (int)(slot % a.page), ut = at % kUnit, row = key_row(ut);
  uint8_t* unit = a.cache + ((block * a.hkv + head) * (a.page / kUnit) + at / kUnit) * (int64_t)unit_bytes(D, G);
  reinterpret_cast<uint32_t*>(unit)[row * (D / 8) + key_word(w, D)] = kc;
  reinterpret_cast<uint32_t*>(unit + off_v(D))[ut * (D / 8) + value_word(w, ut, D)] = vc;
  if (w % (G / 8) == 0) {
    const int g = w / (G / 8);
    uint16_t* ks = reinterpret_cast<uint16_t*>(unit + off_ks(D)) + row * 2 * NG;
    ks[g] = (uint16_t)ksz;
    ks[NG + g] = (uint16_t)(ksz >> 16);
    reinterpret_cast<uint32_t*>(unit + off_vs(D, G))[ut * NG + g] = vsz;
  }
}

template <typename T, int D, int G>
cudaError_t launch(const WriteArgs& a, cudaStream_t st) {
  const int64_t per = kThreads / (D / 8);
  const int64_t blocks = (a.n + per - 1) / per * a.hkv;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const auto fits = [](const void* p, int64_t s0, int64_t s1) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 * (int64_t)sizeof(T) % 16 == 0 && s1 * (int64_t)sizeof(T) % 16 == 0;
  };
  if (fits(a.k, a.k_tok, a.k_head) && fits(a.v, a.v_tok, a.v_head))
    write_kernel<T, D, G, true><<<(unsigned)blocks, kThreads, 0, st>>>(a);
  else
    write_kernel<T, D, G, false><<<(unsigned)blocks, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_shape(const WriteArgs& a, cudaStream_t st) {
  if (a.d == 64) return a.group == 32 ? launch<T, 64, 32>(a, st) : launch<T, 64, 64>(a, st);
  if (a.group == 32) return launch<T, 128, 32>(a, st);
  return a.group == 64 ? launch<T, 128, 64>(a, st) : launch<T, 128, 128>(a, st);
}

}  // namespace

cudaError_t launch_write(const WriteArgs& a, cudaStream_t st) {
  if (a.type == FQ_F16) return launch_shape<__half>(a, st);
  if (a.type == FQ_BF16) return launch_shape<__nv_bfloat16>(a, st);
  return launch_shape<float>(a, st);
}

}  // namespace kv4
}  // namespace fq
