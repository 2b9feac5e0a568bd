// Quantised write of new keys and values into the 4-bit paged cache.
//
// Per (token, kv head, group of G coordinates), all in fp32:
//   z = fp16(min),  s = fp16((max - z) * fp32(1/15)),  c = clamp(rint((x - z) * (1 / s)), 0, 15)
// (c = 0 where s = 0); the cache then stands for c s + z.  The record keeps z and s in 16 bits, so
// the codes are taken against the rounded z and s: what is lost to their rounding is not lost twice.
// A NaN makes its group's min, max, z and s NaN: the group reads as NaN and its codes are 0.
//
// Bound by HBM: 2 d elements in, d + 8 d / G bytes out (and 2 d elements with the values) per (token,
// kv head).  One thread takes 8 coordinates (a 16-byte load and one 32-bit word of codes) of a
// token's key and of its value; a block takes the same kv head of 2048 / d consecutive tokens, whose
// rows share units: their 4-byte stores join to whole sectors in L2.  What it computes is kept to
// about 20 instructions per element, or it would be bound by their issue: rounding on floats (adding
// 1.5 2^23 rounds to the nearest even integer), no clamping where a group's two ends round to 0 and
// 15 by themselves, codes joined by exact FMAs.  Measured: 65,536 tokens, 8 kv heads of 128, bf16, values
// written too, 621 MB: 120 us, 5,160 GB/s, 0.79 of a copy's; 5,003 tokens, 3 heads of 64, fp32: 4.3 us.
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

__device__ __forceinline__ uint32_t pack2(__half, float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The least and the largest of three, NaN if one of them is (fminf and fmaxf leave a NaN out); one instruction.
__device__ __forceinline__ float min3(float a, float b, float c) {
  float y;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// The same of two.
__device__ __forceinline__ float min2(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max2(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Quantises this thread's 8 coordinates with the other lanes of its group; returns the code word
// and, in `sz`, the group's s (low half) and z.
template <typename T, int G>
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t& sz, T* values) {
  float lo = min3(min3(x[0], x[1], x[2]), min3(x[3], x[4], x[5]), min2(x[6], x[7]));
  float hi = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max2(x[6], x[7]));
#pragma unroll
  for (int m = 1; m < G / 8; m <<= 1) {
    lo = min2(lo, __shfl_xor_sync(~0u, lo, m));
    hi = max2(hi, __shfl_xor_sync(~0u, hi, m));
  }
  const __half z16 = __float2half_rn(min2(max2(lo, -65504.f), 65504.f));
  const float z = __half2float(z16);
  const __half s16 = __float2half_rn(min2(max2((hi - z) * (1.0f / 15.0f), 0.f), 65504.f));
  const float s = __half2float(s16);
  const float inv = s > 0.f ? 1.0f / s : 0.f;
  sz = (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(z16) << 16);
  const float magic = 12582912.f;  // 1.5 2^23: what is added to it is rounded to an integer
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __fmul_rn(__fsub_rn(x[i], z), inv);
  // The roundings of z and s seldom move a group's ends past half a step.  In a group with a NaN all of c is
  // NaN, the test fails, and the clamping, which leaves a NaN out, makes it 0.
  if (!((lo - z) * inv >= -0.5f && (hi - z) * inv < 15.5f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(c[i], 0.f), 15.f);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __fadd_rn(__fadd_rn(c[i], magic), -magic);
  if (values) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        reinterpret_cast<float4*>(values)[i] = make_float4(fmaf(c[4 * i], s, z), fmaf(c[4 * i + 1], s, z),
                                                           fmaf(c[4 * i + 2], s, z), fmaf(c[4 * i + 3], s, z));
    } else {
      uint4 w;
      w.x = pack2(T{}, fmaf(c[0], s, z), fmaf(c[1], s, z));
      w.y = pack2(T{}, fmaf(c[2], s, z), fmaf(c[3], s, z));
      w.z = pack2(T{}, fmaf(c[4], s, z), fmaf(c[5], s, z));
      w.w = pack2(T{}, fmaf(c[6], s, z), fmaf(c[7], s, z));
      *reinterpret_cast<uint4*>(values) = w;
    }
  }
  // four codes in the low 16 bits of a float between 2^23 and 2^24
  const float low = fmaf(c[3], 4096.f, fmaf(c[2], 256.f, fmaf(c[1], 16.f, c[0] + 8388608.f)));
  const float high = fmaf(c[7], 4096.f, fmaf(c[6], 256.f, fmaf(c[5], 16.f, c[4] + 8388608.f)));
  return __byte_perm(__float_as_uint(low), __float_as_uint(high), 0x5410);
}

template <typename T, int D, int G, bool VEC>
__global__ void __launch_bounds__(kThreads, 6) write_kernel(WriteArgs a, int page_shift) {
  constexpr int kLanes = D / 8, NG = D / G;
  const uint32_t head = blockIdx.x % (uint32_t)a.hkv;
  const int tok = blockIdx.x / (uint32_t)a.hkv * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int w = threadIdx.x % kLanes;  // this thread's word of 8 coordinates
  const bool in = tok < a.n;
  const int t = in ? tok : (int)a.n - 1;  // all lanes take part in the shuffles
  float kx[8], vx[8];
  load8<T, VEC>(static_cast<const T*>(a.k) + t * a.k_tok + head * a.k_head + 8 * w, kx);
  load8<T, VEC>(static_cast<const T*>(a.v) + t * a.v_tok + head * a.v_head + 8 * w, vx);
  const int slot = __ldg(a.slots + t);
  const int64_t dense = ((int64_t)t * a.hkv + head) * D + 8 * w;
  uint32_t ksz, vsz;
  const uint32_t kc = quantise<T, G>(kx, ksz, in && a.k_values ? static_cast<T*>(a.k_values) + dense : nullptr);
  const uint32_t vc = quantise<T, G>(vx, vsz, in && a.v_values ? static_cast<T*>(a.v_values) + dense : nullptr);
  if (!in || slot < 0 || (slot >> page_shift) >= a.n_blocks) return;
  const int ut = slot % kUnit, row = key_row(ut);
  const int64_t page = (int64_t)(slot >> page_shift) * a.hkv + head;
  uint8_t* unit = a.cache + ((page << (page_shift - 4)) + ((slot & (a.page - 1)) >> 4)) * unit_bytes(D, G);
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
  int shift = 4;
  while ((1 << shift) < a.page) ++shift;
  const auto fits = [](const void* p, int64_t s0, int64_t s1) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 * (int64_t)sizeof(T) % 16 == 0 && s1 * (int64_t)sizeof(T) % 16 == 0;
  };
  if (fits(a.k, a.k_tok, a.k_head) && fits(a.v, a.v_tok, a.v_head))
    write_kernel<T, D, G, true><<<(unsigned)blocks, kThreads, 0, st>>>(a, shift);
  else
    write_kernel<T, D, G, false><<<(unsigned)blocks, kThreads, 0, st>>>(a, shift);
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
