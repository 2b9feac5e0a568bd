// What the two attention kernels over the 4-bit cache share: how items are cut, how q is read and
// out written, small wrappers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.h"
#include "sm100_ptx.cuh"

namespace fq {
namespace kv4 {

constexpr int kCtas = 148;  // one block per SM

// Weights are fp16 numbers in the products, whose range ends at 2^16 and at 2^-25.  They are taken against a
// number kLow below the row's maximum, which moves when a score passes that maximum by kLag: the largest weights
// are 2^7, never above 2^15, and one of 2^-32 of the largest still counts.  Against the maximum itself those
// below 2^-25 were lost; 131,072 such tokens together weigh up to 1/256 of the largest.
constexpr float kLow = 7.f, kLag = 8.f;

struct Seq {
  int n, m, q0, rows, blocks;  // tokens, query tokens, first row of q, rows per kv head, row blocks of NB
  int past;                    // tokens that the first query token sees, none if below 1
};

template <int NB>
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b, int r) {
  Seq s;
  s.n = min(max(__ldg(a.kv_lens + b), 0), a.max_blocks * a.page);
  s.q0 = b;
  s.m = 1;
  if (a.cu_q) {
    s.q0 = __ldg(a.cu_q + b);
    const int q1 = __ldg(a.cu_q + b + 1);
    s.m = s.q0 >= 0 && q1 > s.q0 && q1 <= a.n_q ? q1 - s.q0 : 0;
  }
  s.rows = min(s.m, a.max_q) * r;  // those past max_q keep their places and are left out
  s.blocks = (s.rows + NB - 1) / NB;
  s.past = s.n - s.m + 1;
  return s;
}

// (x & MASK) | bits in one instruction, the mask in it
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "n"(MASK), "r"(bits));
  return y;
}

__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int BYTES>
__device__ __forceinline__ void lds(uint32_t at, uint32_t* x) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(at));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[0]) : "r"(at));
}

template <typename T>
__device__ __forceinline__ float q_float(uint16_t x) {
  if constexpr (sizeof(T) == 2 && !__is_same(T, __half)) return __uint_as_float((uint32_t)x << 16);
  else return __half2float(__ushort_as_half(x));
}
template <typename T>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
  if constexpr (__is_same(T, __half)) {
    return u32(__floats2half2_rn(a, b));
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

}  // namespace kv4
}  // namespace fq
