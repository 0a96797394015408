// 8-bit codes of a cache with block scales: exact conversions to f16.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace pa {

// Denominators sum a weight over its V scale, up to 2^15 times 2^100 (kLeastScale) a key; counted in units of 2^20
// they stay below 2^127 for 2^30 keys of one row.
constexpr float kDenScale = 0x1p-20f;
constexpr float kDenBias = 20.f;

// log2 of such a denominator, which under the largest V scales is subnormal (lg2 takes those for 0).
__device__ __forceinline__ float lg2_den(float l) { return l < 1.f ? lg2(l * 0x1p60f) - 60.f : lg2(l); }

// Two e4m3 codes (the low or high half of w) as f16x2, exactly.
template <int HALF>
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (HALF == 0) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  }
  return r;
}

// A byte of ones for each NaN among four e4m3 codes.
__device__ __forceinline__ uint32_t e4m3_nan4(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// Two int8 codes as f16x2, exactly.  x holds the codes with their sign bits
// flipped (u = code + 128); SEL picks two bytes and puts 0x64 above each:
// 0x6400 + u is the f16 number 1024 + u, and 1152 = 0x6480 taken off leaves the code.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t int8x2_to_f16x2(uint32_t x) {
  const uint32_t h = __byte_perm(x, 0x64646464u, SEL);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
  return r;
}

// D = A(16x16, row) * B(16x8, col) + D, f16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace pa
