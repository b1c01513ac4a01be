// dsa_paged_quant.cuh -- the bytes of a row of a quantised cache, and its codes as numbers.
#pragma once
#include <cuda_fp16.h>

#include "dsa_device.cuh"

namespace dsa {

// Where the parts of a row of D channels lie, Q of them quantised to BITS bits (see include/dsa.h).
struct QuantRow {
  int blocks;  // block scales (4 bits)
  int scale;   // s
  int tail;    // the other channels
  int bytes;   // of the row
};
__host__ __device__ constexpr QuantRow quant_row(int D, int Q, int bits) {
  const int blocks = bits == 8 ? Q : Q / 2, scale = bits == 8 ? Q : Q / 2 + Q / 16;
  const int tail = (scale + 4 + 15) / 16 * 16;
  return QuantRow{blocks, scale, tail, tail + (2 * (D - Q) + 15) / 16 * 16};
}
__host__ __device__ constexpr bool quant_row_ok(int D, int Q, int bits) {
  return (bits == 8 || bits == 4) && Q >= 64 && Q % 64 == 0 && D >= Q && D <= 1024 && (D - Q) % 8 == 0;
}

// Two codes (the lower one in the lower half) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// The four pairs of codes e2m1 of a word, in the order of their channels.
__device__ __forceinline__ void e2m1x8_f16x2(uint32_t v, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(v));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 f16x2_floats(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

}  // namespace dsa
