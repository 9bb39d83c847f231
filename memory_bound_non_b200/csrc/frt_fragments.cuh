// Operands of the tensor-core kernels that read NVFP4.
#pragma once

#include "frt_device.cuh"

namespace frt {

// NVFP4 codes as the 16-bit operands of mma.m16n8k16.  An e2m1 value times an
// e4m3 factor has at most 6 significant bits and lies in [2^-10, 2688], so
// code * sf is exact in binary16; the fp32 global scale is applied to sums.

// Eight e2m1 codes (element 0 in the low nibble) -> four binary16 pairs.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Four e4m3 codes (low byte first) -> two binary16 pairs.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
}
// One e4m3 code in both halves.
__device__ __forceinline__ uint32_t e4m3_to_both(uint32_t code) {
  uint32_t h;
  asm("{\n\t.reg .b16 w;\n\tcvt.u16.u32 w, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, w;\n\t}" : "=r"(h) : "r"(code * 0x0101u));
  return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// D += A B on a 16x16 by 16x8 tile, binary16 operands, fp32 sums.  With
// g = lane / 4 and t = lane % 4: a = {(g, 2t), (g + 8, 2t), (g, 2t + 8),
// (g + 8, 2t + 8)} (row, first of two columns), b = {(2t, g), (2t + 8, g)}
// (first of two rows, column), d = {(g, 2t), (g, 2t + 1), (g + 8, 2t),
// (g + 8, 2t + 1)}.
__device__ __forceinline__ void mma_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 binary16 tile held as (row g, columns 2t, 2t + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Power of two that brings magnitude amax (> 0) into [2^14, 2^15), at most 2^most
// (with 127: below 2^-113 the bf16 numbers, multiples of 2^-133, are exact in
// binary16 all the same); 1 for zero and NaN amax.  Beside an infinity the finite
// numbers stay finite.
__device__ __forceinline__ float pow2_to_half_range(float amax, int most = 127) {
  const int e = min((int)(__float_as_uint(amax) >> 23) - 127, 127);  // amax >= 0; subnormals count as 2^-127
  if (!(amax > 0.0f)) return 1.0f;
  return __int_as_float((min(14 - e, most) + 127) << 23);  // (14 - e >= -113)
}
// The largest power for which `scale` divided by it is a normal number.
__device__ __forceinline__ int most_pow2(float scale) {
  return min((int)(__float_as_uint(scale) >> 23 & 0xFF) - 1, 127);
}

}  // namespace frt
