// Matrix fragments of the decode kernels (decode.cu, paged_decode.cu): softmax
// weights packed to 16 bits, and key and value rows of bf16 or int8 codes as
// mma.sync operands.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace aircache {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi, float& lo_r, float& hi_r) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  lo_r = __low2float(t);
  hi_r = __high2float(t);
  return *reinterpret_cast<uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi, float& lo_r, float& hi_r) {
  __half2 t = __floats2half2_rn(lo, hi);
  lo_r = __low2float(t);
  hi_r = __high2float(t);
  return *reinterpret_cast<uint32_t*>(&t);
}
// D(16x8, fp32) += A(16x16, f16, row) * B(16x8, f16, col)
__device__ __forceinline__ void mma_f16_16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The int8 path multiplies in f16 (codes are exact there), the bf16 path in bf16.
template <bool F16>
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16) {
    mma_f16_16816(c, a, b0, b1);
  } else {
    mma_bf16_16816(c, a, b0, b1);
  }
}
// P leaves the int8 path's softmax scaled by 2^14 (its largest weight, 1,
// becomes 16384 < 65504): weights down to 2^-28 stay normal f16 numbers.
constexpr float kP16 = 16384.f;

__device__ __forceinline__ void ldsm_x4_trans(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Two int8 codes (the bytes `sel` picks of u4, whose top bits the caller has
// flipped) -> two f16, exactly, without a conversion instruction: code c
// becomes the unsigned byte u = c + 128 (flip
// the top bit), the byte permute places u in the low mantissa bits of the f16
// 0x6400 (= 1024), so the half is 1024 + u, and one packed subtraction of 1152
// leaves c (every integer below 2048 is an f16).
__device__ __forceinline__ uint32_t widen2_f16(uint32_t u4, uint32_t sel) {
  uint32_t t = __byte_perm(u4, 0x64646464u, sel);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&t), __float2half2_rn(1152.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset within an int8 tile of the 128-byte swizzle (D = 128: rows of
// 128 bytes, 16-byte pieces XORed with the row mod 8) or the 64-byte swizzle
// (D = 64: pieces XORed with bits 7-8 of the offset), as the TMA copy places
// them (each tile starts on a 1024-byte boundary).
template <int D>
__device__ __forceinline__ int swz8(int off) {
  return off ^ (((off >> 7) & (D == 128 ? 7 : 3)) << 4);
}

}  // namespace aircache
