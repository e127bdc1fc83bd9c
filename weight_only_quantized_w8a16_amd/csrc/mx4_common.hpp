// mx4_common.hpp -- device helpers of the microscaled 4-bit (MX4) kernels:
// the layouts of include/qgemm.h, scale bytes, and the gfx950 conversions.
//
// A scale byte s reaches the conversion instructions as the exponent field
// of an fp32 operand; they read that field alone, s = 0 as 2^-127 and
// s = 255 as NaN (checked for every code and scale byte by the tests).
#pragma once

#include "qg_common.hpp"
#include "qg_launch.hpp"

namespace qg {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Tiled scales: dwords of four 128-k blocks, 64 lanes per (16 rows x 512 k).
__host__ __device__ constexpr int mx4_scale_windows(int K) { return (K + 511) / 512; }

// Byte b (0 .. 3) of a scale word as an fp32 operand of the conversions.
__device__ __forceinline__ float mx4_scale_operand(uint32_t word, int b) {
  return __uint_as_float(((word >> (8 * b)) & 0xFFu) << 23);
}

// One 32-bit word of eight codes -> eight values in the 16-bit type DT:
// exact in bf16, rounded to nearest even in fp16.
template <int DT>
__device__ __forceinline__ u32x4 mx4_word_to_operand(uint32_t w, float scale) {
  u32x4 r;
  if constexpr (DT == kFP16) {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3));
  } else {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  }
  return r;
}

// 16 x 16 x 128 product of two MX4 fragments (lane: row or column lane % 16,
// block lane / 16 of the 128 k), each lane's block scale in byte B of its
// scale word.
template <int B>
__device__ __forceinline__ f32x4 mx4_mfma(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x4 x = __builtin_bit_cast(i32x4, a), y = __builtin_bit_cast(i32x4, b);
  constexpr int kFP4 = 4;   // operand format code
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1),
      __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1), c, kFP4, kFP4, B,
      static_cast<int>(sa), B, static_cast<int>(sb));
}

}  // namespace qg
