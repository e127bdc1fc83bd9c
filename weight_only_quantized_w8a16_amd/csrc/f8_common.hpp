// f8_common.hpp -- device helpers of the block-scaled 8-bit float (F8)
// kernels: e4m3 codes, power-of-two scales, the gate's activation, and the
// gfx950 matrix instruction.
#pragma once

#include "qg_common.hpp"
#include "qg_launch.hpp"

namespace qg {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__host__ __device__ constexpr int f8_blocks(int x) { return x / 128 + (x % 128 != 0); }   // of 128
__host__ __device__ constexpr int f8_pad16(int x) { return (x + 15) / 16 * 16; }

// The scale of a block whose largest magnitude has the bits `top` (0 ..
// 0x7FFFFFFF): 2^e with the smallest e >= -126 for which top / 2^e <= 448, 1
// for zeros, NaN if a NaN or an infinity is among them.  448 = 1.75 * 2^8, so e
// is top's exponent less 8, and one more for a mantissa above 1.75.  A power
// of two loses nothing against top / 448: e4m3's steps are relative, and the
// 17 binades below 448 stay as they are but for one.  It makes x / 2^e exact,
// so a code is x's nearest whichever precision computes it.
struct F8Scale {
  float scale;
  bool bad;
  __device__ __forceinline__ explicit F8Scale(int top) {
    int e = max((top >> 23) - 135 + ((top & 0x7FFFFF) > 0x600000 ? 1 : 0), -126);
    e = top == 0 ? 0 : e;
    bad = top >= 0x7F800000;
    scale = bad ? __builtin_nanf("") : __int_as_float((e + 127) << 23);
  }
};
// Whether a scale is a normal power of two, as the matrix instruction's own are.
__device__ __forceinline__ bool f8_power(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x807FFFFFu) == 0 && u - 0x800000u < 0x7F000000u;
}
__device__ __forceinline__ int f8_top(int top, float v) { return max(top, __float_as_int(v) & 0x7FFFFFFF); }

// Four values / scale (a power of two; at most 448 then) -> codes, rounded to nearest even.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d, float scale) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  const s16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(s16x2{0, 0}, a, b, scale, false);
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, c, d, scale, true));
}
// Two codes of a word (its low or high half) -> values, exact.
template <bool HIGH>
__device__ __forceinline__ f32x2 f8_unpack2(uint32_t w) {
  const auto v = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), HIGH);
  return f32x2{v[0], v[1]};
}

// The gate: act(g) = g s with s = sigmoid(y), y = g (silu) or
// 2 sqrt(2 / pi) (g + 0.044715 g^3) (gelu, in its tanh form: (1 + tanh(y / 2)) / 2
// = s).  The sigmoid keeps its relative precision where 1 + tanh cancels, down to 2^-126;
// below (y < -87.3) the reciprocal gives 0, an error of g 2^-126 at most.
// act'(g) = s + g s (1 - s) y'; where s (1 - s) is 0 the second term is, though
// y' may be infinite.
constexpr float kGelu = 1.5957691216057308f;
__device__ __forceinline__ float f8_sigmoid(float y) { return __builtin_amdgcn_rcpf(1.0f + __expf(-y)); }
__device__ __forceinline__ float f8_gate_arg(float g, int act) {
  return act == QG_GATE_GELU ? kGelu * (g + 0.044715f * (g * g * g)) : g;
}
__device__ __forceinline__ float f8_gate(float g, int act) { return g * f8_sigmoid(f8_gate_arg(g, act)); }
__device__ __forceinline__ float f8_gate_slope(float g, int act, float &value) {
  const float s = f8_sigmoid(f8_gate_arg(g, act)), t = s * (1.0f - s);
  const float dy = act == QG_GATE_GELU ? kGelu * (1.0f + 0.134145f * (g * g)) : 1.0f;
  value = g * s;
  return t > 0.0f ? s + g * t * dy : s;
}

// 16 x 16 x 128 product of two e4m3 fragments on zero: lane (nl, q) holds row (or
// column) nl, 32 of the 128 k.
__device__ __forceinline__ f32x4 f8_mfma(i32x8 a, i32x8 b) {
  constexpr int kFP8 = 0;   // operand format code
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, kFP8, kFP8, 0, 0, 0, 0);
}
// The same on c, each lane's value of its row scaled by 2^(e - 127), e of 1 .. 254 in
// the low byte.
__device__ __forceinline__ f32x4 f8_mfma_powers(i32x8 a, i32x8 b, f32x4 c, uint32_t ea, uint32_t eb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, static_cast<int>(ea), 0, static_cast<int>(eb));
}
__device__ __forceinline__ i32x8 f8_frag(u32x4 lo, u32x4 hi) {
  return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
               static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
}

}  // namespace qg
