// Device helpers shared by the 4-bit products' kernels.
#pragma once

#include "q4_internal.h"
#include "q8_device.h"

namespace dmuon {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 codes' words as a matrix operand: 4-bit operands take the first four.
__device__ __forceinline__ i32x8 codes_operand(const u32x4 &w) {
  return i32x8{static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w), 0, 0, 0, 0};
}

// acc += 16 outputs by 16 rows over 128 codes: a lane's 32 codes of each operand
// (one block of the format) and the words whose bytes IB and IA are their scales.
template <int IB, int IA>
__device__ __forceinline__ f32x4 q4_product(const u32x4 &b, uint32_t sb, const u32x4 &a, uint32_t sa, f32x4 acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes_operand(b), codes_operand(a), acc, 4, 4, IB,
                                                          static_cast<int>(sb), IA, static_cast<int>(sa));
}

// 2^(byte - 128) as fp32, half of a scale byte's scale; NaN for kQ4Nan.
__device__ __forceinline__ float q4_half_scale(uint32_t byte) {
  return __uint_as_float(byte == kQ4Nan ? 0x7fc00000u : (byte - 1) << 23);
}

// Eight codes (a word) times a power of two as bf16, exactly.
__device__ __forceinline__ bf16x8 q4_expand8(uint32_t w, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

}  // namespace dmuon
