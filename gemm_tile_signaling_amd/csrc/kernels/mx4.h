// Vector types and the 4-bit (MX) format's conversions, shared by the kernels
// of the 4-bit operators and the mixture-of-experts layer.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fo {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

// Scale byte of a block whose largest magnitude has the fp32 bits `top`:
// exponent field - 2, at least 0; 255 (NaN) for an infinity or a NaN.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255 ? 255 : e > 2 ? e - 2 : 0;
}

// 2^(byte - 127) as the scaled conversions read it (they take the exponent
// field alone, 255 as NaN; byte 0 is 2^-127, a denormal in fp32).
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

template <typename T>
__device__ __forceinline__ u32x2 pack4(f32x4 v);
template <>
__device__ __forceinline__ u32x2 pack4<__bf16>(f32x4 v) {
  return __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}
template <>
__device__ __forceinline__ u32x2 pack4<_Float16>(f32x4 v) {
  return __builtin_bit_cast(u32x2, __builtin_convertvector(v, f16x4));
}

// One scaled MFMA on 4-bit operands: lane l holds 32 values of row l % 32 (l % 16)
// of each operand and their scale in byte SA (SB) of sa (sb).
template <int SA, int SB>
__device__ __forceinline__ f32x16 mx4_mma32(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x16 c) {
  const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, SA, (int)sa, SB, (int)sb);
}
template <int SA, int SB>
__device__ __forceinline__ f32x4 mx4_mma16(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c) {
  const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, SA, (int)sa, SB, (int)sb);
}

}  // namespace fo
