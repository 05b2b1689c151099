// Device-side helpers shared by the gfx950 kernels of the MoE layer library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8_t;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
typedef __attribute__((__vector_size__(8 * sizeof(int)))) int i32x8_t;
typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4_t;

constexpr int kWave = 64;
constexpr int kXcds = 8;  // MI355X: 8 accelerator complex dies, 32 CUs each, one L2 per die

// bf16 <-> fp32. bf16 is the upper half of a binary32; the narrowing is the hardware's: to nearest
// even, subnormals kept, NaN stays NaN. (As integer arithmetic, u + 0x7FFF + bit 16, it gives the same
// for all 2^32 patterns but NaN, of which one of all ones carries into the sign and becomes 0.)
__device__ __forceinline__ float bf16_bits_to_f32(uint32_t u16) {
  return __uint_as_float(u16 << 16);
}
// Two fp32 -> packed bf16x2 (lo in bits 0..15).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float f) {
  return pack_bf16x2(f, f) & 0xFFFFu;
}

// Two fp32 -> two OCP e4m3 codes (round to nearest even) in the low 16 bits.
__device__ __forceinline__ uint32_t cvt_fp8x2(float a, float b) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

// How a row whose largest magnitude is m meets 8- and 4-bit experts: codes e4m3(v * up), values
// code * down; up = 448 / m and down = m / 448, or 1 and 1 for a row of zeros. Below m = 1.3e-36
// 448 / m is past fp32 (a zero times it would be NaN): 2^127 and 2^-127 there, codes up to 224, and
// the smallest bf16 value, 2^-133, still has a normal code.
struct RowScale {
  float up, down;
};
__device__ __forceinline__ RowScale row_scale_e4m3(float m) {
  if (!(m > 0.f)) return {1.f, 1.f};
  const float up = 448.f / m;
  if (up == __builtin_inff()) return {0x1p127f, 0x1p-127f};
  return {up, m / 448.f};
}

// relu(a)^2; NaN stays NaN (a > 0 ? a * a : 0 would make it 0).
__device__ __forceinline__ float sqrelu(float a) { return a <= 0.f ? 0.f : a * a; }

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Hardware hands workgroup b to die b % 8. Remap so each die walks one contiguous range of
// logical tiles: neighbouring tiles (which share weight or activation panels) then share an L2.
// nblk must be a multiple of 8.
__device__ __forceinline__ int xcd_logical_block(int b, int nblk) {
  return (b % kXcds) * (nblk / kXcds) + b / kXcds;
}

}  // namespace moe
