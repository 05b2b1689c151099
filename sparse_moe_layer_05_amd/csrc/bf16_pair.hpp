// Values kept as the sum of two bf16.
#pragma once

#include "common.hpp"

namespace moe {

// What rounding two fp32 to the packed bf16 `hi` left over, packed too: v = hi + rest up to 2^-17 of
// v. Nothing where hi is infinite (inf - inf would make the pair's sum NaN).
__device__ __forceinline__ uint32_t bf16x2_rest(float a, float b, uint32_t hi) {
  const float x = bf16_bits_to_f32(hi & 0xFFFF), y = bf16_bits_to_f32(hi >> 16);
  return pack_bf16x2(__builtin_isinf(x) ? 0.f : a - x, __builtin_isinf(y) ? 0.f : b - y);
}

}  // namespace moe
