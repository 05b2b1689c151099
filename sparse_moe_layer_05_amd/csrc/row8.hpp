// Rows of bf16 or fp32 values taken eight elements at a time (one 16-byte load or two), and sums
// over the lanes that hold a row.
#pragma once

#include "common.hpp"
#include "gemm.hpp"

namespace moe {

// Eight consecutive elements as they lie in memory.
template <Elt T> struct Raw8;
template <> struct Raw8<Elt::BF16> { uint4 q; };
template <> struct Raw8<Elt::F32> { float4 a, b; };

template <Elt T>
__device__ __forceinline__ Raw8<T> load8(const void* p, int64_t i) {
  if constexpr (T == Elt::BF16) {
    return {*(const uint4*)((const uint16_t*)p + i)};
  } else {
    return {*(const float4*)((const float*)p + i), *(const float4*)((const float*)p + i + 4)};
  }
}

template <Elt T>
__device__ __forceinline__ Raw8<T> zero8() {
  if constexpr (T == Elt::BF16) return {make_uint4(0, 0, 0, 0)};
  else return {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
}

template <Elt T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&v)[8]) {
  if constexpr (T == Elt::BF16) {
    const uint32_t w[4] = {r.q.x, r.q.y, r.q.z, r.q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
  }
}

// Some rows of n elements as a buffer of their own: elements past their end, and every element of
// absent rows, load as zeros and store nothing, so that lanes need no branch.
constexpr uint32_t kAway = 1u << 29;   // an element past the end of any buffer
template <Elt T>
struct RowBuffer {
  static constexpr uint32_t kElt = T == Elt::BF16 ? 2 : 4;
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  __amdgpu_buffer_rsrc_t r;
  // rows [row, row + rows); none if rows <= 0 or base is nullptr
  __device__ __forceinline__ RowBuffer(const void* base, int64_t row, int rows, int n)
      : r(__builtin_amdgcn_make_buffer_rsrc((char*)base + row * n * kElt, (short)0,
                                            base && rows > 0 ? (int)(rows * n * kElt) : 0,
                                            0x00020000)) {}
  // LAST: the lines are marked as the first to leave the caches
  template <bool LAST = false>
  __device__ __forceinline__ Raw8<T> load(uint32_t col) const {
    constexpr int kAux = LAST ? 2 : 0;
    Raw8<T> out;
    if constexpr (T == Elt::BF16) {
      out.q = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, col * kElt, 0, kAux));
    } else {
      out.a = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(r, col * kElt, 0, kAux));
      out.b = __builtin_bit_cast(float4,
                                 __builtin_amdgcn_raw_buffer_load_b128(r, col * kElt + 16, 0, kAux));
    }
    return out;
  }
  template <int N>
  __device__ __forceinline__ void load(const uint32_t (&col)[N], Raw8<T> (&out)[N], bool last) const {
    if (last) {   // the same in every lane
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = load<true>(col[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = load<false>(col[i]);
    }
  }
  template <bool LAST = false>
  __device__ __forceinline__ void store(uint32_t col, const Raw8<T>& v) const {
    constexpr int kAux = LAST ? 2 : 0;
    if constexpr (T == Elt::BF16) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v.q), r, col * kElt, 0, kAux);
    } else {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v.a), r, col * kElt, 0, kAux);
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v.b), r, col * kElt + 16, 0,
                                             kAux);
    }
  }
};

// Hides from the compiler that r was unpacked before, so that a later pass over a row unpacks it again
// instead of keeping both forms in registers.
__device__ __forceinline__ void forget(Raw8<Elt::BF16>& r) {
  asm volatile("" : "+v"(r.q.x), "+v"(r.q.y), "+v"(r.q.z), "+v"(r.q.w));
}
__device__ __forceinline__ void forget(Raw8<Elt::F32>&) {}

template <Elt T>
__device__ __forceinline__ Raw8<T> pack8(const float (&v)[8]) {
  if constexpr (T == Elt::BF16)
    return {make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]))};
  else
    return {make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7])};
}

template <Elt T>
__device__ __forceinline__ void store8(void* p, int64_t i, const Raw8<T>& r) {
  if constexpr (T == Elt::BF16) {
    *(uint4*)((uint16_t*)p + i) = r.q;
  } else {
    *(float4*)((float*)p + i) = r.a;
    *(float4*)((float*)p + i + 4) = r.b;
  }
}

// Sum over the 64 lanes of a wave, in every lane: rows of 16 lanes by shifts of 1, 2, 4 and 8, then
// the rows' last lanes passed on; lane 63 ends with the total (a lane without a source adds 0).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);   // row_shr:1
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);   // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);   // row_bcast:31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// Sum over the first 16 lanes, in every lane.
__device__ __forceinline__ float row16_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 15));
}
// Sum over aligned groups of 8, 16 or 32 lanes, in every lane: lane i meets i ^ 1, i ^ 2, then 7 - i
// and 15 - i of its eight and sixteen, whose sums are those of the other half.
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
  static_assert(LANES == 8 || LANES == 16 || LANES == 32);
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true));
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true));
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true));
  if constexpr (LANES >= 16)
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true));
  if constexpr (LANES == 32) v += __shfl_xor(v, 16);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

}  // namespace moe
