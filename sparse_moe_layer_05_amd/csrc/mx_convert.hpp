// Conversion to and from the OCP microscaling formats (MX v1.0) on gfx950.
//
// A block of 32 consecutive elements v_i shares the scale X = 2^(floor(log2 max|v_i|) - emax),
// emax = 2 (E2M1) or 8 (E4M3), stored as the E8M0 code log2(X) + 127 (clamped at 0; 0 for a zero
// block); the elements are v_i / X rounded to nearest even and saturated. floor(log2) of a normal
// fp32 is its exponent field, and a subnormal maximum clamps to code 0 either way, so the code is
// max(0, field(max) - emax). v_i / X is a multiplication by a power of two: exact, except where
// the quotient is far below the smallest element and rounds to zero all the same.
// A block that holds a NaN or an infinity gets scale code 255 (NaN) and zero elements.
//
// A lane takes 16 bytes at a time, so a block is shared by four lanes (bf16) or eight (fp32); its
// maximum comes from two or three lane permutations, no LDS. Rows are contiguous, so a matrix is
// one run of blocks. Each thread takes kIter such loads, all in flight together. HBM bound: 29696 x
// 2688 fp32 to MXFP4 (362 MB) 82 to 90 us, back 67 to 72 us (4.0 to 5.4 TB/s; a large copy 4.8).
// Included once, by backward.hip: these kernels are part of that object, so that the library stays the
// objects that its parts are linked from elsewhere (host code under the sanitizers).
#pragma once

#include "common.hpp"
#include "mx.hpp"

namespace moe {
namespace {
namespace mx_convert {

constexpr int kIter = 4;      // groups of elements per thread
constexpr int kThreads = 256;

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Largest value over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  // quad_perm [1, 0, 3, 2], then [2, 3, 0, 1]
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
}

// 2^(code - 127) for code 0 .. 254.
__device__ __forceinline__ float e8m0(uint32_t code) {
  return __uint_as_float(code ? code << 23 : 0x00400000u);
}

// Elements a lane takes at once: one 16-byte load.
template <Elt XT> constexpr int kEpt = XT == Elt::BF16 ? 8 : 4;
template <Elt XT>
__device__ __forceinline__ void unpack(uint4 q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (XT == Elt::BF16) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    } else {
      v[j] = __uint_as_float(w[j]);
    }
  }
}

template <Elt XT, Elt FMT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const uint4* __restrict__ x,
                                                               int64_t ng,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  constexpr int E = kEpt<XT>, L = kMxBlockElts / E;   // lanes of a block: 4 or 8
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kIter) + threadIdx.x;
  uint4 in[kIter];
#pragma unroll
  for (int q = 0; q < kIter; ++q) {
    const int64_t g = first + q * kThreads;
    in[q] = g < ng ? x[g] : make_uint4(0, 0, 0, 0);   // blocks are whole: so are their lanes
  }
#pragma unroll
  for (int q = 0; q < kIter; ++q) {
    const int64_t g = first + q * kThreads;
    float v[E];
    unpack<XT>(in[q], v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    m = quad_max(m);
    if constexpr (L == 8)   // row_half_mirror: lane i of eight meets lane 7 - i
      m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));
    const bool bad = m >= 0x7F800000u;
    constexpr int emax = FMT == Elt::MXFP4 ? 2 : 8;
    const int code = max(0, (int)(m >> 23) - emax);
    const float inv = bad ? 0.f : e8m0(254 - code);
    float e[E];
#pragma unroll
    for (int j = 0; j < E; ++j) e[j] = bad ? 0.f : v[j] * inv;
    uint32_t c[2] = {0, 0};
    if constexpr (FMT == Elt::MXFP4) {   // rounds to nearest even and saturates at 6
      c[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[0], e[0], e[1], 1.f, 0);
      c[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[0], e[2], e[3], 1.f, 1);
      if constexpr (E == 8) {
        c[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[0], e[4], e[5], 1.f, 2);
        c[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[0], e[6], e[7], 1.f, 3);
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) e[j] = fminf(fmaxf(e[j], -448.f), 448.f);
#pragma unroll
      for (int j = 0; j < E / 4; ++j)
        c[j] = cvt_fp8x2(e[4 * j], e[4 * j + 1]) | cvt_fp8x2(e[4 * j + 2], e[4 * j + 3]) << 16;
    }
    if (g < ng) {
      constexpr int B = FMT == Elt::MXFP4 ? E / 2 : E;   // bytes of this lane's codes
      if constexpr (B == 2) *(uint16_t*)(codes + g * 2) = (uint16_t)c[0];
      else if constexpr (B == 4) *(uint32_t*)(codes + g * 4) = c[0];
      else *(uint2*)(codes + g * 8) = make_uint2(c[0], c[1]);
      if ((threadIdx.x & (L - 1)) == 0) scales[g / L] = bad ? 255 : (uint8_t)code;
    }
  }
}

template <Elt FMT, Elt XT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales,
                                                                 int64_t n8, void* __restrict__ x) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kIter) + threadIdx.x;
  uint2 c[kIter];
  uint32_t sc[kIter];
#pragma unroll
  for (int q = 0; q < kIter; ++q) {
    const int64_t g = first + q * kThreads;
    if (g >= n8) continue;
    if constexpr (FMT == Elt::MXFP4) c[q] = make_uint2(*(const uint32_t*)(codes + g * 4), 0);
    else c[q] = *(const uint2*)(codes + g * 8);
    sc[q] = scales[g >> 2];
  }
#pragma unroll
  for (int q = 0; q < kIter; ++q) {
    const int64_t g = first + q * kThreads;
    if (g >= n8) break;
    const float s = sc[q] == 255 ? __uint_as_float(0x7FC00000u) : e8m0(sc[q]);
    f32x2_t v[4];
    if constexpr (FMT == Elt::MXFP4) {
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q].x, 1.f, 0);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q].x, 1.f, 1);
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q].x, 1.f, 2);
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q].x, 1.f, 3);
    } else {
      v[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[q].x, false);
      v[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[q].x, true);
      v[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[q].y, false);
      v[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[q].y, true);
    }
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v[j >> 1][j & 1] * s;
    if constexpr (XT == Elt::BF16) {
      uint32_t w[4];   // exact for every normal bf16
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(o[2 * j], o[2 * j + 1]);
      *(uint4*)((uint16_t*)x + g * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float* d = (float*)x + g * 8;
      *(float4*)d = make_float4(o[0], o[1], o[2], o[3]);
      *(float4*)(d + 4) = make_float4(o[4], o[5], o[6], o[7]);
    }
  }
}

dim3 grid_of(int64_t groups) {
  return dim3((unsigned)((groups + kThreads * kIter - 1) / (kThreads * kIter)));
}

}  // namespace mx_convert
}  // namespace

using namespace mx_convert;

hipError_t launch_mx_quantize(const void* x, Elt xt, int64_t n, Elt fmt, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
  if (n <= 0) return hipSuccess;
  if (n % kMxBlockElts || n > kMxMaxElts) return hipErrorInvalidValue;
#define MOE_MXQ(X, F)                                                                     \
  hipLaunchKernelGGL((mx_quantize_kernel<X, F>), grid_of(n / kEpt<X>), dim3(kThreads), 0, s, \
                     (const uint4*)x, n / kEpt<X>, codes, scales)
  const bool f4 = fmt == Elt::MXFP4;
  if (xt == Elt::BF16) {
    if (f4) MOE_MXQ(Elt::BF16, Elt::MXFP4); else MOE_MXQ(Elt::BF16, Elt::MXFP8);
  } else {
    if (f4) MOE_MXQ(Elt::F32, Elt::MXFP4); else MOE_MXQ(Elt::F32, Elt::MXFP8);
  }
#undef MOE_MXQ
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, Elt fmt, int64_t n,
                                void* x, Elt xt, hipStream_t s) {
  if (n <= 0) return hipSuccess;
  if (n % kMxBlockElts || n > kMxMaxElts) return hipErrorInvalidValue;
  const int64_t n8 = n / 8;
#define MOE_MXD(F, X)                                                                             \
  hipLaunchKernelGGL((mx_dequantize_kernel<F, X>), grid_of(n8), dim3(kThreads), 0, s, codes,      \
                     scales, n8, x)
  const bool f4 = fmt == Elt::MXFP4;
  if (xt == Elt::BF16) {
    if (f4) MOE_MXD(Elt::MXFP4, Elt::BF16); else MOE_MXD(Elt::MXFP8, Elt::BF16);
  } else {
    if (f4) MOE_MXD(Elt::MXFP4, Elt::F32); else MOE_MXD(Elt::MXFP8, Elt::F32);
  }
#undef MOE_MXD
  return hipGetLastError();
}

}  // namespace moe
