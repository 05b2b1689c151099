// Token rows into expert order and back, with weights, and the gradients of both (gfx950).
//
//   spread      out[pos[t, j]] = w[t, j] in[t]                 (sort; its inverse's gradient)
//   gather      out[t] = add[t] + sum_j w[t, j] in[pos[t, j]]  (back; the sort's gradient)
//   dots        dw[t, j] = <a[t], b[pos[t, j]]>                (gradient of the weights, with either)
//
// All are bound by HBM: a token's row is read or written once, its k rows once each. A wave takes
// 512 columns of one token, eight elements a lane, and walks the token's k rows.
// Included once, by routing.hip.
#pragma once

#include "common.hpp"
#include "row8.hpp"
#include "token_rows.hpp"

namespace moe {
namespace {
namespace token_rows {

constexpr int kSeg = 8 * kWave;   // columns of a wave
constexpr int kBatch = 8;         // rows in flight

// A token's k positions and weights, one a lane; position -1 where the pair is dropped.
struct Pairs {
  int pos;
  float w;
};
__device__ __forceinline__ Pairs load_pairs(const TokenRows& p, int t, int lane) {
  Pairs q{-1, 0.f};
  if (lane < p.k) {
    const int64_t i = (int64_t)t * p.k + lane;
    const int r = p.pos[i];
    q.pos = (unsigned)r < (unsigned)p.n_rows ? r : -1;
    q.w = p.weights ? p.weights[i] : 1.f;
  }
  return q;
}
__device__ __forceinline__ int pos_of(const Pairs& q, int j) {
  return __builtin_amdgcn_readlane(q.pos, j);
}
__device__ __forceinline__ float weight_of(const Pairs& q, int j) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(q.w), j));
}

template <Elt T, bool WEIGHTED>
__global__ __launch_bounds__(256) void spread_kernel(TokenRows p, const void* __restrict__ in,
                                                     void* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int nseg = (p.D + kSeg - 1) / kSeg;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t = (int)(unit / nseg);
  if (t >= p.T) return;
  const int c = (int)(unit - (int64_t)t * nseg) * kSeg + lane * 8;
  const Pairs pr = load_pairs(p, t, lane);
  const bool in_row = c < p.D;
  Raw8<T> r = zero8<T>();
  if (in_row) r = load8<T>(in, (int64_t)t * p.D + c);
  float v[8];
  if constexpr (WEIGHTED) unpack8<T>(r, v);
  for (int j = 0; j < p.k; ++j) {
    const int row = pos_of(pr, j);
    if (row < 0) continue;
    if constexpr (WEIGHTED) {
      const float w = weight_of(pr, j);
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = w * v[i];
      r = pack8<T>(u);
    }
    if (in_row) store8<T>(out, (int64_t)row * p.D + c, r);
  }
}

template <Elt IN, Elt OUT>
__global__ __launch_bounds__(256) void gather_kernel(TokenRows p, const void* __restrict__ in,
                                                     const void* add, void* out) {
  const int lane = threadIdx.x & 63;
  const int nseg = (p.D + kSeg - 1) / kSeg;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t = (int)(unit / nseg);
  if (t >= p.T) return;
  const int c = (int)(unit - (int64_t)t * nseg) * kSeg + lane * 8;
  const Pairs pr = load_pairs(p, t, lane);
  if (c >= p.D) return;
  float acc[8] = {};
  if (add) unpack8<OUT>(load8<OUT>(add, (int64_t)t * p.D + c), acc);
  for (int j0 = 0; j0 < p.k; j0 += kBatch) {
    Raw8<IN> r[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int row = j0 + b < p.k ? pos_of(pr, j0 + b) : -1;
      if (row >= 0) r[b] = load8<IN>(in, (int64_t)row * p.D + c);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (j0 + b >= p.k || pos_of(pr, j0 + b) < 0) continue;
      const float w = weight_of(pr, j0 + b);
      float v[8];
      unpack8<IN>(r[b], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
    }
  }
  store8<OUT>(out, (int64_t)t * p.D + c, pack8<OUT>(acc));
}

constexpr int kDotWaves = 8;   // waves of a workgroup that shares a token's dot products

// A workgroup per token; wave v takes the columns v * 512 + n * waves * 512. SPREAD: writes
// out[pos] = w a[t] (a: IN, rows and out: ROWS); else out[t] = sum_j w rows[pos] (rows and a: ROWS,
// out: IN). Dots of a wave go through LDS and are added in wave order.
template <Elt IN, Elt ROWS, bool SPREAD>
__global__ __launch_bounds__(kDotWaves * 64) void dot_kernel(TokenRows p, const void* a,
                                                             const void* rows, void* out,
                                                             float* __restrict__ dweights) {
  __shared__ float part[kDotWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int waves = blockDim.x >> 6;
  const int t = blockIdx.x;
  const Pairs pr = load_pairs(p, t, lane);
  float dot = 0.f;   // of pair `lane`
  for (int c0 = wave * kSeg; c0 < p.D; c0 += waves * kSeg) {
    const int c = c0 + lane * 8;
    const bool in_row = c < p.D;
    constexpr Elt AT = SPREAD ? IN : ROWS;
    float av[8] = {}, acc[8] = {};
    if (in_row) unpack8<AT>(load8<AT>(a, (int64_t)t * p.D + c), av);
    for (int j0 = 0; j0 < p.k; j0 += kBatch) {
      Raw8<ROWS> r[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int row = j0 + b < p.k ? pos_of(pr, j0 + b) : -1;
        r[b] = zero8<ROWS>();
        if (row >= 0 && in_row) r[b] = load8<ROWS>(rows, (int64_t)row * p.D + c);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int row = j0 + b < p.k ? pos_of(pr, j0 + b) : -1;
        if (row < 0) continue;
        const float w = weight_of(pr, j0 + b);
        float v[8], d = 0.f;
        unpack8<ROWS>(r[b], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) d = fmaf(av[i], v[i], d);
        d = wave_sum(in_row ? d : 0.f);
        if (lane == j0 + b) dot += d;
        if constexpr (SPREAD) {
          float u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = w * av[i];
          if (in_row) store8<ROWS>(out, (int64_t)row * p.D + c, pack8<ROWS>(u));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
        }
      }
    }
    if constexpr (!SPREAD)
      if (in_row) store8<IN>(out, (int64_t)t * p.D + c, pack8<IN>(acc));
  }
  part[wave][lane] = dot;
  __syncthreads();
  if (wave == 0 && lane < p.k) {
    float d = 0.f;
    for (int v = 0; v < waves; ++v) d += part[v][lane];
    dweights[(int64_t)t * p.k + lane] = pr.pos >= 0 ? d : 0.f;
  }
}

dim3 seg_grid(const TokenRows& p) {
  const int64_t units = (int64_t)p.T * ((p.D + kSeg - 1) / kSeg);
  return dim3((unsigned)((units + 3) / 4));
}
dim3 dot_block(int D) {
  const int n = (D + kSeg - 1) / kSeg;
  return dim3(64 * (n < kDotWaves ? n : kDotWaves));
}

}  // namespace token_rows
}  // namespace

using namespace token_rows;

hipError_t launch_spread_rows(const TokenRows& p, Elt t, const void* in, void* out, hipStream_t s) {
  if (p.T <= 0) return hipSuccess;
#define MOE_SPREAD(X, W) \
  hipLaunchKernelGGL((spread_kernel<X, W>), seg_grid(p), dim3(256), 0, s, p, in, out)
  if (t == Elt::BF16) {
    if (p.weights) MOE_SPREAD(Elt::BF16, true); else MOE_SPREAD(Elt::BF16, false);
  } else {
    if (p.weights) MOE_SPREAD(Elt::F32, true); else MOE_SPREAD(Elt::F32, false);
  }
#undef MOE_SPREAD
  return hipGetLastError();
}

hipError_t launch_gather_rows(const TokenRows& p, Elt in_t, const void* in, const void* add,
                              Elt out_t, void* out, const void* other, float* dweights,
                              hipStream_t s) {
  if (p.T <= 0) return hipSuccess;
  const bool bi = in_t == Elt::BF16, bo = out_t == Elt::BF16;
  if (dweights) {
#define MOE_GATHER_DOT(O, I)                                                                     \
  hipLaunchKernelGGL((dot_kernel<O, I, false>), dim3(p.T), dot_block(p.D), 0, s, p, other, in, out, \
                     dweights)
    if (bi) {
      if (bo) MOE_GATHER_DOT(Elt::BF16, Elt::BF16); else MOE_GATHER_DOT(Elt::F32, Elt::BF16);
    } else {
      if (bo) MOE_GATHER_DOT(Elt::BF16, Elt::F32); else MOE_GATHER_DOT(Elt::F32, Elt::F32);
    }
#undef MOE_GATHER_DOT
    return hipGetLastError();
  }
#define MOE_GATHER(I, O) \
  hipLaunchKernelGGL((gather_kernel<I, O>), seg_grid(p), dim3(256), 0, s, p, in, add, out)
  if (bi) {
    if (bo) MOE_GATHER(Elt::BF16, Elt::BF16); else MOE_GATHER(Elt::BF16, Elt::F32);
  } else {
    if (bo) MOE_GATHER(Elt::F32, Elt::BF16); else MOE_GATHER(Elt::F32, Elt::F32);
  }
#undef MOE_GATHER
  return hipGetLastError();
}

hipError_t launch_spread_dot(const TokenRows& p, Elt in_t, const void* in, Elt rows_t,
                             const void* rows, void* out, float* dweights, hipStream_t s) {
  if (p.T <= 0) return hipSuccess;
#define MOE_SPREAD_DOT(I, R)                                                                      \
  hipLaunchKernelGGL((dot_kernel<I, R, true>), dim3(p.T), dot_block(p.D), 0, s, p, in, rows, out, \
                     dweights)
  if (in_t == Elt::BF16) {
    if (rows_t == Elt::BF16) MOE_SPREAD_DOT(Elt::BF16, Elt::BF16);
    else MOE_SPREAD_DOT(Elt::BF16, Elt::F32);
  } else {
    if (rows_t == Elt::BF16) MOE_SPREAD_DOT(Elt::F32, Elt::BF16);
    else MOE_SPREAD_DOT(Elt::F32, Elt::F32);
  }
#undef MOE_SPREAD_DOT
  return hipGetLastError();
}

}  // namespace moe
