// The norms before and after a block, fused with its gate, its residual and the next block's norm,
// and their gradients (gfx950).
//
//   n(v) = v / sqrt(mean(v^2) + eps)
//   y = x + scale a z, z = n(f) w or f w, a = gate or sigmoid(gate) or 1;  h = n(y) w_next
//   gradient of n at v against g:  r (g - n(v) mean(g n(v))), r = 1 / sqrt(mean(v^2) + eps)
//
// Bound by HBM: each row is read once and held in registers between its sums and its result, so
// neither pass keeps statistics for the other. A row is held by 64 lanes (up to 2048 columns) or by
// a workgroup of 128 to 512, at most 32 columns a lane. y is rounded before the next norm reads it:
// the backward pass, which has y as it is stored, then differentiates the same function.
// Sums run in fp32; where a sum of squares passes fp32 (values beyond 1e18) it is taken again in
// fp64, a branch that no ordinary row takes.
// Included once, by backward.hip.
#pragma once

#include "block_norm.hpp"
#include "common.hpp"
#include "row8.hpp"

#include <type_traits>

namespace moe {
namespace {
namespace block_norm {

// Sums of N values over the TPR lanes of a row (waves of a workgroup add through LDS in order).
template <int TPR, int N, typename F>
__device__ __forceinline__ void row_sum(F (&v)[N], double* lds) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    F* red = (F*)lds;
    const int wave = threadIdx.x >> 6;
    __syncthreads();   // the last sums' reads are done
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      F s = red[i];
#pragma unroll
      for (int q = 1; q < W; ++q) s += red[q * N + i];
      v[i] = s;
    }
  }
}

__device__ __forceinline__ void load_w8(const void* w, Elt t, int c, float (&v)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
  } else if (t == Elt::BF16) {
    unpack8<Elt::BF16>(load8<Elt::BF16>(w, c), v);
  } else {
    unpack8<Elt::F32>(load8<Elt::F32>(w, c), v);
  }
}

// A gate's value and what its derivative multiplies by: sigmoid(q) and 1 - sigmoid(q), neither from
// the other (1 - a would lose all of a small one); without a sigmoid q and 1.
struct GateValue {
  float a, rest;
};
__device__ __forceinline__ GateValue gate_value(float q, bool sigmoid) {
  if (!sigmoid) return {q, 1.f};
  const float e = expf(-fabsf(q)), inv = 1.f / (1.f + e);
  return q < 0.f ? GateValue{e * inv, inv} : GateValue{inv, e * inv};
}

__device__ __forceinline__ float inv_rms(float ss, int H, float eps) {
  return 1.f / sqrtf(ss / (float)H + eps);
}
__device__ __forceinline__ bool too_big(float s) { return fabsf(s) == __builtin_inff(); }

// 1 / rms of the row held in v; ss: its fp32 sum of squares.
template <int TPR, int NC>
__device__ __forceinline__ float row_inv_rms(const float (&v)[NC][8], float ss, int H, float eps,
                                             double* lds) {
  if (__builtin_expect(too_big(ss), 0)) {   // the same in every lane of the row
    double d[1] = {0.0};
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) d[0] += (double)v[i][e] * v[i][e];
    row_sum<TPR, 1>(d, lds);
    return (float)(1.0 / sqrt(d[0] / H + eps));
  }
  return inv_rms(ss, H, eps);
}

template <int TPR> constexpr int kThreadsOf = TPR < 256 ? (TPR == 64 ? 256 : TPR) : TPR;
template <int TPR> constexpr int kRowsOf = kThreadsOf<TPR> / TPR;

template <Elt T, int TPR, int NC, bool RES>
__global__ __launch_bounds__(kThreadsOf<TPR>) void block_forward_kernel(BlockShape b,
                                                                        BlockForward p) {
  __shared__ double lds[TPR > 64 ? TPR / 64 : 1];
  const int lane = threadIdx.x % TPR;
  const int row = blockIdx.x * kRowsOf<TPR> + threadIdx.x / TPR;
  if (row >= b.T) return;   // whole waves, and workgroups where a row has a barrier
  const int64_t base = (int64_t)row * b.H;
  int col[NC];
  bool ok[NC];
  Raw8<T> xr[NC], fr[NC], gr[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    col[i] = (lane + i * TPR) * 8;
    ok[i] = col[i] < b.H;
    xr[i] = fr[i] = gr[i] = zero8<T>();
    if (!ok[i]) continue;
    xr[i] = load8<T>(p.x, base + col[i]);
    if constexpr (RES) {
      fr[i] = load8<T>(p.f, base + col[i]);
      if (b.gate_kind == Gate::Element) gr[i] = load8<T>(p.gate, base + col[i]);
    }
  }
  float v[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) unpack8<T>(xr[i], v[i]);
  if constexpr (RES) {
    float rf = 1.f;
    if (b.norm) {
      float fv[NC][8], ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        unpack8<T>(fr[i], fv[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] = fmaf(fv[i][e], fv[i][e], ss[0]);
      }
      row_sum<TPR, 1>(ss, lds);
      rf = row_inv_rms<TPR, NC>(fv, ss[0], b.H, b.eps, lds);
    }
    float at = b.scale;   // scale, times the row's gate
    if (b.gate_kind == Gate::Token) {
      const float q = ((const float*)p.gate)[row];
      at *= gate_value(q, b.sigmoid).a;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!ok[i]) continue;
      float w[8], f[8], g[8];
      load_w8(p.w, b.w_t, col[i], w);
      unpack8<T>(fr[i], f);
      unpack8<T>(gr[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float z = f[e] * rf * w[e] * at;
        if (b.gate_kind == Gate::Element) z *= gate_value(g[e], b.sigmoid).a;
        v[i][e] += z;
      }
      const Raw8<T> out = pack8<T>(v[i]);
      store8<T>(p.y, base + col[i], out);
      unpack8<T>(out, v[i]);
    }
    if (!p.h) return;
  }
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[0] = fmaf(v[i][e], v[i][e], ss[0]);
  row_sum<TPR, 1>(ss, lds);
  const float r = row_inv_rms<TPR, NC>(v, ss[0], b.H, b.eps, lds);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!ok[i]) continue;
    float w[8], o[8];
    load_w8(p.w_next, b.w_t, col[i], w);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = v[i][e] * r * w[e];
    store8<T>(p.h, base + col[i], pack8<T>(o));
  }
}

// Rows walker, walker + walkers, .. of one walker (a wave, or a workgroup where a row needs one);
// its sums of dw and dw_next over its rows go to rows `walker` of two slabs [walkers][H].
template <Elt T, Elt DH, int TPR, int NC, bool RES>
__global__ __launch_bounds__(kThreadsOf<TPR>) void block_backward_kernel(BlockShape b,
                                                                         BlockBackward p,
                                                                         int walkers,
                                                                         float* part_w,
                                                                         float* part_n) {
  __shared__ double lds[TPR > 64 ? 3 * TPR / 64 : 1];
  const int lane = threadIdx.x % TPR;
  const int walker = blockIdx.x * kRowsOf<TPR> + threadIdx.x / TPR;
  if (walker >= walkers) return;
  int col[NC];
  bool ok[NC];
  float sw[NC][8] = {}, sn[NC][8] = {};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    col[i] = (lane + i * TPR) * 8;
    ok[i] = col[i] < b.H;
  }
  for (int row = walker; row < b.T; row += walkers) {
    const int64_t base = (int64_t)row * b.H;
    Raw8<T> yr[NC], dr[NC], fr[NC], gr[NC];
    Raw8<DH> hr[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      yr[i] = dr[i] = fr[i] = gr[i] = zero8<T>();
      hr[i] = zero8<DH>();
      if (!ok[i]) continue;
      if (p.dh) {
        yr[i] = load8<T>(p.y, base + col[i]);
        hr[i] = load8<DH>(p.dh, base + col[i]);
      }
      if (p.dy) dr[i] = load8<T>(p.dy, base + col[i]);
      if constexpr (RES) {
        fr[i] = load8<T>(p.f, base + col[i]);
        if (b.gate_kind == Gate::Element) gr[i] = load8<T>(p.gate, base + col[i]);
      }
    }
    // sum y^2, sum (dh w_next) y, sum f^2
    float s[3] = {0.f, 0.f, 0.f};
    float d[NC][8];   // d, the gradient reaching y
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float y[8], h[8], w[8] = {}, f[8];
      unpack8<T>(yr[i], y);
      unpack8<DH>(hr[i], h);
      unpack8<T>(fr[i], f);
      if (p.dh && ok[i]) load_w8(p.w_next, b.w_t, col[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[i][e] = h[e] * w[e];
        s[0] = fmaf(y[e], y[e], s[0]);
        s[1] = fmaf(d[i][e], y[e], s[1]);
        s[2] = fmaf(f[e], f[e], s[2]);
      }
    }
    row_sum<TPR, 3>(s, lds);
    if (p.dh) {
      float r = inv_rms(s[0], b.H, b.eps), m = s[1] * r / (float)b.H;
      if (__builtin_expect(too_big(s[0]) || too_big(s[1]), 0)) {   // both sums again, in fp64
        double q[2] = {0.0, 0.0};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          float y[8];
          unpack8<T>(yr[i], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            q[0] += (double)y[e] * y[e];
            q[1] += (double)d[i][e] * y[e];
          }
        }
        row_sum<TPR, 2>(q, lds);
        const double rd = 1.0 / sqrt(q[0] / b.H + b.eps);
        r = (float)rd;
        m = (float)(q[1] * rd / b.H);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float y[8], h[8];
        unpack8<T>(yr[i], y);
        unpack8<DH>(hr[i], h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = y[e] * r;
          d[i][e] = r * (d[i][e] - n * m);
          sn[i][e] = fmaf(h[e], n, sn[i][e]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float dy[8];
      unpack8<T>(dr[i], dy);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[i][e] += dy[e];
      if (ok[i]) store8<T>(p.dx, base + col[i], pack8<T>(d[i]));
    }
    if constexpr (RES) {
      float rf = 1.f;
      if (b.norm) {
        rf = inv_rms(s[2], b.H, b.eps);
        if (__builtin_expect(too_big(s[2]), 0)) {
          float fv[NC][8];
#pragma unroll
          for (int i = 0; i < NC; ++i) unpack8<T>(fr[i], fv[i]);
          rf = row_inv_rms<TPR, NC>(fv, s[2], b.H, b.eps, lds);
        }
      }
      GateValue gt = {1.f, 1.f};   // the row's gate
      if (b.gate_kind == Gate::Token) gt = gate_value(((const float*)p.gate)[row], b.sigmoid);
      // sum d a w n(f): the mean in the norm's gradient and, with a = 1, the token gate's gradient
      float q[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!ok[i]) continue;
        float w[8], f[8], g[8], o[8];
        load_w8(p.w, b.w_t, col[i], w);
        unpack8<T>(fr[i], f);
        unpack8<T>(gr[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = f[e] * rf;
          const float ds = d[i][e] * b.scale;
          float a = gt.a;
          if (b.gate_kind == Gate::Element) {
            const GateValue ge = gate_value(g[e], b.sigmoid);
            a = ge.a;
            o[e] = ds * n * w[e] * ge.rest * (b.sigmoid ? a : 1.f);
          }
          const float dz = ds * a;
          sw[i][e] = fmaf(dz, n, sw[i][e]);
          d[i][e] = dz * w[e];
          // (a token's gate is taken out again: its own gradient needs the sum without it)
          q[0] = fmaf(b.gate_kind == Gate::Token ? ds * w[e] : d[i][e], n, q[0]);
        }
        if (b.gate_kind == Gate::Element && p.dgate)
          store8<T>(p.dgate, base + col[i], pack8<T>(o));
      }
      if (b.norm || b.gate_kind == Gate::Token) row_sum<TPR, 1>(q, lds);
      if (b.gate_kind == Gate::Token && lane == 0 && p.dgate)
        ((float*)p.dgate)[row] = q[0] * gt.rest * (b.sigmoid ? gt.a : 1.f);
      const float m = b.norm ? (b.gate_kind == Gate::Token ? q[0] * gt.a : q[0]) / (float)b.H : 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!ok[i]) continue;
        float f[8], o[8];
        unpack8<T>(fr[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e] = b.norm ? rf * (d[i][e] - f[e] * rf * m) : d[i][e];
        store8<T>(p.df, base + col[i], pack8<T>(o));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!ok[i]) continue;
    if (part_w) store8<Elt::F32>(part_w, (int64_t)walker * b.H + col[i], pack8<Elt::F32>(sw[i]));
    if (part_n) store8<Elt::F32>(part_n, (int64_t)walker * b.H + col[i], pack8<Elt::F32>(sn[i]));
  }
}

// out[c] = sum of the slab's rows in a fixed order: 16 columns a workgroup, 64 rows at a time.
constexpr int kRedCols = 16, kRedRows = 64;
__global__ __launch_bounds__(kRedCols * kRedRows) void block_reduce_kernel(const float* part_w,
                                                                           const float* part_n,
                                                                           int walkers, int H,
                                                                           float* dw,
                                                                           float* dw_next) {
  __shared__ float red[kRedRows][kRedCols + 1];
  const float* part = blockIdx.y ? part_n : part_w;
  float* out = blockIdx.y ? dw_next : dw;
  if (!out) return;
  const int c = threadIdx.x % kRedCols, g = threadIdx.x / kRedCols;
  const int col = blockIdx.x * kRedCols + c;
  float s = 0.f;
  if (col < H)
    for (int r = g; r < walkers; r += kRedRows) s += part[(int64_t)r * H + col];
  red[g][c] = s;
  __syncthreads();
#pragma unroll
  for (int o = kRedRows / 2; o >= 1; o >>= 1) {
    if (g < o) red[g][c] += red[g + o][c];
    __syncthreads();
  }
  if (g == 0 && col < H) out[col] = red[0][c];
}

// Rows are held by the fewest lanes that take at most 32 columns each.
template <typename Fn>
hipError_t with_shape(int H, Fn&& fn) {
  const int g = (H + 7) / 8;
#define MOE_SHAPE(TPR, NC) fn(std::integral_constant<int, TPR>(), std::integral_constant<int, NC>())
  if (g <= 64) MOE_SHAPE(64, 1);
  else if (g <= 128) MOE_SHAPE(64, 2);
  else if (g <= 192) MOE_SHAPE(64, 3);
  else if (g <= 256) MOE_SHAPE(64, 4);
  else if (g <= 384) MOE_SHAPE(128, 3);
  else if (g <= 512) MOE_SHAPE(128, 4);
  else if (g <= 768) MOE_SHAPE(256, 3);
  else if (g <= 1024) MOE_SHAPE(256, 4);
  else if (g <= 1536) MOE_SHAPE(512, 3);
  else MOE_SHAPE(512, 4);
#undef MOE_SHAPE
  return hipGetLastError();
}

// Walkers of the backward pass: each ends with a row of partial sums, so many rows get few.
int block_walkers(int T, int H) {
  const int most = 1024;
  (void)H;
  return T < most ? T : most;
}

}  // namespace block_norm
}  // namespace

using namespace block_norm;

hipError_t launch_block_forward(const BlockShape& b, const BlockForward& p, hipStream_t s) {
  if (b.T <= 0) return hipSuccess;
  if (b.H > kBlockMaxH) return hipErrorInvalidValue;
  return with_shape(b.H, [&](auto tpr, auto nc) {
    constexpr int TPR = tpr(), NC = nc();
    const dim3 grid((unsigned)((b.T + kRowsOf<TPR> - 1) / kRowsOf<TPR>)), block(kThreadsOf<TPR>);
    if (b.t == Elt::BF16) {
      if (p.f) hipLaunchKernelGGL((block_forward_kernel<Elt::BF16, TPR, NC, true>), grid, block, 0, s, b, p);
      else hipLaunchKernelGGL((block_forward_kernel<Elt::BF16, TPR, NC, false>), grid, block, 0, s, b, p);
    } else {
      if (p.f) hipLaunchKernelGGL((block_forward_kernel<Elt::F32, TPR, NC, true>), grid, block, 0, s, b, p);
      else hipLaunchKernelGGL((block_forward_kernel<Elt::F32, TPR, NC, false>), grid, block, 0, s, b, p);
    }
  });
}

size_t block_part_floats(int T, int H) { return 2 * (size_t)block_walkers(T, H) * H; }

hipError_t launch_block_backward(const BlockShape& b, const BlockBackward& p, hipStream_t s) {
  if (b.H > kBlockMaxH) return hipErrorInvalidValue;
  const int walkers = block_walkers(b.T, b.H);
  float* part_w = p.dw ? p.part : nullptr;
  float* part_n = p.dw_next ? p.part + (size_t)walkers * b.H : nullptr;
  if (b.T > 0) {
    const hipError_t e = with_shape(b.H, [&](auto tpr, auto nc) {
      constexpr int TPR = tpr(), NC = nc();
      const dim3 grid((unsigned)((walkers + kRowsOf<TPR> - 1) / kRowsOf<TPR>)), block(kThreadsOf<TPR>);
#define MOE_BWD(X, DH, RES) \
  hipLaunchKernelGGL((block_backward_kernel<X, DH, TPR, NC, RES>), grid, block, 0, s, b, p, walkers, part_w, part_n)
      if (b.t == Elt::F32) {
        if (p.f) MOE_BWD(Elt::F32, Elt::F32, true); else MOE_BWD(Elt::F32, Elt::F32, false);
      } else if (p.dh_t == Elt::F32) {
        if (p.f) MOE_BWD(Elt::BF16, Elt::F32, true); else MOE_BWD(Elt::BF16, Elt::F32, false);
      } else {
        if (p.f) MOE_BWD(Elt::BF16, Elt::BF16, true); else MOE_BWD(Elt::BF16, Elt::BF16, false);
      }
#undef MOE_BWD
    });
    if (e != hipSuccess) return e;
  }
  if (!p.dw && !p.dw_next) return hipSuccess;
  hipLaunchKernelGGL(block_reduce_kernel, dim3((b.H + kRedCols - 1) / kRedCols, 2),
                     dim3(kRedCols * kRedRows), 0, s, part_w, part_n, walkers, b.H, p.dw, p.dw_next);
  return hipGetLastError();
}

}  // namespace moe
