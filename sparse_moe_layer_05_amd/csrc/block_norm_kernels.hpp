// The norms before and after a block, fused with its gate, its residual and the next block's norm,
// and their gradients (gfx950).
//
//   n(v) = v / sqrt(mean(v^2) + eps)
//   y = x + scale a z, z = n(f) w or f w, a = gate or sigmoid(gate) or 1;  h = n(y) w_next
//   gradient of n at v against g:  r (g - n(v) mean(g n(v))), r = 1 / sqrt(mean(v^2) + eps)
//
// Bound by HBM: each row is read once and held in registers between its sums and its result (but for the
// longest ones' gradients, see with_backward_shape), so neither pass keeps statistics for the other. A row
// is held by 8 to 64 lanes of a wave, or by a workgroup where it is long. The forward pass reads weights
// after the row's sum, a group of columns at a time: at 2688 columns one row with both norms waits for
// eight loads in turn. y is rounded before the next norm reads it: the backward pass, which
// has y as it is stored, then differentiates the same function. Sums run in fp32; where a sum of
// squares passes fp32 it is taken again of smaller values, a branch that no ordinary row takes.
// Measured (bf16; a copy of 4 GiB reaches 4.7 TB/s): forward with both norms and a gate per token, 8192
// x 2688, 32 to 36 us, 4.9 to 5.6 TB/s; one row 4.6 us, of one norm alone 2.5; backward with both norms and
// a gate per element, 8192 x 4096, 95 us, 5.9 TB/s, and 6 us for the weights' gradients; with a gate per
// token, 8192 x 2688, 58 and 5 us. Rows none of which has a gradient from the next norm: up to 5% more.
// Included once, by backward.hip.
#pragma once

#include "block_norm.hpp"
#include "common.hpp"
#include "row8.hpp"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {
namespace block_norm {

// Sums over the TPR lanes of a row, in every lane. Where a row has several waves each adds all waves'
// sums, one a lane. Two slots take turns, so one barrier a sum is enough: whoever writes a slot again
// has passed the barrier of the other one, behind which nobody still reads it.
template <int TPR>
struct RowSum {
  static constexpr int W = TPR > 64 ? TPR / 64 : 1, kSlot = 3 * W;
  float* lds;     // 2 * kSlot
  int slot = 0;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N <= 3 && W <= 16);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (TPR < 64) v[i] = group_sum<TPR>(v[i]);
      else v[i] = wave_sum(v[i]);
    }
    if constexpr (W > 1) {
      const int lane = threadIdx.x & 63;
      float* const at = lds + slot;
      slot = kSlot - slot;
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) at[i * W + (threadIdx.x >> 6)] = v[i];
      // (LDS alone is waited for: loads of the next row stay in flight)
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = row16_sum(lane < W ? at[i * W + lane] : 0.f);
    }
  }
};

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
  // p = exp(-|q| / 2) = 2^t (1 + r ln 2), t + r = -|q| log2(e) / 2 to 48 bits, and exp(-|q|) = p p: the
  // hardware's 2^t has no subnormal results, a product has. From 104 on p p rounds to 0 (a NaN stays).
  const float x = fabsf(q) > 104.f ? -104.f : -fabsf(q);
  const float t = x * 0.72134751f;
  const float r = fmaf(x, 9.62981515e-9f, fmaf(x, 0.72134751f, -t));
  const float p2 = __builtin_amdgcn_exp2f(t), p = fmaf(p2 * r, 0.693147182f, p2);
  // 1 / (1 + p p), 1 + p p in [1, 2]: the hardware's reciprocal and one Newton step
  const float u = fmaf(p, p, 1.f), v = __builtin_amdgcn_rcpf(u), inv = fmaf(v, fmaf(-u, v, 1.f), v);
  return q < 0.f ? GateValue{p * (p * inv), inv} : GateValue{inv, p * (p * inv)};
}

__device__ __forceinline__ float inv_rms(float ss, int H, float eps) {
  return 1.f / sqrtf(ss / (float)H + eps);
}
__device__ __forceinline__ bool too_big(float s) { return fabsf(s) == __builtin_inff(); }

// Rows whose sum of squares passes fp32 (values beyond 2^57) are summed again with their values times
// kFar: 2^48 at most, while values that then underflow are below 2^-60 of the row's largest.
constexpr float kFar = 0x1p-80f;
__device__ __forceinline__ float inv_rms_far(float ss, int H, float eps) {   // of the values times kFar
  return 1.f / sqrtf(ss / (float)H + eps * kFar * kFar);
}

// 1 / rms of the row held in v; ss: its fp32 sum of squares.
template <int TPR, Elt T, int NC>
__device__ __forceinline__ float row_inv_rms(Raw8<T> (&v)[NC], float ss, int H, float eps,
                                             RowSum<TPR>& sum) {
  if (__builtin_expect(too_big(ss), 0)) {   // the same in every lane of the row
    float d[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float u[8];
      forget(v[i]);
      unpack8<T>(v[i], u);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[0] = fmaf(u[e] * kFar, u[e] * kFar, d[0]);
    }
    sum(d);
    return inv_rms_far(d[0], H, eps) * kFar;
  }
  return inv_rms(ss, H, eps);
}

// The gradient's mean(g n(v)) is taken as sum(g v) r / H, in the same reduction as sum(v^2). Where that
// leaves fp32, though the mean does not, or is so small that products of it may have been subnormal
// (16384 of them lose 2^-136 in all, 2^-36 of kLeastDot), or zero, as in a row without a gradient, it is
// taken again of the normalised row: sum(g n) / H, or sum(g (n / H)) unless the sum is small. (The norm of
// f sums g n(f) at once, which only large gradients take out of fp32.)
constexpr float kLeastDot = 0x1p-100f;
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_inff(); }
template <int TPR, Elt T, int NC>
__device__ __forceinline__ float far_mean(const float (&g)[NC][8], Raw8<T> (&v)[NC], float r, bool small,
                                          float inv_h, RowSum<TPR>& sum) {
  const float part = small ? 1.f : inv_h;
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float u[8];
    forget(v[i]);
    unpack8<T>(v[i], u);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[0] = fmaf(g[i][e], u[e] * r * part, q[0]);
  }
  sum(q);
  return small ? q[0] * inv_h : q[0];
}

// Where a lane works: rows of TPR lanes each, several of them side by side in a wave where they are
// short, and four waves a workgroup unless a row needs a workgroup of its own.
template <int TPR> constexpr int kThreadsOf = TPR <= 64 ? 256 : TPR;
template <int TPR> constexpr int kRowsOf = kThreadsOf<TPR> / TPR;         // rows of a workgroup
template <int TPR> constexpr int kRowsOfWave = TPR < 64 ? 64 / TPR : 1;
template <int TPR, int NC>
struct Place {
  int lane, sub;       // lane of its row, row of the wave's
  int row0;            // the wave's first row: the same in every lane, so that addresses are scalar
  uint32_t at[NC];     // the lane's elements, counted from the first row; kAway past the row
  __device__ __forceinline__ explicit Place(int H) {
    lane = TPR <= 64 ? threadIdx.x & (TPR - 1) : threadIdx.x;
    sub = TPR < 64 ? (threadIdx.x & 63) / TPR : 0;
    row0 = blockIdx.x * kRowsOf<TPR>;
    if constexpr (TPR <= 64)
      row0 += __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kRowsOfWave<TPR>;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int col = group(i) * 8;
      at[i] = col < H ? (uint32_t)(sub * H + col) : kAway;
    }
  }
  __device__ __forceinline__ int group(int i) const { return lane + i * TPR; }
  __device__ __forceinline__ bool in_row(int i) const { return at[i] != kAway; }
  // rows of the wave at `row` that there are
  __device__ __forceinline__ static int rows(int row, int T) { return min(T - row, kRowsOfWave<TPR>); }
};

// RES: y and, where p.h is given, the next norm of it; else h alone, the norm of x.
template <Elt T, int TPR, int NC, bool RES>
__global__ __launch_bounds__(kThreadsOf<TPR>) void block_forward_kernel(BlockShape b,
                                                                        BlockForward p) {
  __shared__ float lds[2 * RowSum<TPR>::kSlot];
  RowSum<TPR> sum{lds};
  const Place<TPR, NC> me(b.H);
  const int rows = me.rows(me.row0, b.T), row = me.row0 + me.sub;
  if (rows <= 0) return;   // whole waves, and workgroups where a row has a barrier
  Raw8<T> xr[NC], fr[NC], gr[NC];
  {
    const RowBuffer<T> x(p.x, me.row0, rows, b.H), f(p.f, me.row0, rows, b.H);
    const RowBuffer<T> g(b.gate_kind == Gate::Element ? p.gate : nullptr, me.row0, rows, b.H);
    x.load(me.at, xr, p.stream);
    if constexpr (RES) {
      f.load(me.at, fr, p.stream);
      g.load(me.at, gr, p.stream);
    }
  }
  if constexpr (RES) {
    float rf = 1.f;
    if (b.norm) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float f[8];
        unpack8<T>(fr[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] = fmaf(f[e], f[e], ss[0]);
      }
      sum(ss);
      rf = row_inv_rms<TPR, T, NC>(fr, ss[0], b.H, b.eps, sum);
    }
    float at = b.scale;   // scale, times the row's gate
    if (b.gate_kind == Gate::Token)
      at *= gate_value(row < b.T ? ((const float*)p.gate)[row] : 0.f, b.sigmoid).a;
    const RowBuffer<T> y(p.y, me.row0, rows, b.H);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!me.in_row(i)) continue;
      float v[8], w[8], f[8], g[8];
      load_w8(p.w, b.w_t, me.group(i) * 8, w);
      unpack8<T>(xr[i], v);
      unpack8<T>(fr[i], f);
      unpack8<T>(gr[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float z = f[e] * rf * w[e] * at;
        if (b.gate_kind == Gate::Element) z *= gate_value(g[e], b.sigmoid).a;
        v[e] += z;
      }
      xr[i] = pack8<T>(v);
      y.store(me.at[i], xr[i]);
    }
    if (!p.h) return;
  }
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float v[8];
    unpack8<T>(xr[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[0] = fmaf(v[e], v[e], ss[0]);
  }
  sum(ss);
  const float r = row_inv_rms<TPR, T, NC>(xr, ss[0], b.H, b.eps, sum);
  const RowBuffer<T> h(p.h, me.row0, rows, b.H);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!me.in_row(i)) continue;
    float v[8], w[8], o[8];
    load_w8(p.w_next, b.w_t, me.group(i) * 8, w);
    unpack8<T>(xr[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = v[e] * r * w[e];
    h.store(me.at[i], pack8<T>(o));
  }
}

// A weight of one lane group's columns, kept in LDS as fp32 for every row of the walk: group g's eight
// values as two 16-byte halves, each half of neighbouring groups side by side.
template <int GROUPS>
struct LdsWeight {
  float4 v[2][GROUPS];
  __device__ void fill(const void* w, Elt t, int H) {
    for (int g = threadIdx.x; g < GROUPS; g += blockDim.x) {
      float u[8] = {};
      if (g * 8 < H) load_w8(w, t, g * 8, u);
      put(g, u);
    }
  }
  __device__ void put(int g, const float (&u)[8]) {
    v[0][g] = make_float4(u[0], u[1], u[2], u[3]);
    v[1][g] = make_float4(u[4], u[5], u[6], u[7]);
  }
  __device__ void add(int g, float (&u)[8]) const {
    float w[8];
    get(g, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] += w[e];
  }
  __device__ void get(int g, float (&u)[8]) const {
    const float4 a = v[0][g], b = v[1][g];
    u[0] = a.x; u[1] = a.y; u[2] = a.z; u[3] = a.w;
    u[4] = b.x; u[5] = b.y; u[6] = b.z; u[7] = b.w;
  }
};

// A workgroup takes every gridDim.x-th kRowsOf rows; sums of dw and dw_next over its rows go to its row
// of two slabs [workgroups][H].
template <Elt T, Elt DH, int TPR, int NC, bool RES>
__global__ __launch_bounds__(kThreadsOf<TPR>) void block_backward_kernel(BlockShape b,
                                                                         BlockBackward p,
                                                                         float* part_w,
                                                                         float* part_n) {
  __shared__ float lds[2 * RowSum<TPR>::kSlot];
  __shared__ LdsWeight<TPR * NC> lw_next;
  __shared__ LdsWeight<RES ? TPR * NC : 1> lw;
  RowSum<TPR> sum{lds};
  const Place<TPR, NC> me(b.H);
  const int step = gridDim.x * kRowsOf<TPR>;
  const float inv_h = 1.f / (float)b.H;
  float sw[NC][8] = {}, sn[NC][8] = {};
  // A row's operands are loaded into the registers of the row before as soon as that row is done
  // with them, so that loads are in flight during the sums, whose barriers wait for LDS alone.
  Raw8<T> yr[NC], dr[NC], fr[NC], gr[NC];
  Raw8<DH> hr[NC];
  const bool element = b.gate_kind == Gate::Element, token = b.gate_kind == Gate::Token;
  const void* const gates = element ? p.gate : nullptr;
  auto load_y = [&](int row) {
    const RowBuffer<T> y(p.dh ? p.y : nullptr, row, me.rows(row, b.T), b.H);
    const RowBuffer<DH> h(p.dh, row, me.rows(row, b.T), b.H);
    y.load(me.at, yr, p.stream);
    h.load(me.at, hr, p.stream);
  };
  auto load_row = [&](Raw8<T>(&r)[NC], const void* base, int row) {
    const RowBuffer<T> rb(base, row, me.rows(row, b.T), b.H);
    rb.load(me.at, r, p.stream);
  };
  load_y(me.row0);
  if constexpr (RES) load_row(fr, p.f, me.row0);
  load_row(dr, p.dy, me.row0);
  if constexpr (RES) load_row(gr, gates, me.row0);
  lw_next.fill(p.w_next, b.w_t, b.H);
  if constexpr (RES) lw.fill(p.w, b.w_t, b.H);
  __syncthreads();
  for (int row0 = me.row0; row0 < b.T; row0 += step) {
    const int next = row0 + step, rows = me.rows(row0, b.T);   // (T and the step are far below 2^30)
    // sum y^2, sum (dh w_next) y, sum f^2
    float s[3] = {0.f, 0.f, 0.f};
    float d[NC][8];   // d, the gradient reaching y
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float y[8], h[8], w[8], f[8];
      unpack8<T>(yr[i], y);
      unpack8<DH>(hr[i], h);
      lw_next.get(me.group(i), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[i][e] = h[e] * w[e];
        s[0] = fmaf(y[e], y[e], s[0]);
        s[1] = fmaf(d[i][e], y[e], s[1]);
      }
      if constexpr (RES) {
        unpack8<T>(fr[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[2] = fmaf(f[e], f[e], s[2]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    sum(s);
    if (p.dh) {
      float r = inv_rms(s[0], b.H, b.eps), m = s[1] * r * inv_h;
      if (__builtin_expect(too_big(s[0]) || !(fabsf(s[1]) >= kLeastDot) || !finite(m), 0)) {
        r = row_inv_rms<TPR, T, NC>(yr, s[0], b.H, b.eps, sum);
        m = far_mean<TPR, T, NC>(d, yr, r, fabsf(s[1]) * r < 1.f, inv_h, sum);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float y[8], h[8];
        forget(yr[i]);
        forget(hr[i]);
        unpack8<T>(yr[i], y);
        unpack8<DH>(hr[i], h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = y[e] * r;
          d[i][e] = r * fmaf(-n, m, d[i][e]);
          sn[i][e] = fmaf(h[e], n, sn[i][e]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    load_y(next);
    {
      const RowBuffer<T> xo(p.dx, row0, rows, b.H);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float dy[8];
        unpack8<T>(dr[i], dy);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] += dy[e];
        xo.store(me.at[i], pack8<T>(d[i]));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    load_row(dr, p.dy, next);
    if constexpr (RES) {
      const float rf = b.norm ? row_inv_rms<TPR, T, NC>(fr, s[2], b.H, b.eps, sum) : 1.f;
      GateValue gt = {1.f, 1.f};   // the row's gate
      const int row = row0 + me.sub;
      if (token) gt = gate_value(row < b.T ? ((const float*)p.gate)[row] : 0.f, b.sigmoid);
      // sum d a w n(f): the mean in the norm's gradient and, with a = 1, the token gate's gradient
      float q[1] = {0.f};
      const RowBuffer<T> go(element ? p.dgate : nullptr, row0, rows, b.H);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float w[8], f[8];
        lw.get(me.group(i), w);
        forget(fr[i]);
        unpack8<T>(fr[i], f);
        if (element) {
          float g[8], o[8];
          unpack8<T>(gr[i], g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const GateValue ge = gate_value(g[e], b.sigmoid);
            const float n = f[e] * rf, ds = d[i][e] * b.scale, dz = ds * ge.a;
            o[e] = (b.sigmoid ? dz : ds) * ge.rest * (n * w[e]);
            sw[i][e] = fmaf(dz, n, sw[i][e]);
            d[i][e] = dz * w[e];
            q[0] = fmaf(d[i][e], n, q[0]);
          }
          go.store(me.at[i], pack8<T>(o));
        } else {
          // (the sum is of the values without the token's gate, whose own gradient needs it so)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float n = f[e] * rf, ds = d[i][e] * b.scale;
            sw[i][e] = fmaf(ds * gt.a, n, sw[i][e]);
            const float dw = ds * w[e];
            q[0] = fmaf(dw, n, q[0]);
            d[i][e] = dw * gt.a;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      load_row(gr, gates, next);
      if (b.norm || token) sum(q);
      if (token && me.lane == 0 && row < b.T && p.dgate)
        ((float*)p.dgate)[row] = q[0] * gt.rest * (b.sigmoid ? gt.a : 1.f);
      float m = b.norm ? q[0] * gt.a * inv_h : 0.f;   // (gt.a is 1 but for a token's gate)
      if (__builtin_expect(!finite(m), 0)) m = far_mean<TPR, T, NC>(d, fr, rf, false, inv_h, sum);
      const RowBuffer<T> fo(p.df, row0, rows, b.H);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float f[8], o[8];
        forget(fr[i]);
        unpack8<T>(fr[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e] = b.norm ? rf * fmaf(-f[e] * rf, m, d[i][e]) : d[i][e];
        fo.store(me.at[i], pack8<T>(o));
        __builtin_amdgcn_sched_barrier(0);
      }
      load_row(fr, p.f, next);
    }
  }
  if constexpr (TPR < 64) {   // the wave's rows
#pragma unroll
    for (int o = TPR; o < 64; o *= 2)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sn[0][e] += __shfl_xor(sn[0][e], o);
        if constexpr (RES) sw[0][e] += __shfl_xor(sw[0][e], o);
      }
  }
  if constexpr (TPR <= 64) {   // the workgroup's waves, one after another
    const int wave = threadIdx.x >> 6;
    for (int q = 0; q < 4; ++q) {
      __syncthreads();
      if (wave != q || me.sub) continue;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (q) {
          lw_next.add(me.group(i), sn[i]);
          if constexpr (RES) lw.add(me.group(i), sw[i]);
        }
        if (q < 3) {
          lw_next.put(me.group(i), sn[i]);
          if constexpr (RES) lw.put(me.group(i), sw[i]);
        }
      }
    }
    if (wave != 3 || me.sub) return;
  }
  const RowBuffer<Elt::F32> pw(part_w, blockIdx.x, 1, b.H), pn(part_n, blockIdx.x, 1, b.H);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (RES) pw.store(me.at[i], pack8<Elt::F32>(sw[i]));
    pn.store(me.at[i], pack8<Elt::F32>(sn[i]));
  }
}

// out[c] = sum of the slab's rows in a fixed order: 32 columns (a cache line, so that no two dies read
// it) a workgroup, eight lanes a row, 128 rows at a time and six times as many in flight.
constexpr int kRedThreads = 1024, kRedRows = kRedThreads / 8, kRedAhead = 6;
__global__ __launch_bounds__(kRedThreads) void block_reduce_kernel(const float* part_w,
                                                                   const float* part_n, int rows,
                                                                   int H, float* dw,
                                                                   float* dw_next) {
  __shared__ float red[kRedThreads / 64][32];
  const float* part = blockIdx.y ? part_n : part_w;
  float* out = blockIdx.y ? dw_next : dw;
  if (!out) return;
  const int quad = threadIdx.x & 7, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 32 + quad * 4;
  float s[4] = {};
  if (col < H)   // (H is a multiple of 16)
    for (int r = threadIdx.x >> 3; r < rows; r += kRedAhead * kRedRows) {
      float4 v[kRedAhead];
#pragma unroll
      for (int i = 0; i < kRedAhead; ++i) {
        const int at = r + i * kRedRows;
        v[i] = at < rows ? *(const float4*)(part + (int64_t)at * H + col) : make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kRedAhead; ++i) {
        s[0] += v[i].x; s[1] += v[i].y; s[2] += v[i].z; s[3] += v[i].w;
      }
    }
#pragma unroll
  for (int o = 8; o < 64; o *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += __shfl_xor(s[e], o);
  if (lane < 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][quad * 4 + e] = s[e];
  __syncthreads();
  const int c = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && c < H) {
    float t = red[0][threadIdx.x];
    for (int w = 1; w < kRedThreads / 64; ++w) t += red[w][threadIdx.x];
    out[c] = t;
  }
}

// Lanes of a row and groups of eight columns a lane. Forward up to four groups: a lane holds three
// operands, at most 115 registers, four waves a SIMD. Backward up to two: it holds five operands, a gradient
// and two sums, 146 registers for bf16 (three waves a SIMD), 186 for fp32 (two), 87 to 111 for the norm
// alone; four groups took 326 and one wave a SIMD. Microseconds with two groups / one on twice the lanes:
// 8192 x 4096 108 / 106, 8192 x 2688 67 / 76, 16384 x 1024 44 / 51.
// A workgroup of 1024 lanes has 128 registers a lane, one of 768 has 168, so the residual's gradient spills
// inside the walk: past 12288 columns 44 bytes a lane (bf16), 100 (bf16 with fp32 dh) or 196 (fp32), fp32
// past 8192 36. As many elements, 8192 x 4096 / 2048 x 16384: bf16 95 / 114 us, fp32 212 / 329, of whose 819
// MB written 390 are spilled.
template <typename Fn>
void with_forward_shape(int H, Fn&& fn) {
  const int g = (H + 7) / 8;
#define MOE_SHAPE(TPR, NC) fn(std::integral_constant<int, TPR>(), std::integral_constant<int, NC>())
  if (g <= 8) MOE_SHAPE(8, 1);
  else if (g <= 16) MOE_SHAPE(16, 1);
  else if (g <= 32) MOE_SHAPE(32, 1);
  else if (g <= 64) MOE_SHAPE(64, 1);
  else if (g <= 128) MOE_SHAPE(64, 2);
  else if (g <= 192) MOE_SHAPE(64, 3);
  else if (g <= 256) MOE_SHAPE(64, 4);
  else if (g <= 384) MOE_SHAPE(128, 3);
  else if (g <= 512) MOE_SHAPE(128, 4);
  else if (g <= 768) MOE_SHAPE(256, 3);
  else if (g <= 1024) MOE_SHAPE(256, 4);
  else if (g <= 1536) MOE_SHAPE(512, 3);
  else MOE_SHAPE(512, 4);
}
template <typename Fn>
void with_backward_shape(int H, Fn&& fn) {
  const int g = (H + 7) / 8;
  if (g <= 8) MOE_SHAPE(8, 1);
  else if (g <= 16) MOE_SHAPE(16, 1);
  else if (g <= 32) MOE_SHAPE(32, 1);
  else if (g <= 64) MOE_SHAPE(64, 1);
  else if (g <= 128) MOE_SHAPE(64, 2);
  else if (g <= 256) MOE_SHAPE(128, 2);
  else if (g <= 384) MOE_SHAPE(192, 2);
  else if (g <= 512) MOE_SHAPE(256, 2);
  else if (g <= 768) MOE_SHAPE(384, 2);
  else if (g <= 1024) MOE_SHAPE(512, 2);
  else if (g <= 1536) MOE_SHAPE(768, 2);
  else MOE_SHAPE(1024, 2);
#undef MOE_SHAPE
}

// Workgroups of the backward pass: 16 waves on each of the 256 CUs, at most 12 where a lane has two groups,
// which is what the registers of the residual's bf16 gradient hold: each ends with a row of partial sums,
// and a second round leaves most CUs idle. Other forms get the same number: fp32 with a residual holds
// eight, so a third of its workgroups run in a second round (8192 x 4096 212 us, 5.2 TB/s); the norm alone
// would hold 16 to 20. Microseconds of bf16 with a residual, 8 / 12 / 16 waves a CU (two groups a lane):
// 8192 x 4096 108 / 108 / 119, 16384 x 1024 47 / 44 / 52, 16384 x 4096 165 / 156 / 184; 8192 x 2688, 6 / 9 / 12
// waves, 81 / 71 / 67.
int backward_groups(int T, int H) {
  int groups = 0;
  with_backward_shape(H, [&](auto tpr, auto nc) {
    constexpr int TPR = tpr(), waves = kThreadsOf<TPR> / 64;
    constexpr int most = nc() == 1 ? 16 : 12;
    constexpr int per_cu = most / waves > 0 ? most / waves : 1;
    groups = std::min((T + kRowsOf<TPR> - 1) / kRowsOf<TPR>, 256 * per_cu);
  });
  return groups;
}

}  // namespace block_norm
}  // namespace

using namespace block_norm;

// Operands and results that together pass the last-level cache (256 MB) are read past it, so that the
// results, which the next call reads, stay. Microseconds with and without, the forward pass alone and
// followed by a product that reads h: 16384 x 4096 (537 MB) 93 / 109 and 152 / 163, 8192 x 4096 52 / 55
// and 87 / 89, but 8192 x 2688 (176 MB) 38 / 37 and 64 / 62, 2048 x 2688 12.2 / 12.2 and 26.3 / 24.5.
// The backward pass: 8192 x 4096 108 / 122, 16384 x 4096 156 / 170, 4096 x 8192 99 / 102.
bool past_cache(const BlockShape& b, int tensors) {
  return (int64_t)b.T * b.H * (b.t == Elt::BF16 ? 2 : 4) * tensors > (int64_t)256 << 20;
}

hipError_t launch_block_forward(const BlockShape& b, const BlockForward& given, hipStream_t s) {
  if (b.T <= 0) return hipSuccess;
  BlockForward p = given;
  p.stream = past_cache(b, (p.f ? 3 : 1) + (p.h ? 1 : 0) + (b.gate_kind == Gate::Element));
  if (b.H > kBlockMaxH) return hipErrorInvalidValue;
  with_forward_shape(b.H, [&](auto tpr, auto nc) {
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
  return hipGetLastError();
}

size_t block_part_floats(int T, int H) { return 2 * (size_t)backward_groups(T, H) * H; }

hipError_t launch_block_backward(const BlockShape& b, const BlockBackward& given, hipStream_t s) {
  BlockBackward p = given;
  p.stream = past_cache(b, 1 + (p.dy ? 1 : 0) + (p.dh ? 2 : 0) + (p.f ? 2 : 0) +
                               (b.gate_kind == Gate::Element ? 2 : 0));
  if (b.H > kBlockMaxH) return hipErrorInvalidValue;
  const int groups = backward_groups(b.T, b.H);
  // a single workgroup's sums are the result (stored 16 bytes at a time)
  const bool one = groups == 1 && (((uintptr_t)p.dw | (uintptr_t)p.dw_next) & 15) == 0;
  float* part_w = !p.dw ? nullptr : one ? p.dw : p.part;
  float* part_n = !p.dw_next ? nullptr : one ? p.dw_next : p.part + (size_t)groups * b.H;
  if (b.T > 0) {
    with_backward_shape(b.H, [&](auto tpr, auto nc) {
      constexpr int TPR = tpr(), NC = nc();
      const dim3 grid((unsigned)groups), block(kThreadsOf<TPR>);
#define MOE_BWD(X, DH, RES) \
  hipLaunchKernelGGL((block_backward_kernel<X, DH, TPR, NC, RES>), grid, block, 0, s, b, p, part_w, part_n)
      if (b.t == Elt::F32) {
        if (p.f) MOE_BWD(Elt::F32, Elt::F32, true); else MOE_BWD(Elt::F32, Elt::F32, false);
      } else if (p.dh_t == Elt::F32) {
        if (p.f) MOE_BWD(Elt::BF16, Elt::F32, true); else MOE_BWD(Elt::BF16, Elt::F32, false);
      } else {
        if (p.f) MOE_BWD(Elt::BF16, Elt::BF16, true); else MOE_BWD(Elt::BF16, Elt::BF16, false);
      }
#undef MOE_BWD
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || one) return e;
  }
  if (!p.dw && !p.dw_next) return hipSuccess;
  hipLaunchKernelGGL(block_reduce_kernel, dim3((b.H + 31) / 32, 2), dim3(kRedThreads), 0, s, part_w,
                     part_n, groups, b.H, p.dw, p.dw_next);
  return hipGetLastError();
}

}  // namespace moe
