// The whole MoE layer for at most 16 tokens ("NVIDIA Nemotron 3: Efficient and Open Intelligence",
// section 2.2, latency-oriented deployment) in three launches, four for LatentMoE.
//
// With so few tokens the layer reads every touched weight once and does almost nothing else, so
// its floor is bytes over HBM bandwidth (a Nano-shaped token in bf16: 160 MB) and its cost beyond
// that is dependent launches. A launch here ends only where every later byte depends on what it
// computed:
//   1 front   router scores; LatentMoE's u = x W_in^T and shared up projection
//   2 up      selection (by every workgroup, from the scores), then h = relu(W_up u)^2 of the
//             touched experts; the shared expert's up projection, whose loads are in flight
//             while the selection runs
//   3 down    y = shared + sum_e g_e W_down[e] h_e: a workgroup owns 16 columns of y over a share
//             of the experts, so the gated sum stays in registers; where a column block is cut
//             into parts, the part that ends last adds them up
//   4 out     LatentMoE: y = z W_out^T + shared
// Nothing is gathered or permuted: up to 16 tokens are the columns of one 16 x 16 matrix-core
// block, so every touched expert meets all tokens at the price of one, and the tokens that did
// not select it are dropped (not multiplied by zero, so a NaN stays in its own row).
//
// Products: the weights are the matrix core's first operand (16 rows), loaded from HBM straight to
// registers. Waves split K and join in LDS in wave order, so results are deterministic. Formats
// and roundings are those of the decode path: 8- and 4-bit experts meet rows quantised per row to
// e4m3 (scale amax / 448), h is rounded to bf16 first.
//
// Router: logits are summed in fp64 and rounded to fp32, so that the selection does not depend on
// the order of the sum; scores and keys as in the router kernels.
// Included once, by routing.hip: these kernels are part of that object, so that the library stays the
// objects that its parts are linked from elsewhere (host code under the sanitizers).
#pragma once

#include <algorithm>

#include "common.hpp"
#include "few.hpp"
#include "topk.hpp"

namespace moe {
namespace {
namespace few_layer {

constexpr int TB = kFewTokens;

// ---------------------------------------------------------------------- weight streams
// A step is KS elements of K, one matrix-core instruction; lane l holds weight row l % 16 and
// token l % 16, group g = l / 16 the elements k_of(c, g) .. of its 16-byte chunks c. Result
// register i of lane l is out[weight row 4 g + i][token l % 16].
template <Elt F> struct Fmt {
  static constexpr bool narrow = F != Elt::BF16;
  static constexpr bool mx = F == Elt::MXFP4 || F == Elt::MXFP8;
  static constexpr int KS = narrow ? 128 : 32;
  static constexpr int bits = F == Elt::MXFP4 ? 4 : (narrow ? 8 : 16);
  static constexpr int CW = F == Elt::MXFP4 ? 1 : (narrow ? 2 : 1);  // 16-byte chunks of weights
  static constexpr int CA = narrow ? 2 : 1;                          // and of activations
  // first element of chunk c in a step
  static __device__ __forceinline__ int kw(int c, int g) {
    return F == Elt::MXFP4 ? 32 * g : (narrow ? 64 * c + 16 * g : 8 * g);
  }
  static __device__ __forceinline__ int ka(int c, int g) { return narrow ? 64 * c + 16 * g : 8 * g; }
};

__device__ __forceinline__ i32x8_t cat(uint4 p, uint4 q) {
  return i32x8_t{(int)p.x, (int)p.y, (int)p.z, (int)p.w, (int)q.x, (int)q.y, (int)q.z, (int)q.w};
}

// acc += W[row, steps s0 .. s1) * A. w: the lane's weight row; wx: its block scales (MX);
// aload(el) loads the lane's token chunk that starts at element el. U steps of loads are in flight
// together; chunks past K are read from the row's start and zeroed on both sides.
template <Elt F, int U, class ALoad>
__device__ __forceinline__ f32x4_t dot_steps(const uint8_t* w, const uint8_t* wx, int K, int s0,
                                             int s1, int g, ALoad aload, f32x4_t acc) {
  using M = Fmt<F>;
  const int kend = min(K, s1 * M::KS);
  for (int s = s0; s < s1; s += U) {
    uint4 wf[U][M::CW];
    uint4 af[U][M::CA];
    int sc[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int k0 = (s + q) * M::KS;
#pragma unroll
      for (int c = 0; c < M::CW; ++c) {
        const int el = k0 + M::kw(c, g);
        wf[q][c] = *(const uint4*)(w + (int64_t)(el < kend ? el : 0) * M::bits / 8);
      }
#pragma unroll
      for (int c = 0; c < M::CA; ++c) {
        const int el = k0 + M::ka(c, g);
        af[q][c] = aload(el < kend ? el : 0);
      }
      if constexpr (M::mx) sc[q] = wx[min(k0 / 32 + g, K / 32 - 1)];
      else sc[q] = 127;
    }
    // no branch on the steps past the end: loads whose use is conditional are moved to it, one by
    // one, instead of being in flight together
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int k0 = (s + q) * M::KS;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 wv[M::CW], av[M::CA];
#pragma unroll
      for (int c = 0; c < M::CW; ++c) wv[c] = k0 + M::kw(c, g) < kend ? wf[q][c] : zero;
#pragma unroll
      for (int c = 0; c < M::CA; ++c) av[c] = k0 + M::ka(c, g) < kend ? af[q][c] : zero;
      if constexpr (!M::narrow)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wv[0]),
                                                     __builtin_bit_cast(bf16x8_t, av[0]), acc, 0,
                                                     0, 0);
      else
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            cat(wv[0], M::CW == 2 ? wv[M::CW - 1] : zero), cat(av[0], av[M::CA - 1]), acc,
            F == Elt::MXFP4 ? 4 : 0, 0, 0, sc[q], 0, 127);
    }
  }
  return acc;
}

// 4 bf16 -> 4 e4m3 codes of v * inv.
__device__ __forceinline__ uint32_t codes4(uint32_t p, uint32_t q, float inv) {
  return cvt_fp8x2(bf16_bits_to_f32(p & 0xFFFF) * inv, bf16_bits_to_f32(p >> 16) * inv) |
         cvt_fp8x2(bf16_bits_to_f32(q & 0xFFFF) * inv, bf16_bits_to_f32(q >> 16) * inv) << 16;
}

// out[t][n0 .. n0 + 15] = act(A1[t] . W1[n] + A2[t] . W2[n]) in bf16, by the NW waves of a
// workgroup, each over a contiguous share of the steps. part: [NW][16][17] floats of LDS.
struct Dense {
  const uint16_t *A1, *W1, *A2, *W2;
  int K1, K2, N, T, sq;
  uint16_t* out;
};
template <int NW, int U>
__device__ __forceinline__ void dense_unit(const Dense& d, int n0, float (*part)[16][17]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int t = min(r, d.T - 1);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  const int st1 = cdiv(d.K1, 32), st = st1 + cdiv(d.K2, 32), per = cdiv(st, NW);
  const int lo = min(st, wave * per), hi = min(st, lo + per);
  auto seg = [&](const uint16_t* A, const uint16_t* W, int K, int a, int b) {
    const uint16_t* row = A + (int64_t)t * K;
    acc = dot_steps<Elt::BF16, U>((const uint8_t*)(W + (int64_t)(n0 + r) * K), nullptr, K, a, b, g,
                                  [&](int el) { return *(const uint4*)(row + el); }, acc);
  };
  if (lo < st1) seg(d.A1, d.W1, d.K1, lo, min(hi, st1));
  if (hi > st1) seg(d.A2, d.W2, d.K2, max(lo, st1) - st1, hi - st1);
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][r][4 * g + i] = acc[i];
  __syncthreads();
  if (threadIdx.x < 64 && r < d.T) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = part[0][r][4 * g + i];
#pragma unroll
      for (int q = 1; q < NW; ++q) v[i] += part[q][r][4 * g + i];
      if (d.sq) v[i] = sqrelu(v[i]);
    }
    *(uint2*)(d.out + (int64_t)r * d.N + n0 + 4 * g) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// ------------------------------------------------------------------------------ 1 front
// Workgroups [0, E): one expert's logits and scores; for LatentMoE then 16 rows each of Ws_up and
// of W_in. Also clears what the later launches raise or count.
template <int TT>
__global__ __launch_bounds__(256) void few_front(FewParams p) {
  __shared__ float part[4][16][17];
  __shared__ double red[4][TT];
  const int tid = threadIdx.x;
  const int nr = p.given ? 0 : p.E;
  const int bid = blockIdx.x;
  const int nz = p.hmax ? few_slots(p.T, p.E, p.k) * TB : 0;
  for (int i = bid * 256 + tid; i < nz; i += gridDim.x * 256) p.hmax[i] = 0;
  for (int i = bid * 256 + tid; i < p.D / 16; i += gridDim.x * 256) p.joined[i] = 0;
  if (bid < nr) {
    double acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.0;
    const uint16_t* w = p.W_r + (int64_t)bid * p.H;
    for (int c = tid * 8; c < p.H; c += 256 * 8) {
      const uint4 wq = *(const uint4*)(w + c);
      uint4 xq[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) xq[t] = *(const uint4*)(p.x + (int64_t)min(t, p.T - 1) * p.H + c);
      const uint32_t wv[4] = {wq.x, wq.y, wq.z, wq.w};
      double wd[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        wd[2 * j] = (double)bf16_bits_to_f32(wv[j] & 0xFFFF);
        wd[2 * j + 1] = (double)bf16_bits_to_f32(wv[j] >> 16);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t xv[4] = {xq[t].x, xq[t].y, xq[t].z, xq[t].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[t] = fma(wd[2 * j], (double)bf16_bits_to_f32(xv[j] & 0xFFFF), acc[t]);
          acc[t] = fma(wd[2 * j + 1], (double)bf16_bits_to_f32(xv[j] >> 16), acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) acc[t] += __shfl_xor(acc[t], o);
      if ((tid & 63) == 0) red[tid >> 6][t] = acc[t];
    }
    __syncthreads();
    if (tid < p.T) {
      const float z = (float)(red[0][tid] + red[1][tid] + red[2][tid] + red[3][tid]);
      p.logits[(int64_t)tid * p.E + bid] = z;
      p.score[(int64_t)tid * p.E + bid] = (float)(1.0 / (1.0 + exp(-(double)z)));
    }
    return;
  }
  if (!p.L) return;
  int n = bid - nr;
  if (n < p.Is / 16) {
    dense_unit<4, 7>(Dense{p.x, p.Ws_up, nullptr, nullptr, p.H, 0, p.Is, p.T, 1, p.hs}, 16 * n, part);
    return;
  }
  n -= p.Is / 16;
  if (n < p.L / 16)
    dense_unit<4, 7>(Dense{p.x, p.W_in, nullptr, nullptr, p.H, 0, p.L, p.T, 0, p.u}, 16 * n, part);
}

// --------------------------------------------------------------------------------- 2 up
// One workgroup of 8 waves per CU. First the shared expert: workgroup n takes 16 rows of Ws_up,
// its waves split K, and the loads are issued before the selection, which needs two round trips to
// the scores and a chain of wave-wide maxima. Then units of (touched expert, 16 rows of W_up), one
// wave each over all of K, double buffered: while a batch of U steps is multiplied the next one
// (of this unit or of the wave's next) is in flight. Activations are read from LDS: bf16 rows, or
// e4m3 codes for 8- and 4-bit experts. NPER * 64 >= E; XLDS: the rows fit (else from L2).
constexpr int kUpWaves = 8;
constexpr int kUpThreads = 64 * kUpWaves;
constexpr size_t kUpRowsLds = 96 * 1024;   // of the staged activations
constexpr int kSharedSteps = 12;   // steps of the shared unit in flight per wave

// LDS row stride of the staged activations, an odd number of 16-byte chunks (16 rows at one chunk
// index then fall on distinct banks).
__host__ __device__ inline int up_stride(int row_bytes) {
  const int c = (row_bytes + 15) / 16;
  return 16 * (c | 1);
}

template <Elt F, int NPER, bool XLDS>
__global__ __launch_bounds__(kUpThreads) void few_up(FewParams p) {
  using M = Fmt<F>;
  __shared__ int idx_l[TB * 64];
  __shared__ float gates_l[TB * 64];
  __shared__ uint32_t emask[NPER * 64];     // tokens that selected expert e
  __shared__ int slot_l[NPER * 64];         // touched experts, ascending
  __shared__ int cnt[NPER];
  __shared__ float part[kUpWaves][16][17];
  __shared__ float row_scale[TB];
  extern __shared__ __attribute__((aligned(16))) uint8_t xl[];  // [T] rows of lds bytes
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int t = min(r, p.T - 1);
  const uint16_t* in = p.L ? p.u : p.x;

  // the shared expert's first loads
  const int nsh = p.L ? 0 : p.Is / 16;
  const int st = cdiv(p.H, 32), sper = cdiv(st, kUpWaves);
  const int slo = min(st, wave * sper), shi = min(st, slo + sper);
  const int send = min(p.H, shi * 32);
  uint4 sw[kSharedSteps], sa[kSharedSteps];
  const uint16_t* srow = p.x + (int64_t)t * p.H;
  if ((int)blockIdx.x < nsh && slo < shi) {
    const uint16_t* w = p.Ws_up + (int64_t)(16 * blockIdx.x + r) * p.H;
#pragma unroll
    for (int q = 0; q < kSharedSteps; ++q) {
      const int el = (slo + q) * 32 + 8 * g;
      sw[q] = *(const uint4*)(w + (el < send ? el : 0));
      sa[q] = *(const uint4*)(srow + (el < send ? el : 0));
    }
  }

  for (int i = tid; i < NPER * 64; i += kUpThreads) emask[i] = 0;
  __syncthreads();
  const int ldx = up_stride(M::narrow ? p.D : 2 * p.D);
  for (int tk = wave; tk < p.T; tk += kUpWaves) {
    // selection of token tk
    bool ok = lane < p.k;
    if (p.given) {
      int e = -1;
      if (ok) {
        e = p.idx_in[tk * p.k + lane];
        idx_l[tk * p.k + lane] = e;
        gates_l[tk * p.k + lane] = p.gates_in[tk * p.k + lane];
      }
      ok = ok && (unsigned)e < (unsigned)p.E;
      for (int j = 0; j < p.k; ++j)   // a repeated expert: its first slot counts
        if (__shfl(e, j) == e && j < lane) ok = false;
      if (!ok && lane < p.k) idx_l[tk * p.k + lane] = -1;
    } else {
      float key[NPER], sc[NPER];
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 64 * i;
        sc[i] = e < p.E ? p.score[(int64_t)tk * p.E + e] : 0.f;
        key[i] = e < p.E ? sc[i] + p.b[e] : 0.f;
      }
      select_topk<NPER, true>(key, sc, lane, p.E, p.k, idx_l + tk * p.k, gates_l + tk * p.k);
    }
    if (ok) atomicOr(&emask[idx_l[tk * p.k + lane]], 1u << tk);
    // its row: bf16 as it is, or e4m3 codes with scale amax / 448 (1 for a zero row)
    const uint16_t* row = in + (int64_t)tk * p.D;
    if constexpr (M::narrow) {
      float m = 0.f;
      for (int c = lane * 8; c < p.D; c += 512) {
        const uint4 v = *(const uint4*)(row + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m = fmaxf(m, fmaxf(fabsf(bf16_bits_to_f32(w[i] & 0xFFFF)), fabsf(bf16_bits_to_f32(w[i] >> 16))));
      }
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
      const float inv = m > 0.f ? 448.f / m : 1.f;
      if (lane == 0) row_scale[tk] = m > 0.f ? m / 448.f : 1.f;
      for (int c = lane * 8; c < p.D; c += 512) {
        const uint4 v = *(const uint4*)(row + c);
        *(uint2*)(xl + tk * ldx + c) = make_uint2(codes4(v.x, v.y, inv), codes4(v.z, v.w, inv));
      }
    } else if constexpr (XLDS) {
      for (int c = lane * 8; c < p.D; c += 512) *(uint4*)(xl + tk * ldx + 2 * c) = *(const uint4*)(row + c);
    }
  }
  __syncthreads();
  // touched experts, ascending
  for (int c = wave; c < NPER; c += kUpWaves) {
    const uint64_t any = __ballot(emask[c * 64 + lane] != 0);
    if (lane == 0) cnt[c] = __popcll(any);
  }
  __syncthreads();
  int n_slots = 0;
#pragma unroll
  for (int c = 0; c < NPER; ++c) {
    const bool mine = c % kUpWaves == wave;
    if (mine) {
      const bool on = emask[c * 64 + lane] != 0;
      const uint64_t any = __ballot(on);
      if (on) slot_l[n_slots + __popcll(any & ((1ull << lane) - 1))] = c * 64 + lane;
    }
    n_slots += cnt[c];
  }
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1) {  // what launch 3 and the caller read
    if (tid == 0) *p.n_slots = n_slots;
    for (int i = tid; i < n_slots; i += kUpThreads) {
      p.slot_e[i] = slot_l[i];
      p.slot_mask[i] = emask[slot_l[i]];
    }
    for (int i = tid; i < n_slots * TB; i += kUpThreads) {
      const int e = slot_l[i / TB], tk = i % TB;
      float v = 0.f;
      if (tk < p.T)
        for (int j = p.k - 1; j >= 0; --j)
          if (idx_l[tk * p.k + j] == e) v = gates_l[tk * p.k + j];
      p.gate_m[i] = v;
    }
    if (!p.given)
      for (int i = tid; i < p.T * p.k; i += kUpThreads) {
        p.idx[i] = idx_l[i];
        p.gates[i] = gates_l[i];
      }
  }

  // the shared expert
  for (int n = blockIdx.x; n < nsh; n += gridDim.x) {
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    int from = slo;
    if (n == (int)blockIdx.x) {
#pragma unroll
      for (int q = 0; q < kSharedSteps; ++q) {
        const bool inside = (slo + q) * 32 + 8 * g < send;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8_t, inside ? sw[q] : zero),
            __builtin_bit_cast(bf16x8_t, inside ? sa[q] : zero), acc, 0, 0, 0);
      }
      from = min(shi, slo + kSharedSteps);
    }
    acc = dot_steps<Elt::BF16, 8>((const uint8_t*)(p.Ws_up + (int64_t)(16 * n + r) * p.H), nullptr,
                                  p.H, from, shi, g,
                                  [&](int el) { return *(const uint4*)(srow + el); }, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][r][4 * g + i] = acc[i];
    __syncthreads();
    if (wave == 0 && r < p.T) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = part[0][r][4 * g + i];
#pragma unroll
        for (int q = 1; q < kUpWaves; ++q) v[i] += part[q][r][4 * g + i];
        v[i] = sqrelu(v[i]);
      }
      *(uint2*)(p.hs + (int64_t)r * p.Is + 16 * n + 4 * g) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
    if (n + (int)gridDim.x < nsh) __syncthreads();
  }

  // routed units: u = wave-slot, + waves of the grid
  const int nb = p.I / 16, total = n_slots * nb, stride = gridDim.x * kUpWaves;
  int u = wave * gridDim.x + blockIdx.x;
  if (u >= total) return;
  constexpr int U = F == Elt::BF16 ? 12 : 7;
  const int steps = cdiv(p.D, M::KS), nbat = cdiv(steps, U);
  struct Unit { const uint8_t *w, *wx; int slot, n0, e; };
  auto resolve = [&](int v) {
    Unit x;
    x.slot = v / nb;
    x.n0 = (v - x.slot * nb) * 16;
    x.e = __builtin_amdgcn_readfirstlane(slot_l[x.slot]);
    const int64_t row = (int64_t)x.e * p.I + x.n0 + r;
    x.w = p.W_up + row * p.D * M::bits / 8;
    x.wx = M::mx ? (const uint8_t*)p.s_up + row * (p.D / 32) : nullptr;
    return x;
  };
  auto issue = [&](const Unit& x, int b, uint4* wf, int* sc) {
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int k0 = (b * U + q) * M::KS;   // chunks past D: the row's start, zeroed when used
#pragma unroll
      for (int c = 0; c < M::CW; ++c) {
        const int el = k0 + M::kw(c, g);
        wf[q * M::CW + c] = *(const uint4*)(x.w + (int64_t)(el < p.D ? el : 0) * M::bits / 8);
      }
      if constexpr (M::mx) sc[q] = x.wx[min(k0 / 32 + g, p.D / 32 - 1)];
      else sc[q] = 127;
    }
  };
  Unit cur = resolve(u), nxt = cur;
  bool more = u + stride < total;
  if (more) nxt = resolve(u + stride);
  int b = 0;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  auto step = [&](uint4* wc, int* sc, uint4* wn, int* sn) {
    const bool last = b + 1 == nbat;
    const bool other = last && more;
    Unit src = cur;
    if (other) src = nxt;
    issue(src, last ? 0 : b + 1, wn, sn);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int k0 = (b * U + q) * M::KS;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 wv[M::CW], av[M::CA];
#pragma unroll
      for (int c = 0; c < M::CW; ++c) wv[c] = k0 + M::kw(c, g) < p.D ? wc[q * M::CW + c] : zero;
#pragma unroll
      for (int c = 0; c < M::CA; ++c) {
        const int el = k0 + M::ka(c, g);
        const int at = el < p.D ? el : 0;
        const uint4 v = M::narrow ? *(const uint4*)(xl + t * ldx + at)
                        : XLDS    ? *(const uint4*)(xl + t * ldx + 2 * at)
                                  : *(const uint4*)(in + (int64_t)t * p.D + at);
        av[c] = el < p.D ? v : zero;
      }
      if constexpr (!M::narrow)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wv[0]),
                                                     __builtin_bit_cast(bf16x8_t, av[0]), acc, 0,
                                                     0, 0);
      else
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            cat(wv[0], M::CW == 2 ? wv[M::CW - 1] : zero), cat(av[0], av[M::CA - 1]), acc,
            F == Elt::MXFP4 ? 4 : 0, 0, 0, sc[q], 0, 127);
    }
    if (!last) {
      ++b;
      return true;
    }
    const bool sel = (emask[cur.e] >> r) & 1;   // bits of tokens below T only
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = acc[i];
      if constexpr (F == Elt::FP8)
        v[i] *= row_scale[t] * ((const float*)p.s_up)[(int64_t)cur.e * p.I + cur.n0 + 4 * g + i];
      else if constexpr (M::mx)
        v[i] *= row_scale[t];
      v[i] = sqrelu(v[i]);
      acc[i] = 0.f;
    }
    const uint32_t lo2 = pack_bf16x2(v[0], v[1]), hi2 = pack_bf16x2(v[2], v[3]);
    if (sel)
      *(uint2*)(p.h + ((int64_t)cur.slot * p.T + r) * p.I + cur.n0 + 4 * g) = make_uint2(lo2, hi2);
    if constexpr (M::narrow) {  // the row's maximum (h >= 0: bf16 bits order as integers)
      uint32_t m = max(max(lo2 << 16, lo2 & 0xFFFF0000u), max(hi2 << 16, hi2 & 0xFFFF0000u));
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if (sel && g == 0) atomicMax(p.hmax + cur.slot * TB + r, m);
    }
    if (!more) return false;
    cur = nxt;
    b = 0;
    u += stride;
    more = u + stride < total;
    if (more) nxt = resolve(u + stride);
    return true;
  };
  uint4 w0[U * M::CW], w1[U * M::CW];
  int s0[U], s1[U];
  issue(cur, 0, w0, s0);
  for (;;) {
    if (!step(w0, s0, w1, s1)) break;
    if (!step(w1, s1, w0, s0)) break;
  }
}

// ------------------------------------------------------------------------------- 3 down
// Workgroup (n, part): 16 columns of y (or z) over a contiguous share of the list (slot, step) of
// all touched experts, which its waves share evenly; the shared expert's steps likewise. Parts of
// a column block are written to fp32 slabs, and the workgroup that ends last adds them in part
// order (a counter that launch 1 cleared; nobody waits). 8- and 4-bit experts: the h rows of the
// share are first turned into e4m3 codes in LDS, as many slots at a time as fit.
constexpr int kDownWaves = 8;
constexpr int kDownThreads = 64 * kDownWaves;
constexpr int kDownRowsLds = 72 * 1024;

template <Elt F>
__global__ __launch_bounds__(kDownThreads) void few_down(FewParams p) {
  using M = Fmt<F>;
  __shared__ float part[kDownWaves][16][17];
  __shared__ int first_row[1024 + 1];          // narrow: first code row of a slot of this pass
  extern __shared__ __attribute__((aligned(16))) uint8_t hq[];  // narrow: code rows
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int t = min(r, p.T - 1);
  const int n0 = blockIdx.x * 16;
  const int parts = gridDim.y, mine = blockIdx.y;
  const int n_slots = *p.n_slots;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  if (p.Is && !p.L) {
    const int steps = cdiv(p.Is, 32), per = cdiv(steps, kDownWaves * parts);
    const int lo = min(steps, (mine * kDownWaves + wave) * per), hi = min(steps, lo + per);
    const uint16_t* row = p.hs + (int64_t)t * p.Is;
    sum = dot_steps<Elt::BF16, 8>((const uint8_t*)(p.Ws_down + (int64_t)(n0 + r) * p.Is), nullptr,
                                  p.Is, lo, hi, g,
                                  [&](int el) { return *(const uint4*)(row + el); }, sum);
  }
  const int spe = cdiv(p.I, M::KS);      // steps per expert
  const int total = n_slots * spe, share = cdiv(total, parts);
  const int begin = min(total, mine * share), end = min(total, begin + share);
  const int ldh = up_stride(p.I);

  // steps [at, stop) of one wave
  auto run = [&](int at, int stop, int pass_slot) {
    while (at < stop) {
      const int slot = at / spe, s0 = at - slot * spe, s1 = min(spe, s0 + stop - at);
      at += s1 - s0;
      const int e = p.slot_e[slot];
      const uint32_t mask = p.slot_mask[slot];
      const int64_t row = (int64_t)e * p.D + n0 + r;
      const bool sel = (mask >> r) & 1;
      float scale = p.gate_m[slot * TB + r];
      // tokens that did not select the expert read another's row (their products are dropped)
      const int src = sel ? r : __ffs(mask) - 1;
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      const uint8_t* w = p.W_down + row * p.I * M::bits / 8;
      const uint8_t* wx = M::mx ? (const uint8_t*)p.s_down + row * (p.I / 32) : nullptr;
      if constexpr (M::narrow) {
        const float m = __uint_as_float(p.hmax[slot * TB + src]);
        scale *= m > 0.f ? m / 448.f : 1.f;
        const uint8_t* q = hq + (first_row[slot - pass_slot] + __popc(mask & ((1u << src) - 1))) * ldh;
        acc = dot_steps<F, 4>(w, wx, p.I, s0, s1, g,
                              [&](int el) { return *(const uint4*)(q + el); }, acc);
      } else {
        const uint16_t* h = p.h + ((int64_t)slot * p.T + src) * p.I;
        acc = dot_steps<F, 8>(w, wx, p.I, s0, s1, g,
                              [&](int el) { return *(const uint4*)(h + el); }, acc);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = acc[i] * scale;
        if constexpr (F == Elt::FP8)
          v *= ((const float*)p.s_down)[(int64_t)e * p.D + n0 + 4 * g + i];
        if (sel) sum[i] += v;
      }
    }
  };
  if constexpr (!M::narrow) {
    const int per = cdiv(end - begin, kDownWaves);
    const int lo = min(end, begin + wave * per);
    run(lo, min(end, lo + per), 0);
  } else {
    const int cap = kDownRowsLds / ldh;   // >= kFewTokens (checked by the launcher)
    for (int at = begin; at < end;) {
      // slots of this pass: as many as have room, at least one
      const int slot0 = at / spe, slot_end = cdiv(end, spe);
      __syncthreads();                    // the pass before is done with the code rows
      if (wave == 0) {
        int rows = 0, n = 0;
        for (int s = slot0; s < slot_end; s += 64) {   // wave-wide prefix of the slots' row counts
          const int c = s + lane < slot_end ? __popc(p.slot_mask[s + lane]) : 0;
          int inc = c;
#pragma unroll
          for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(inc, o);
            if (lane >= o) inc += v;
          }
          const bool fits = s + lane < slot_end && rows + inc <= cap;
          if (fits) first_row[s - slot0 + lane] = rows + inc - c;
          const int k = __popcll(__ballot(fits));
          n += k;
          rows += k ? __shfl(inc, k - 1) : 0;
          if (k < 64) break;
        }
        if (lane == 0) part[0][0][16] = __int_as_float(n);
      }
      __syncthreads();
      const int n = __float_as_int(part[0][0][16]);
      for (int s = slot0; s < slot0 + n; ++s) {
        const uint32_t mask = p.slot_mask[s];
        int j = first_row[s - slot0];
        for (uint32_t m = mask; m; m &= m - 1, ++j) {   // rows dealt to the waves
          if (j % kDownWaves != wave) continue;
          const int tk = __ffs(m) - 1;
          const float top = __uint_as_float(p.hmax[s * TB + tk]);
          const float inv = top > 0.f ? 448.f / top : 1.f;
          const uint16_t* h = p.h + ((int64_t)s * p.T + tk) * p.I;
          for (int c = lane * 8; c < p.I; c += 512) {
            const uint4 v = *(const uint4*)(h + c);
            *(uint2*)(hq + j * ldh + c) = make_uint2(codes4(v.x, v.y, inv), codes4(v.z, v.w, inv));
          }
        }
      }
      __syncthreads();
      const int stop = min(end, (slot0 + n) * spe);
      const int per = cdiv(stop - at, kDownWaves);
      const int lo = min(stop, at + wave * per);
      run(lo, min(stop, lo + per), slot0);
      at = stop;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][r][4 * g + i] = sum[i];
  __syncthreads();
  if (wave != 0) return;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = part[0][r][4 * g + i];
#pragma unroll
    for (int q = 1; q < kDownWaves; ++q) v[i] += part[q][r][4 * g + i];
  }
  if (parts > 1) {
    float* slab = p.slabs + ((int64_t)blockIdx.x * parts) * 256 + lane * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __hip_atomic_store(slab + mine * 256 + i, v[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // the slab is written through to memory (agent scope); wait for that, then count
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int before = 0;
    if (lane == 0)
      before = __hip_atomic_fetch_add(p.joined + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__builtin_amdgcn_readfirstlane(before) != parts - 1) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0.f;
      for (int q = 0; q < parts; ++q)
        v[i] += __hip_atomic_load(slab + q * 256 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  uint16_t* out = p.L ? p.z : p.y;
  if (r < p.T)
    *(uint2*)(out + (int64_t)r * p.D + n0 + 4 * g) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// -------------------------------------------------------------------------------- 4 out
__global__ __launch_bounds__(512) void few_out(FewParams p) {
  __shared__ float part[8][16][17];
  dense_unit<8, 8>(Dense{p.z, p.W_out, p.hs, p.Ws_down, p.L, p.Is, p.H, p.T, 0, p.y},
                   16 * blockIdx.x, part);
}

template <Elt F, bool XLDS>
hipError_t run_up(const FewParams& p, int grid, size_t lds, hipStream_t s) {
  const dim3 block(kUpThreads);
  if (p.E <= 128) hipLaunchKernelGGL((few_up<F, 2, XLDS>), dim3(grid), block, lds, s, p);
  else if (p.E <= 512) hipLaunchKernelGGL((few_up<F, 8, XLDS>), dim3(grid), block, lds, s, p);
  else hipLaunchKernelGGL((few_up<F, 16, XLDS>), dim3(grid), block, lds, s, p);
  return hipGetLastError();
}

template <Elt F>
hipError_t run_down(const FewParams& p, hipStream_t s) {
  size_t lds = 0;
  if (Fmt<F>::narrow) {
    // room for every pair's code row, or as many as kDownRowsLds holds
    const int64_t ldh = up_stride(p.I), rows = std::min<int64_t>((int64_t)p.T * p.k, kDownRowsLds / ldh);
    if (rows < std::min(p.T * p.k, p.T)) return hipErrorInvalidValue;
    lds = (size_t)(rows * ldh);
  }
  hipLaunchKernelGGL((few_down<F>), dim3(p.D / 16, few_parts(p.D)), dim3(kDownThreads), lds, s, p);
  return hipGetLastError();
}

}  // namespace few_layer
}  // namespace

using namespace few_layer;

hipError_t launch_few_front(const FewParams& p, hipStream_t s) {
  if (p.T < 1 || p.T > kFewTokens) return hipErrorInvalidValue;
  const int front = (p.given ? 0 : p.E) + (p.L ? p.Is / 16 + p.L / 16 : 0);
  const dim3 grid(std::max(front, 1)), block(256);
  if (p.T == 1) hipLaunchKernelGGL((few_front<1>), grid, block, 0, s, p);
  else if (p.T <= 4) hipLaunchKernelGGL((few_front<4>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((few_front<16>), grid, block, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_few_up(const FewParams& p, hipStream_t s) {
  // one workgroup per CU; fewer when all the units there can be need fewer
  const int64_t units = (int64_t)few_slots(p.T, p.E, p.k) * (p.I / 16);
  const int64_t want = std::max<int64_t>(units, p.L ? 1 : p.Is / 16);
  const int grid = (int)std::min<int64_t>(256, want);
  const size_t narrow = (size_t)p.T * up_stride(p.D), wide = (size_t)p.T * up_stride(2 * p.D);
  switch (p.ex) {
    case Elt::BF16:
      return wide <= kUpRowsLds ? run_up<Elt::BF16, true>(p, grid, wide, s)
                                : run_up<Elt::BF16, false>(p, grid, 0, s);
    case Elt::FP8: return run_up<Elt::FP8, true>(p, grid, narrow, s);
    case Elt::MXFP4: return run_up<Elt::MXFP4, true>(p, grid, narrow, s);
    case Elt::MXFP8: return run_up<Elt::MXFP8, true>(p, grid, narrow, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_few_down(const FewParams& p, hipStream_t s) {
  switch (p.ex) {
    case Elt::BF16: return run_down<Elt::BF16>(p, s);
    case Elt::FP8: return run_down<Elt::FP8>(p, s);
    case Elt::MXFP4: return run_down<Elt::MXFP4>(p, s);
    case Elt::MXFP8: return run_down<Elt::MXFP8>(p, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_few_out(const FewParams& p, hipStream_t s) {
  hipLaunchKernelGGL(few_out, dim3(p.H / 16), dim3(512), 0, s, p);
  return hipGetLastError();
}

}  // namespace moe
