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
// registers and multiplied as bf16: e4m3 and E2M1 elements times their block scales are bf16
// numbers (but for E4M3 elements below 2^-133, in blocks of scale code 2 or less, which round), and
// so are e4m3 activation codes, while the 8- and 4-bit instructions cut products (13 bits below the
// largest of eight) and thereby move roundings of h, one in some hundred rows its
// quantisation scale and with it 4% of the row. The conversions hide under the loads. Waves split
// K and join in LDS in wave order: results are deterministic.
//
// Formats as on the decode path: 8- and 4-bit experts meet rows quantised per row to e4m3 (scale
// amax / 448), h rounded to bf16 first. Where the definition does not round, intermediates are
// kept as the sum of two bf16 (16 bits; the shared expert's h, a bf16 expert's h, LatentMoE's z),
// multiplied in two instructions by the weights that are in registers anyway. Where it rounds to bf16
// and a row's largest element then sets its e4m3 scale (h of 8- and 4-bit experts, LatentMoE's u), the
// sum is widened to fp64 every 256 products and rounded once: in fp32 some hundred rows held one
// whose scale, and with it most of its codes, fell on the other side of a bf16 border (6 tokens
// through LatentMoE with e4m3 experts: y 4.8e-3 off, 1.66e-3 now; 0 to 1 us a call). What fp32 sums
// of 256 leave makes that rarer, not impossible.
//
// Router: logits are summed in fp64 and rounded to fp32, so that the selection does not depend on
// the order of the sum; scores and keys as in the router kernels.
// Included once, by routing.hip: these kernels are part of that object, so that the library stays
// the objects that its parts are linked from elsewhere (host code under the sanitizers).
#pragma once

#include <algorithm>
#include <type_traits>

#include "bf16_pair.hpp"
#include "common.hpp"
#include "few.hpp"
#include "topk.hpp"

namespace moe {
namespace {
namespace few_layer {

constexpr int TB = kFewTokens;

// ---------------------------------------------------------------------- weight streams
// A step is KS elements of K: MF matrix-core instructions. Lane l holds weight row l % 16 and
// token l % 16; group g = l / 16 holds, of both operands and for instruction j of a step, the 8
// elements from k_of(j, g) on (any order of k serves: both sides use the same). bf16: one 16-byte
// chunk of 8 elements. 8- and 4-bit weights: 32 consecutive elements a lane, one block scale.
// Result register i of lane l is out[weight row 4 g + i][token l % 16].
template <Elt F> struct Fmt {
  static constexpr bool narrow = F != Elt::BF16;
  static constexpr bool mx = F == Elt::MXFP4 || F == Elt::MXFP8;
  static constexpr int KS = narrow ? 128 : 32, MF = narrow ? 4 : 1;
  static constexpr int bits = F == Elt::MXFP4 ? 4 : (narrow ? 8 : 16);
  static constexpr int CW = F == Elt::BF16 || F == Elt::MXFP4 ? 1 : 2;  // 16-byte chunks of weights
  static constexpr int EC = 128 / bits;                                // elements of a chunk
  static __device__ __forceinline__ int kw(int c, int g) { return (narrow ? 32 : 8) * g + EC * c; }
  static __device__ __forceinline__ int k_of(int j, int g) { return (narrow ? 32 : 8) * g + 8 * j; }
};

// One step's weights of a lane.
template <Elt F> struct WStep {
  uint4 c[Fmt<F>::CW];
  int sc;   // E8M0 code (MX)
};
// Loads step s of the row at w (wx: its block scales). Chunks at or past kend are read from the
// row's start; mask_step zeroes them.
template <Elt F>
__device__ __forceinline__ void load_step(WStep<F>& x, const uint8_t* w, const uint8_t* wx, int s,
                                          int kend, int K, int g) {
  using M = Fmt<F>;
#pragma unroll
  for (int c = 0; c < M::CW; ++c) {
    const int el = s * M::KS + M::kw(c, g);
    x.c[c] = *(const uint4*)(w + (int64_t)(el < kend ? el : 0) * M::bits / 8);
  }
  if constexpr (M::mx) x.sc = wx[min(s * 4 + g, K / 32 - 1)];
}
template <Elt F>
__device__ __forceinline__ void mask_step(WStep<F>& x, int s, int kend, int g) {
  using M = Fmt<F>;
#pragma unroll
  for (int c = 0; c < M::CW; ++c)
    if (s * M::KS + M::kw(c, g) >= kend) x.c[c] = make_uint4(0, 0, 0, 0);
}
// Both sides of a product past the end of K are zeroed: zero times an infinity is NaN.
__device__ __forceinline__ void zero_if(bool past, uint4& v) {
  if (past) v = make_uint4(0, 0, 0, 0);
}
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bits_of(bf16x2_t v) { return __builtin_bit_cast(uint32_t, v); }
// Instruction j's weight fragment in bf16.
template <Elt F>
__device__ __forceinline__ bf16x8_t wfrag(const WStep<F>& x, int j) {
  uint4 o = x.c[0];
  if constexpr (F == Elt::MXFP4) {
    const float s = __uint_as_float((uint32_t)x.sc << 23);
    const uint32_t w = j == 0 ? x.c[0].x : j == 1 ? x.c[0].y : j == 2 ? x.c[0].z : x.c[0].w;
    o = make_uint4(bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3)));
  } else if constexpr (Fmt<F>::narrow) {
    const float s = Fmt<F>::mx ? __uint_as_float((uint32_t)x.sc << 23) : 1.f;
    const uint4 c = j < 2 ? x.c[0] : x.c[Fmt<F>::CW - 1];
    const uint32_t lo = j & 1 ? c.z : c.x, hi = j & 1 ? c.w : c.y;
    o = make_uint4(bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true)));
  }
  return __builtin_bit_cast(bf16x8_t, o);
}
__device__ __forceinline__ f32x4_t mul(bf16x8_t w, uint4 a, f32x4_t acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8_t, a), acc, 0, 0, 0);
}

// 8 bf16 -> the bf16 values of their e4m3 codes: e4m3(v * inv).
__device__ __forceinline__ uint32_t code2(uint32_t p, float inv) {
  const uint32_t c = cvt_fp8x2(bf16_bits_to_f32(p & 0xFFFF) * inv, bf16_bits_to_f32(p >> 16) * inv);
  return bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.f, false));
}
__device__ __forceinline__ uint4 codes8(uint4 v, float inv) {
  return make_uint4(code2(v.x, inv), code2(v.y, inv), code2(v.z, inv), code2(v.w, inv));
}

// Four fp32 as a pair of bf16 each, v = hi + lo up to 2^-17 of v, at column n of row o.
__device__ __forceinline__ void store_pair(uint16_t* hi, uint16_t* lo, int64_t at, const float* v) {
  const uint2 h = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  *(uint2*)(hi + at) = h;
  *(uint2*)(lo + at) = make_uint2(bf16x2_rest(v[0], v[1], h.x), bf16x2_rest(v[2], v[3], h.y));
}

// Four sums of one lane. A Sum of doubles takes the matrix core's fp32 sums of a batch of steps at a
// time, each batch from zero: where a value is rounded to bf16 and the largest of them sets its
// row's scale, a sum that rounds with every instruction now and then falls on the other side of a
// bf16 border, and most codes of the row move with it.
template <class T> struct Sum {
  T v[4] = {0, 0, 0, 0};
  __device__ __forceinline__ f32x4_t start() const {   // what a batch begins with
    if constexpr (sizeof(T) == 4) return f32x4_t{v[0], v[1], v[2], v[3]};
    else return f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void take(f32x4_t acc) {   // and what it ends with
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = sizeof(T) == 4 ? (T)acc[i] : v[i] + (T)acc[i];
  }
};
__device__ __forceinline__ double sqrelu(double a) { return a <= 0.0 ? 0.0 : a * a; }
using moe::sqrelu;

// sum += W[row, steps s0 .. s1) * (A + A2) of bf16 rows in memory, U steps of loads in flight.
// No branch on the steps past the end: loads whose use is conditional are moved to it, one by
// one, instead of being in flight together.
template <int U, bool LO, class T>
__device__ __forceinline__ void dot_rows(const uint16_t* w, const uint16_t* a, const uint16_t* a2,
                                         int K, int s0, int s1, int g, Sum<T>& sum) {
  const int kend = min(K, s1 * 32);
  for (int s = s0; s < s1; s += U) {
    uint4 wf[U], af[U], bf[LO ? U : 1];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int el = (s + q) * 32 + 8 * g, at = el < kend ? el : 0;
      wf[q] = *(const uint4*)(w + at);
      af[q] = *(const uint4*)(a + at);
      if constexpr (LO) bf[q] = *(const uint4*)(a2 + at);
    }
    f32x4_t acc = sum.start();
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const bool past = (s + q) * 32 + 8 * g >= kend;
      zero_if(past, wf[q]);
      zero_if(past, af[q]);
      if constexpr (LO) zero_if(past, bf[q]);
      acc = mul(__builtin_bit_cast(bf16x8_t, wf[q]), af[q], acc);
      if constexpr (LO) acc = mul(__builtin_bit_cast(bf16x8_t, wf[q]), bf[q], acc);
    }
    sum.take(acc);
  }
}

// out[t][n0 .. n0 + 15] = act(A1[t] . W1[n] + A2[t] . W2[n]) by the NW waves of a workgroup, each
// over a contiguous share of the steps, summed in S. LO: the activations are pairs. out_lo: so is the
// result.
struct Dense {
  const uint16_t *A1, *A1lo, *W1, *A2, *A2lo, *W2;
  int K1, K2, N, T, sq;
  uint16_t *out, *out_lo;
};
template <int NW, int U, bool LO, class S>
__device__ __forceinline__ void dense_unit(const Dense& d, int n0, S (*part)[16][17]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int t = min(r, d.T - 1);
  Sum<S> acc;
  const int st1 = cdiv(d.K1, 32), st = st1 + cdiv(d.K2, 32), per = cdiv(st, NW);
  const int lo = min(st, wave * per), hi = min(st, lo + per);
  if (lo < st1)
    dot_rows<U, LO>(d.W1 + (int64_t)(n0 + r) * d.K1, d.A1 + (int64_t)t * d.K1,
                    d.A1lo + (int64_t)t * d.K1, d.K1, lo, min(hi, st1), g, acc);
  if (hi > st1)
    dot_rows<U, LO>(d.W2 + (int64_t)(n0 + r) * d.K2, d.A2 + (int64_t)t * d.K2,
                    d.A2lo + (int64_t)t * d.K2, d.K2, max(lo, st1) - st1, hi - st1, g, acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][r][4 * g + i] = acc.v[i];
  __syncthreads();
  if (threadIdx.x < 64 && r < d.T) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      S x = part[0][r][4 * g + i];
#pragma unroll
      for (int q = 1; q < NW; ++q) x += part[q][r][4 * g + i];
      v[i] = (float)(d.sq ? sqrelu(x) : x);
    }
    const int64_t at = (int64_t)r * d.N + n0 + 4 * g;
    if (d.out_lo)
      store_pair(d.out, d.out_lo, at, v);
    else
      *(uint2*)(d.out + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// ------------------------------------------------------------------------------ 1 front
// Workgroups [0, E): one expert's logits and scores; for LatentMoE then 16 rows each of Ws_up and
// of W_in. Also clears what the later launches raise or count.
template <int TT>
__global__ __launch_bounds__(256) void few_front(FewParams p) {
  __shared__ double part[4][16][17];   // u is rounded to bf16
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
    dense_unit<4, 8, false>(Dense{p.x, p.x, p.Ws_up, nullptr, nullptr, nullptr, p.H, 0, p.Is, p.T,
                                  1, p.hs, p.hs_lo}, 16 * n, part);
    return;
  }
  n -= p.Is / 16;
  if (n < p.L / 16)
    dense_unit<4, 8, false>(Dense{p.x, p.x, p.W_in, nullptr, nullptr, nullptr, p.H, 0, p.L, p.T, 0,
                                  p.u, nullptr}, 16 * n, part);
}

// --------------------------------------------------------------------------------- 2 up
// One workgroup per CU. First the shared expert: workgroup n takes 16 rows of Ws_up, its waves
// split K, and the loads are issued before the selection, which needs two round trips to the scores
// and a chain of wave-wide maxima. Then units of (touched expert, 16 rows of W_up), one wave each
// over all of K, double buffered: while a batch of U steps is multiplied the next one (of this unit
// or of the wave's next) is in flight. Activations are read from LDS, as bf16 rows or the bf16
// values of their e4m3 codes, zeros up to a whole step. NPER * 64 >= E; XLDS: the rows fit (else
// bf16 ones are read from L2).
// bf16: 8 waves with 12 steps a batch (one token 48.6 us per layer; 16 waves with 6 steps 50.9;
// two or four waves sharing a unit's K 53 and more). 8- and 4-bit weights, whose units are shorter
// and leave an uneven second round: 16 waves (MXFP4, 4 tokens: 58.8 us against 61.3; e4m3, 16
// tokens: 164 against 165). A plain read of the same 80 MB takes 14.5 us, in this pattern (16 rows
// of 64 bytes an instruction) 16 to 18.
// More than 512 experts: 8 waves whatever the weights, as 16 scores and keys a lane beside the shared
// expert's loads need more than the 128 registers of 16 waves (E 1024, k 8, H 2048, I 512, MXFP4: 4
// tokens 43.5 us against 53 with 80 registers in scratch, 16 tokens 88 against 96).
template <Elt F, int NPER> constexpr int kUpWaves = F == Elt::BF16 || NPER > 8 ? 8 : 16;
constexpr size_t kUpRowsLds = 130 * 1024;   // of the staged activations
// steps of the shared unit in flight per wave
template <Elt F, int NPER> constexpr int kSharedSteps = kUpWaves<F, NPER> == 8 ? 12 : 6;

// LDS row stride in bytes of K staged elements, whole steps of 128 and an odd number of 16-byte
// chunks (16 rows at one chunk index then fall on distinct banks).
__host__ __device__ inline int lds_stride(int K) { return (K + 127) / 128 * 256 + 16; }

template <Elt F, int NPER, bool XLDS>
__global__ __launch_bounds__((64 * kUpWaves<F, NPER>)) void few_up(FewParams p) {
  using M = Fmt<F>;
  constexpr int NWV = kUpWaves<F, NPER>, NTH = 64 * NWV, SS = kSharedSteps<F, NPER>;
  __shared__ int idx_l[TB * 64];
  __shared__ float gates_l[TB * 64];
  __shared__ uint32_t emask[NPER * 64];     // tokens that selected expert e
  __shared__ int slot_l[NPER * 64];         // touched experts, ascending
  __shared__ int cnt[NPER];
  __shared__ float part[NWV / 2][16][17];
  __shared__ float row_scale[TB];
  extern __shared__ __attribute__((aligned(16))) uint8_t xl[];  // [T] rows of ldx bytes
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int t = min(r, p.T - 1);
  const uint16_t* in = p.L ? p.u : p.x;

  // the shared expert's first loads
  const int nsh = p.L ? 0 : p.Is / 16;
  const int st = cdiv(p.H, 32), sper = cdiv(st, NWV);
  const int slo = min(st, wave * sper), shi = min(st, slo + sper);
  const int send = min(p.H, shi * 32);
  uint4 sw[SS], sa[SS];
  const uint16_t* srow = p.x + (int64_t)t * p.H;
  if ((int)blockIdx.x < nsh && slo < shi) {
    const uint16_t* w = p.Ws_up + (int64_t)(16 * blockIdx.x + r) * p.H;
#pragma unroll
    for (int q = 0; q < SS; ++q) {
      const int el = (slo + q) * 32 + 8 * g, at = el < send ? el : 0;
      sw[q] = *(const uint4*)(w + at);
      sa[q] = *(const uint4*)(srow + at);
    }
  }

  for (int i = tid; i < NPER * 64; i += NTH) emask[i] = 0;
  __syncthreads();
  const int ldx = lds_stride(p.D);
  for (int tk = wave; tk < p.T; tk += NWV) {
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
    // its row: bf16 as it is, or e4m3 codes
    const uint16_t* row = in + (int64_t)tk * p.D;
    float inv = 1.f;
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
      const RowScale rs = row_scale_e4m3(m);
      inv = rs.up;
      if (lane == 0) row_scale[tk] = rs.down;
    }
    if constexpr (XLDS)
      for (int c = lane * 8; c < ldx / 2; c += 512) {   // the last chunk: zeros for steps past the end
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < p.D) v = *(const uint4*)(row + c);
        *(uint4*)(xl + tk * ldx + 2 * c) = M::narrow ? codes8(v, inv) : v;
      }
  }
  __syncthreads();
  // touched experts, ascending
  for (int c = wave; c < NPER; c += NWV) {
    const uint64_t any = __ballot(emask[c * 64 + lane] != 0);
    if (lane == 0) cnt[c] = __popcll(any);
  }
  __syncthreads();
  int n_slots = 0;
#pragma unroll
  for (int c = 0; c < NPER; ++c) {
    if (c % NWV == wave) {
      const bool on = emask[c * 64 + lane] != 0;
      const uint64_t any = __ballot(on);
      if (on) slot_l[n_slots + __popcll(any & ((1ull << lane) - 1))] = c * 64 + lane;
    }
    n_slots += cnt[c];
  }
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1) {  // what launch 3 and the caller read
    if (tid == 0) *p.n_slots = n_slots;
    for (int i = tid; i < n_slots; i += NTH) {
      p.slot_e[i] = slot_l[i];
      p.slot_mask[i] = emask[slot_l[i]];
    }
    for (int i = tid; i < n_slots * TB; i += NTH) {
      const int e = slot_l[i / TB], tk = i % TB;
      float v = 0.f;
      if (tk < p.T)
        for (int j = p.k - 1; j >= 0; --j)
          if (idx_l[tk * p.k + j] == e) v = gates_l[tk * p.k + j];
      p.gate_m[i] = v;
    }
    if (!p.given)
      for (int i = tid; i < p.T * p.k; i += NTH) {
        p.idx[i] = idx_l[i];
        p.gates[i] = gates_l[i];
      }
  }

  // the shared expert
  for (int n = blockIdx.x; n < nsh; n += gridDim.x) {
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    int from = slo;
    if (n == (int)blockIdx.x && slo < shi) {
#pragma unroll
      for (int q = 0; q < SS; ++q) {
        const bool past = (slo + q) * 32 + 8 * g >= send;
        zero_if(past, sw[q]);
        zero_if(past, sa[q]);
        acc = mul(__builtin_bit_cast(bf16x8_t, sw[q]), sa[q], acc);
      }
      from = min(shi, slo + SS);
    }
    Sum<float> sum;
    sum.take(acc);
    dot_rows<4, false>(p.Ws_up + (int64_t)(16 * n + r) * p.H, srow, srow, p.H, from, shi, g, sum);
    acc = sum.start();
    constexpr int half = NWV / 2;   // the upper half's sums, then the lower's added to them
    if (wave >= half)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave - half][r][4 * g + i] = acc[i];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][r][4 * g + i] += acc[i];
    __syncthreads();
    if (wave == 0 && r < p.T) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = part[0][r][4 * g + i];
#pragma unroll
        for (int q = 1; q < half; ++q) v[i] += part[q][r][4 * g + i];
        v[i] = sqrelu(v[i]);
      }
      store_pair(p.hs, p.hs_lo, (int64_t)r * p.Is + 16 * n + 4 * g, v);
    }
    if (n + (int)gridDim.x < nsh) __syncthreads();
  }

  // routed units: wave-slot, + waves of the grid
  const int nb = p.I / 16, total = n_slots * nb, stride = gridDim.x * NWV;
  int u = wave * gridDim.x + blockIdx.x;
  if (u >= total) return;
  constexpr int U = F == Elt::BF16 ? 12 : 2;
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
  Unit cur = resolve(u), nxt = cur;
  bool more = u + stride < total;
  if (more) nxt = resolve(u + stride);
  int b = 0;
  Sum<std::conditional_t<M::narrow, double, float>> sum;   // (bf16 experts' h is kept as a pair)
  // none: the same number of loads, all of the row's start
  auto issue = [&](const Unit& x, int bb, WStep<F>* w, bool none) {
    const int s = none ? 0 : bb * U, to = none ? 0 : p.D;
#pragma unroll
    for (int q = 0; q < U; ++q) load_step<F>(w[q], x.w, x.wx, s + q, to, p.D, g);
  };
  auto step = [&](WStep<F>* wc, WStep<F>* wn) {
    const bool last = b + 1 == nbat;
    Unit src = cur;
    if (last && more) src = nxt;
    // always the same number of loads, so that the wait for a batch leaves the next in flight
    issue(src, last ? 0 : b + 1, wn, last && !more);
    f32x4_t acc = sum.start();
#pragma unroll
    for (int q = 0; q < U; ++q) {
      mask_step<F>(wc[q], b * U + q, p.D, g);
#pragma unroll
      for (int j = 0; j < M::MF; ++j) {
        const int el = (b * U + q) * M::KS + M::k_of(j, g);
        uint4 a;
        if constexpr (XLDS) {
          a = *(const uint4*)(xl + t * ldx + 2 * (b * U + q < steps ? el : ldx / 2 - 8));
        } else {
          a = *(const uint4*)(in + (int64_t)t * p.D + (el < p.D ? el : 0));
          zero_if(el >= p.D, a);
        }
        acc = mul(wfrag<F>(wc[q], j), a, acc);
      }
    }
    sum.take(acc);
    if (!last) {
      ++b;
      return true;
    }
    const bool sel = (emask[cur.e] >> r) & 1;   // bits of tokens below T only
    const int64_t at = ((int64_t)cur.slot * p.T + r) * p.I + cur.n0 + 4 * g;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      auto x = sum.v[i];
      if constexpr (M::narrow) x *= row_scale[t];
      if constexpr (F == Elt::FP8) x *= ((const float*)p.s_up)[(int64_t)cur.e * p.I + cur.n0 + 4 * g + i];
      v[i] = (float)sqrelu(x);
      sum.v[i] = 0;
    }
    if constexpr (!M::narrow) {
      if (sel) store_pair(p.h, p.h_lo, at, v);
    } else {
      const uint32_t lo2 = pack_bf16x2(v[0], v[1]), hi2 = pack_bf16x2(v[2], v[3]);
      if (sel) *(uint2*)(p.h + at) = make_uint2(lo2, hi2);
      // the row's maximum (h >= 0: bf16 bits order as integers)
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
  WStep<F> w0[U], w1[U];
  issue(cur, 0, w0, false);
  for (;;) {
    if (!step(w0, w1)) break;
    if (!step(w1, w0)) break;
  }
}

// ------------------------------------------------------------------------------- 3 down
// Workgroup (n, part): 16 columns of y (or z) over a contiguous share of the list (slot, step) of
// all touched experts, which its waves share evenly, double buffered across slots; the shared
// expert's steps likewise, their loads issued first of all. Parts of a column block go to fp32
// slabs, and the workgroup that ends last adds them in part order (a counter that launch 1
// cleared; nobody waits). 8- and 4-bit experts: the h rows of the share are first turned into e4m3
// codes (as bf16) in LDS, as many slots at a time as fit.
constexpr int kDownWaves = 8;
constexpr int kDownThreads = 64 * kDownWaves;
constexpr int kDownRowsLds = 64 * 1024;
constexpr int kDownShared = 5;   // steps of the shared expert in flight per wave

template <Elt F>
__global__ __launch_bounds__(kDownThreads, 4) void few_down(FewParams p, int cap) {
  using M = Fmt<F>;
  __shared__ float part[kDownWaves][16][17];
  __shared__ int first_row[1024];              // narrow: first code row of a slot of this pass
  extern __shared__ __attribute__((aligned(16))) uint8_t hq[];  // narrow: cap code rows
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int t = min(r, p.T - 1);
  const int n0 = blockIdx.x * 16;
  const int parts = gridDim.y, mine = blockIdx.y;

  // the shared expert's first loads
  const int nss = p.Is && !p.L ? cdiv(p.Is, 32) : 0, sper = cdiv(nss, kDownWaves * parts);
  const int slo = min(nss, (mine * kDownWaves + wave) * sper), shi = min(nss, slo + sper);
  const int send = min(p.Is, shi * 32);
  uint4 sw[kDownShared];
  const uint16_t* shrow = p.hs + (int64_t)t * p.Is;
  const uint16_t* slrow = p.hs_lo + (int64_t)t * p.Is;
  const uint16_t* swrow = p.Ws_down + (int64_t)(n0 + r) * p.Is;
  if (slo < shi) {
#pragma unroll
    for (int q = 0; q < kDownShared; ++q) {
      const int el = (slo + q) * 32 + 8 * g, at = el < send ? el : 0;
      sw[q] = *(const uint4*)(swrow + at);
    }
  }
  const int n_slots = *p.n_slots;
  const int spe = cdiv(p.I, M::KS);      // steps per expert
  const int total = n_slots * spe, share = cdiv(total, parts);
  const int begin = min(total, mine * share), end = min(total, begin + share);
  const int ldh = lds_stride(p.I);
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  auto shared_part = [&]() {
    if (slo >= shi) return;
#pragma unroll
    for (int q = 0; q < kDownShared; ++q) {
      const int el = (slo + q) * 32 + 8 * g, at = el < send ? el : 0;
      uint4 hi = *(const uint4*)(shrow + at), lo = *(const uint4*)(slrow + at);
      zero_if(el >= send, sw[q]);
      zero_if(el >= send, hi);
      zero_if(el >= send, lo);
      sum = mul(__builtin_bit_cast(bf16x8_t, sw[q]), hi, sum);
      sum = mul(__builtin_bit_cast(bf16x8_t, sw[q]), lo, sum);
    }
    Sum<float> rest;
    rest.take(sum);
    dot_rows<2, true>(swrow, shrow, slrow, p.Is, min(shi, slo + kDownShared), shi, g, rest);
    sum = rest.start();
  };

  // one wave's steps [at, stop), in batches of up to U steps of one slot
  constexpr int U = F == Elt::BF16 ? 4 : (F == Elt::MXFP8 ? 1 : 2);
  struct Pos {
    int slot, s, s1;           // batch: steps s .. of the slot, which ends (here) at s1
    const uint8_t *w, *wx;
    const uint16_t *a, *a2;    // bf16: the token's h; narrow: a is its code row in LDS
    float scale;
    bool sel;
    int row;                   // this lane's weight row
  };
  auto enter = [&](int at, int stop, int pass_slot) {   // the batch that starts at step `at`
    Pos x;
    x.slot = at / spe;
    x.s = at - x.slot * spe;
    x.s1 = min(spe, x.s + stop - at);
    const int e = p.slot_e[x.slot];
    const uint32_t mask = p.slot_mask[x.slot];
    x.sel = (mask >> r) & 1;
    // tokens that did not select the expert read another's row (their products are dropped)
    const int src = x.sel ? r : __ffs(mask) - 1;
    x.row = e * p.D + n0 + r;
    x.w = p.W_down + (int64_t)x.row * p.I * M::bits / 8;
    x.wx = M::mx ? (const uint8_t*)p.s_down + (int64_t)x.row * (p.I / 32) : nullptr;
    x.scale = p.gate_m[x.slot * TB + r];
    if constexpr (M::narrow) {
      x.scale *= row_scale_e4m3(__uint_as_float(p.hmax[x.slot * TB + src])).down;
      x.a = (const uint16_t*)(hq + (first_row[x.slot - pass_slot] +
                                    __popc(mask & ((1u << src) - 1))) * ldh);
      x.a2 = nullptr;
    } else {
      x.a = p.h + ((int64_t)x.slot * p.T + src) * p.I;
      x.a2 = p.h_lo + ((int64_t)x.slot * p.T + src) * p.I;
    }
    return x;
  };
  struct Batch {
    WStep<F> w[U];
    uint4 a[M::narrow ? 1 : U], b[M::narrow ? 1 : U];
  };
  // none: the same number of loads, all of the row's start
  auto issue = [&](const Pos& x, Batch& o, bool none) {
    const int kend = none ? 0 : min(p.I, x.s1 * M::KS), s = none ? 0 : x.s;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      load_step<F>(o.w[q], x.w, x.wx, s + q, kend, p.I, g);
      if constexpr (!M::narrow) {
        const int el = (s + q) * M::KS + M::k_of(0, g), at = el < kend ? el : 0;
        o.a[q] = *(const uint4*)(x.a + at);
        o.b[q] = *(const uint4*)(x.a2 + at);
      }
    }
  };
  auto run = [&](int at, int stop, int pass_slot, bool first) {
    if (at >= stop) {
      if (first) shared_part();
      return;
    }
    Pos cur = enter(at, stop, pass_slot);
    Batch b0, b1;
    issue(cur, b0, false);
    if (first) shared_part();
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    auto step = [&](Batch& bc, Batch& bn) {
      const int took = min(U, cur.s1 - cur.s);
      at += took;
      const bool slot_done = cur.s + took == cur.s1, done = at >= stop;
      Pos nxt = cur;
      if (!done && slot_done) nxt = enter(at, stop, pass_slot);
      else if (!done) nxt.s = cur.s + took;
      issue(nxt, bn, done);
      const int kend = min(p.I, cur.s1 * M::KS);
#pragma unroll
      for (int q = 0; q < U; ++q) {
        mask_step<F>(bc.w[q], cur.s + q, kend, g);
#pragma unroll
        for (int j = 0; j < M::MF; ++j) {
          const bf16x8_t w = wfrag<F>(bc.w[q], j);
          if constexpr (M::narrow) {
            const int el = min(cur.s + q, spe - 1) * M::KS + M::k_of(j, g);
            acc = mul(w, *(const uint4*)(cur.a + el), acc);
          } else {
            const bool past = (cur.s + q) * M::KS + M::k_of(0, g) >= kend;
            zero_if(past, bc.a[q]);
            zero_if(past, bc.b[q]);
            acc = mul(w, bc.a[q], acc);
            acc = mul(w, bc.b[q], acc);
          }
        }
        // reads of later steps' codes stay behind (they would only add registers: at most 128, so
        // that two workgroups fit a CU)
        if constexpr (M::narrow) __builtin_amdgcn_sched_barrier(0);
      }
      if (slot_done) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[i] * cur.scale;
          if constexpr (F == Elt::FP8)
            v *= ((const float*)p.s_down)[cur.row - r + 4 * g + i];
          if (cur.sel) sum[i] += v;
          acc[i] = 0.f;
        }
      }
      cur = nxt;
      return !done;
    };
    for (;;) {
      if (!step(b0, b1)) break;
      if (!step(b1, b0)) break;
    }
  };
  if constexpr (!M::narrow) {
    const int per = cdiv(end - begin, kDownWaves);
    const int lo = min(end, begin + wave * per);
    run(lo, min(end, lo + per), 0, true);
  } else {
    bool first = true;
    for (int at = begin; at < end || first;) {
      // slots of this pass: as many as have room (cap >= kFewTokens rows: at least one)
      const int slot0 = at / spe, slot_end = at < end ? cdiv(end, spe) : slot0;
      if (!first) __syncthreads();        // the pass before is done with the code rows
      int rows = 0, n = 0;                // every wave: prefix of the slots' row counts
      for (int s = slot0; s < slot_end; s += 64) {
        const int c = s + lane < slot_end ? __popc(p.slot_mask[s + lane]) : 0;
        int inc = c;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int v = __shfl_up(inc, o);
          if (lane >= o) inc += v;
        }
        const bool fits = s + lane < slot_end && rows + inc <= cap;
        if (fits && wave == 0) first_row[s - slot0 + lane] = rows + inc - c;
        const int k = __popcll(__ballot(fits));
        n += k;
        rows += k ? __shfl(inc, k - 1) : 0;
        if (k < 64) break;
      }
      n = __builtin_amdgcn_readfirstlane(n);
      int j = 0;
      for (int s = slot0; s < slot0 + n; ++s) {
        const uint32_t mask = p.slot_mask[s];
        for (uint32_t m = mask; m; m &= m - 1, ++j) {   // rows dealt to the waves
          if (j % kDownWaves != wave) continue;
          const int tk = __ffs(m) - 1;
          const float inv = row_scale_e4m3(__uint_as_float(p.hmax[s * TB + tk])).up;
          const uint16_t* h = p.h + ((int64_t)s * p.T + tk) * p.I;
          for (int c = lane * 8; c < ldh / 2 - 8; c += 512) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (c < p.I) v = *(const uint4*)(h + c);
            *(uint4*)(hq + j * ldh + 2 * c) = codes8(v, inv);
          }
        }
      }
      __syncthreads();
      const int stop = min(end, (slot0 + n) * spe);
      const int per = cdiv(stop - at, kDownWaves);
      const int lo = min(stop, at + wave * per);
      run(lo, min(stop, lo + per), slot0, first);
      first = false;
      at = stop;
    }
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
    // Release by hand: an agent-scope store is written through to where every die reads it, so the
    // slab is there once the wait below is over, and the statement keeps the compiler from moving
    // the stores past it; then the part is counted. (A release fence would write back the whole
    // L2 too: 18 us more on a Nano-shaped token.) The acquire is the part that reads the slabs: no
    // load of them may go before the count, and none may be served from what this die's caches
    // held earlier.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int before = 0;
    if (lane == 0)
      before = __hip_atomic_fetch_add(p.joined + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__builtin_amdgcn_readfirstlane(before) != parts - 1) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0.f;
    for (int q = 0; q < parts; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] += __hip_atomic_load(slab + q * 256 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (r < p.T) {
    const int64_t at = (int64_t)r * p.D + n0 + 4 * g;
    if (p.L)
      store_pair(p.z, p.z_lo, at, v);
    else
      *(uint2*)(p.y + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// -------------------------------------------------------------------------------- 4 out
__global__ __launch_bounds__(512) void few_out(FewParams p) {
  __shared__ float part[8][16][17];
  dense_unit<8, 4, true>(Dense{p.z, p.z_lo, p.W_out, p.hs, p.hs_lo, p.Ws_down, p.L, p.Is, p.H, p.T,
                               0, p.y, nullptr}, 16 * blockIdx.x, part);
}

template <Elt F, int NPER, bool XLDS>
hipError_t run_up(const FewParams& p, int grid, size_t lds, hipStream_t s) {
  hipLaunchKernelGGL((few_up<F, NPER, XLDS>), dim3(grid), dim3(64 * kUpWaves<F, NPER>), lds, s, p);
  return hipGetLastError();
}
template <Elt F, bool XLDS>
hipError_t run_up(const FewParams& p, int grid, size_t lds, hipStream_t s) {
  if (p.E <= 128) return run_up<F, 2, XLDS>(p, grid, lds, s);
  if (p.E <= 512) return run_up<F, 8, XLDS>(p, grid, lds, s);
  return run_up<F, 16, XLDS>(p, grid, lds, s);
}

template <Elt F>
hipError_t run_down(const FewParams& p, hipStream_t s) {
  int rows = 0;
  if (Fmt<F>::narrow)  // every pair's code row, or what kDownRowsLds holds, but a slot's at least
    rows = std::min(p.T * p.k, std::max(kDownRowsLds / lds_stride(p.I), p.T));
  hipLaunchKernelGGL((few_down<F>), dim3(p.D / 16, few_parts(p.D)), dim3(kDownThreads),
                     (size_t)rows * lds_stride(p.I), s, p, rows);
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
  const size_t lds = (size_t)p.T * lds_stride(p.D);
  if (p.ex != Elt::BF16 && lds > kUpRowsLds) return hipErrorInvalidValue;
  switch (p.ex) {
    case Elt::BF16:
      return lds <= kUpRowsLds ? run_up<Elt::BF16, true>(p, grid, lds, s)
                               : run_up<Elt::BF16, false>(p, grid, 0, s);
    case Elt::FP8: return run_up<Elt::FP8, true>(p, grid, lds, s);
    case Elt::MXFP4: return run_up<Elt::MXFP4, true>(p, grid, lds, s);
    case Elt::MXFP8: return run_up<Elt::MXFP8, true>(p, grid, lds, s);
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
