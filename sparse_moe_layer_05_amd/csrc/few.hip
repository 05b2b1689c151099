// The whole MoE layer for at most 16 tokens ("NVIDIA Nemotron 3: Efficient and Open Intelligence",
// section 2.2, latency-oriented deployment) in three launches, four for LatentMoE.
//
// With so few tokens the layer reads every touched weight once and does almost nothing else, so
// its floor is bytes over HBM bandwidth (a Nano-shaped token in bf16: 160 MB) and its cost beyond
// that is dependent launches. A launch here ends only where every later byte depends on what it
// computed:
//   1 front   router scores; the shared expert's up projection; LatentMoE's u = x W_in^T
//   2 up      selection (by every workgroup, from the scores), then h = relu(W_up u)^2 of the
//             touched experts
//   3 down    y = shared + sum_e g_e W_down[e] h_e: a workgroup owns 16 columns of y over all
//             experts, so the gated sum stays in registers and there is nothing to combine
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
#include <algorithm>

#include "common.hpp"
#include "few.hpp"
#include "topk.hpp"

namespace moe {
namespace {

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
// aload(el) loads the lane's token chunk that starts at element el, aconv turns what it loaded
// into the operand's 16 bytes. U steps of loads are in flight together; chunks past K are read
// from the row's start and zeroed on both sides.
template <Elt F, int U, class ALoad, class AConv>
__device__ __forceinline__ f32x4_t dot_steps(const uint8_t* w, const uint8_t* wx, int K, int s0,
                                             int s1, int g, ALoad aload, AConv aconv,
                                             f32x4_t acc) {
  using M = Fmt<F>;
  using Raw = decltype(aload(0));
  for (int s = s0; s < s1; s += U) {
    uint4 wf[U][M::CW];
    Raw af[U][M::CA];
    int sc[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int k0 = min(s + q, s1 - 1) * M::KS;
#pragma unroll
      for (int c = 0; c < M::CW; ++c) {
        const int el = k0 + M::kw(c, g);
        wf[q][c] = *(const uint4*)(w + (int64_t)(el < K ? el : 0) * M::bits / 8);
      }
#pragma unroll
      for (int c = 0; c < M::CA; ++c) {
        const int el = k0 + M::ka(c, g);
        af[q][c] = aload(el < K ? el : 0);
      }
      if constexpr (M::mx) sc[q] = wx[min(k0 / 32 + g, K / 32 - 1)];
      else sc[q] = 127;
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (s + q >= s1) break;
      const int k0 = (s + q) * M::KS;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 wv[M::CW], av[M::CA];
#pragma unroll
      for (int c = 0; c < M::CW; ++c) wv[c] = k0 + M::kw(c, g) < K ? wf[q][c] : zero;
#pragma unroll
      for (int c = 0; c < M::CA; ++c) av[c] = k0 + M::ka(c, g) < K ? aconv(af[q][c]) : zero;
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

__device__ __forceinline__ uint4 keep(uint4 v) { return v; }

// 16 bf16 -> 16 e4m3 codes of v * inv.
struct Raw16 { uint4 a, b; };
__device__ __forceinline__ uint32_t codes4(uint32_t p, uint32_t q, float inv) {
  return cvt_fp8x2(bf16_bits_to_f32(p & 0xFFFF) * inv, bf16_bits_to_f32(p >> 16) * inv) |
         cvt_fp8x2(bf16_bits_to_f32(q & 0xFFFF) * inv, bf16_bits_to_f32(q >> 16) * inv) << 16;
}
__device__ __forceinline__ uint4 codes16(const Raw16& r, float inv) {
  return make_uint4(codes4(r.a.x, r.a.y, inv), codes4(r.a.z, r.a.w, inv),
                    codes4(r.b.x, r.b.y, inv), codes4(r.b.z, r.b.w, inv));
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
                                  [&](int el) { return *(const uint4*)(row + el); }, keep, acc);
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
// Workgroups [0, E): one expert's logits and scores; then 16 rows each of Ws_up and of W_in.
template <int TT>
__global__ __launch_bounds__(256) void few_front(FewParams p) {
  __shared__ float part[4][16][17];
  __shared__ double red[4][TT];
  const int tid = threadIdx.x;
  const int nr = p.given ? 0 : p.E;
  const int bid = blockIdx.x;
  if (p.hmax) {  // the maxima that launch 2 raises
    const int n = few_slots(p.T, p.E, p.k) * TB;
    for (int i = bid * 256 + tid; i < n; i += gridDim.x * 256) p.hmax[i] = 0;
  }
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
// Units of (touched expert, 16 rows of W_up); a workgroup of 16 waves takes four units at a time,
// four waves splitting K of each. NPER * 64 >= E.
constexpr int kUpWaves = 16;

template <Elt F, int NPER>
__global__ __launch_bounds__(1024) void few_up(FewParams p) {
  using M = Fmt<F>;
  __shared__ int idx_l[TB * 64];
  __shared__ float gates_l[TB * 64];
  __shared__ uint32_t emask[NPER * 64];     // tokens that selected expert e
  __shared__ int slot_l[NPER * 64];         // touched experts, ascending
  __shared__ int cnt[kUpWaves];
  __shared__ float part[2][kUpWaves][16][17];
  __shared__ float row_scale[TB];
  extern __shared__ __attribute__((aligned(16))) uint8_t xq[];  // [T][D + 16] e4m3 (narrow)
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const uint16_t* in = p.L ? p.u : p.x;
  for (int i = tid; i < NPER * 64; i += 1024) emask[i] = 0;
  __syncthreads();

  // selection: wave t, token t
  if (wave < p.T) {
    const int t = wave;
    bool ok = lane < p.k;
    if (p.given) {
      int e = -1;
      if (ok) {
        e = p.idx_in[t * p.k + lane];
        idx_l[t * p.k + lane] = e;
        gates_l[t * p.k + lane] = p.gates_in[t * p.k + lane];
      }
      ok = ok && (unsigned)e < (unsigned)p.E;
      for (int j = 0; j < p.k; ++j)   // a repeated expert: its first slot counts
        if (__shfl(e, j) == e && j < lane) ok = false;
      if (!ok && lane < p.k) idx_l[t * p.k + lane] = -1;
    } else {
      float key[NPER], sc[NPER];
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 64 * i;
        sc[i] = e < p.E ? p.score[(int64_t)t * p.E + e] : 0.f;
        key[i] = e < p.E ? sc[i] + p.b[e] : 0.f;
      }
      select_topk<NPER, true>(key, sc, lane, p.E, p.k, idx_l + t * p.k, gates_l + t * p.k);
    }
    if (ok) atomicOr(&emask[idx_l[t * p.k + lane]], 1u << t);
  }
  // 8- and 4-bit experts: this wave's token row in e4m3, scale amax / 448 (1 for a zero row)
  const int ldq = p.D + 16;
  if constexpr (M::narrow) {
    if (wave < p.T) {
      const uint16_t* row = in + (int64_t)wave * p.D;
      float m = 0.f;
      auto each = [&](uint4 v, auto f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f(w[i]);
      };
      for (int c = lane * 8; c < p.D; c += 512)
        each(*(const uint4*)(row + c), [&](uint32_t w) {
          m = fmaxf(m, fmaxf(fabsf(bf16_bits_to_f32(w & 0xFFFF)), fabsf(bf16_bits_to_f32(w >> 16))));
        });
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
      const float inv = m > 0.f ? 448.f / m : 1.f;
      if (lane == 0) row_scale[wave] = m > 0.f ? m / 448.f : 1.f;
      for (int c = lane * 8; c < p.D; c += 512) {
        const uint4 v = *(const uint4*)(row + c);
        *(uint2*)(xq + wave * ldq + c) = make_uint2(codes4(v.x, v.y, inv), codes4(v.z, v.w, inv));
      }
    }
  }
  __syncthreads();
  // touched experts, ascending
  const uint32_t em = wave < NPER ? emask[wave * 64 + lane] : 0;
  const uint64_t any = __ballot(em != 0);
  if (lane == 0) cnt[wave] = __popcll(any);
  __syncthreads();
  int base = 0, n_slots = 0;
#pragma unroll
  for (int i = 0; i < kUpWaves; ++i) {
    base += i < wave ? cnt[i] : 0;
    n_slots += cnt[i];
  }
  if (em) slot_l[base + __popcll(any & ((1ull << lane) - 1))] = wave * 64 + lane;
  __syncthreads();
  if (blockIdx.x == 0) {  // what launch 3 and the caller read
    if (tid == 0) *p.n_slots = n_slots;
    for (int i = tid; i < n_slots; i += 1024) {
      p.slot_e[i] = slot_l[i];
      p.slot_mask[i] = emask[slot_l[i]];
    }
    for (int i = tid; i < n_slots * TB; i += 1024) {
      const int e = slot_l[i / TB], t = i % TB;
      float v = 0.f;
      if (t < p.T)
        for (int j = p.k - 1; j >= 0; --j)
          if (idx_l[t * p.k + j] == e) v = gates_l[t * p.k + j];
      p.gate_m[i] = v;
    }
    if (!p.given)
      for (int i = tid; i < p.T * p.k; i += 1024) {
        p.idx[i] = idx_l[i];
        p.gates[i] = gates_l[i];
      }
  }

  const int nb = p.I / 16, total = n_slots * nb;
  const int grp = wave >> 2, kw = wave & 3;
  const int steps = cdiv(p.D, M::KS), per = cdiv(steps, 4);
  const int lo = min(steps, kw * per), hi = min(steps, lo + per);
  const int t = min(r, p.T - 1);
  int par = 0;
  for (int first = 0; first < total; first += gridDim.x * 4, par ^= 1) {
    const int unit = first + grp * gridDim.x + blockIdx.x;
    const bool live = unit < total;
    const int slot = live ? unit / nb : 0, n0 = live ? (unit % nb) * 16 : 0;
    const int e = slot_l[slot];
    const int64_t row = (int64_t)e * p.I + n0 + r;
    if (live) {
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      const uint8_t* w = p.W_up + row * p.D * M::bits / 8;
      const uint8_t* wx = M::mx ? (const uint8_t*)p.s_up + row * (p.D / 32) : nullptr;
      if constexpr (M::narrow)
        acc = dot_steps<F, 3>(w, wx, p.D, lo, hi, g,
                              [&](int el) { return *(const uint4*)(xq + t * ldq + el); }, keep, acc);
      else
        acc = dot_steps<F, 7>(w, wx, p.D, lo, hi, g,
                              [&](int el) { return *(const uint4*)(in + (int64_t)t * p.D + el); },
                              keep, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i) part[par][wave][r][4 * g + i] = acc[i];
    }
    __syncthreads();
    if (live && kw == 0) {
      const bool sel = (emask[e] >> r) & 1;   // bits of tokens below T only
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = part[par][wave][r][4 * g + i];
#pragma unroll
        for (int q = 1; q < 4; ++q) v[i] += part[par][wave + q][r][4 * g + i];
        if constexpr (F == Elt::FP8)
          v[i] *= row_scale[t] * ((const float*)p.s_up)[(int64_t)e * p.I + n0 + 4 * g + i];
        else if constexpr (M::mx)
          v[i] *= row_scale[t];
        v[i] = sqrelu(v[i]);
      }
      const uint32_t lo2 = pack_bf16x2(v[0], v[1]), hi2 = pack_bf16x2(v[2], v[3]);
      if (sel) *(uint2*)(p.h + ((int64_t)slot * p.T + r) * p.I + n0 + 4 * g) = make_uint2(lo2, hi2);
      if constexpr (M::narrow) {  // the row's maximum (h >= 0: bf16 bits order as integers)
        uint32_t m = max(max(lo2 << 16, lo2 & 0xFFFF0000u), max(hi2 << 16, hi2 & 0xFFFF0000u));
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (sel && g == 0) atomicMax(p.hmax + slot * TB + r, m);
      }
    }
  }
}

// ------------------------------------------------------------------------------- 3 down
// A workgroup owns 16 columns of y (or z). Its waves share the routed steps of all touched experts
// evenly, in one contiguous range each, and the shared expert's steps likewise.
constexpr int kDownWaves = 16;

template <Elt F>
__global__ __launch_bounds__(1024) void few_down(FewParams p) {
  using M = Fmt<F>;
  __shared__ float part[kDownWaves][16][17];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int t = min(r, p.T - 1);
  const int n0 = blockIdx.x * 16;
  const int n_slots = *p.n_slots;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  if (p.Is && !p.L) {
    const int steps = cdiv(p.Is, 32), per = cdiv(steps, kDownWaves);
    const int lo = min(steps, wave * per), hi = min(steps, lo + per);
    const uint16_t* row = p.hs + (int64_t)t * p.Is;
    sum = dot_steps<Elt::BF16, 8>((const uint8_t*)(p.Ws_down + (int64_t)(n0 + r) * p.Is), nullptr,
                                  p.Is, lo, hi, g,
                                  [&](int el) { return *(const uint4*)(row + el); }, keep, sum);
  }
  const int spe = cdiv(p.I, M::KS);      // steps per expert
  const int total = n_slots * spe, per = cdiv(total, kDownWaves);
  int at = min(total, wave * per);
  const int end = min(total, at + per);
  while (at < end) {
    const int slot = at / spe, s0 = at - slot * spe, s1 = min(spe, s0 + end - at);
    at += s1 - s0;
    const int e = p.slot_e[slot];
    const int64_t row = (int64_t)e * p.D + n0 + r;
    const bool sel = (p.slot_mask[slot] >> r) & 1;
    const float gate = p.gate_m[slot * TB + r];
    // rows that launch 2 did not write are read as another token's (their products are dropped)
    const int src = __ffs(p.slot_mask[slot]) - 1;
    const uint16_t* h = p.h + ((int64_t)slot * p.T + (sel ? r : src)) * p.I;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    const uint8_t* w = p.W_down + row * p.I * M::bits / 8;
    const uint8_t* wx = M::mx ? (const uint8_t*)p.s_down + row * (p.I / 32) : nullptr;
    float scale = gate;
    if constexpr (M::narrow) {
      const float m = __uint_as_float(p.hmax[slot * TB + (sel ? r : src)]);
      const float inv = m > 0.f ? 448.f / m : 1.f;
      scale *= m > 0.f ? m / 448.f : 1.f;
      acc = dot_steps<F, 2>(w, wx, p.I, s0, s1, g,
                            [&](int el) {
                              return Raw16{*(const uint4*)(h + el), *(const uint4*)(h + el + 8)};
                            },
                            [&](const Raw16& v) { return codes16(v, inv); }, acc);
    } else {
      acc = dot_steps<F, 8>(w, wx, p.I, s0, s1, g,
                            [&](int el) { return *(const uint4*)(h + el); }, keep, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = acc[i] * scale;
      if constexpr (F == Elt::FP8)
        v *= ((const float*)p.s_down)[(int64_t)e * p.D + n0 + 4 * g + i];
      if (sel) sum[i] += v;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][r][4 * g + i] = sum[i];
  __syncthreads();
  if (tid < 64 && r < p.T) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = part[0][r][4 * g + i];
#pragma unroll
      for (int q = 1; q < kDownWaves; ++q) v[i] += part[q][r][4 * g + i];
    }
    uint16_t* out = p.L ? p.z : p.y;
    *(uint2*)(out + (int64_t)r * p.D + n0 + 4 * g) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// -------------------------------------------------------------------------------- 4 out
__global__ __launch_bounds__(512) void few_out(FewParams p) {
  __shared__ float part[8][16][17];
  dense_unit<8, 8>(Dense{p.z, p.W_out, p.hs, p.Ws_down, p.L, p.Is, p.H, p.T, 0, p.y},
                   16 * blockIdx.x, part);
}

template <Elt F>
hipError_t run_up(const FewParams& p, int grid, hipStream_t s) {
  const size_t lds = Fmt<F>::narrow ? (size_t)p.T * (p.D + 16) : 0;
  if (p.E <= 128) hipLaunchKernelGGL((few_up<F, 2>), dim3(grid), dim3(1024), lds, s, p);
  else if (p.E <= 512) hipLaunchKernelGGL((few_up<F, 8>), dim3(grid), dim3(1024), lds, s, p);
  else hipLaunchKernelGGL((few_up<F, 16>), dim3(grid), dim3(1024), lds, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_front(const FewParams& p, hipStream_t s) {
  if (p.T < 1 || p.T > kFewTokens) return hipErrorInvalidValue;
  const int front = (p.given ? 0 : p.E) + p.Is / 16 + p.L / 16;
  if (front == 0 && !p.hmax) return hipSuccess;
  const dim3 grid(std::max(front, 1)), block(256);
  if (p.T == 1) hipLaunchKernelGGL((few_front<1>), grid, block, 0, s, p);
  else if (p.T <= 4) hipLaunchKernelGGL((few_front<4>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((few_front<16>), grid, block, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_few_up(const FewParams& p, hipStream_t s) {
  // one workgroup per CU; fewer when all the units there can be need fewer
  const int64_t units = (int64_t)few_slots(p.T, p.E, p.k) * (p.I / 16);
  const int grid = (int)std::min<int64_t>(256, (units + 3) / 4);
  switch (p.ex) {
    case Elt::BF16: return run_up<Elt::BF16>(p, grid, s);
    case Elt::FP8: return run_up<Elt::FP8>(p, grid, s);
    case Elt::MXFP4: return run_up<Elt::MXFP4>(p, grid, s);
    case Elt::MXFP8: return run_up<Elt::MXFP8>(p, grid, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_few_down(const FewParams& p, hipStream_t s) {
  const dim3 grid(p.D / 16), block(64 * kDownWaves);
  switch (p.ex) {
    case Elt::BF16: hipLaunchKernelGGL((few_down<Elt::BF16>), grid, block, 0, s, p); break;
    case Elt::FP8: hipLaunchKernelGGL((few_down<Elt::FP8>), grid, block, 0, s, p); break;
    case Elt::MXFP4: hipLaunchKernelGGL((few_down<Elt::MXFP4>), grid, block, 0, s, p); break;
    case Elt::MXFP8: hipLaunchKernelGGL((few_down<Elt::MXFP8>), grid, block, 0, s, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_few_out(const FewParams& p, hipStream_t s) {
  hipLaunchKernelGGL(few_out, dim3(p.H / 16), dim3(512), 0, s, p);
  return hipGetLastError();
}

}  // namespace moe
