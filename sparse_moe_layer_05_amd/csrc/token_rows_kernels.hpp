// Token rows into expert order and back, with weights, and the gradients of both (gfx950).
//
//   spread      out[pos[t, j]] = w[t, j] in[t]                 (sort; its inverse's gradient)
//   gather      out[t] = add[t] + sum_j w[t, j] in[pos[t, j]]  (back; the sort's gradient)
//   dots        dw[t, j] = <a[t], b[pos[t, j]]>                (gradient of the weights, with either)
//
// All are bound by HBM: a token's row is read or written once, its k rows once each. A wave takes
// 512 columns of one token, eight elements a lane, and walks the token's k rows in batches of up to eight,
// of whose loads the compiler keeps some or all in flight (gather_kernel, token_kernel). Rows are buffers
// of their own (RowBuffer): a dropped pair's has no size, so no lane branches.
// Measured (a copy of 4 GiB reaches 4.7 TB/s): spread of 8192 tokens to 6 experts, 2688 bf16 columns,
// 51 us, 6.1 TB/s; gated sum of 1001 tokens, 24 slots a quarter of them kept, 1024 fp32 columns, 7.2 us,
// 4.3 TB/s; gradients of the gated sum, 4096 tokens, 24 slots, 1024 bf16 columns, 86 us, 4.8 TB/s.
// Included once, by routing.hip.
#pragma once

#include "common.hpp"
#include "row8.hpp"
#include "token_rows.hpp"

#include <algorithm>

namespace moe {
namespace {
namespace token_rows {

constexpr int kSeg = 8 * kWave;   // columns of a wave
constexpr int kMostBatch = 8;     // rows in flight

// A token's k positions and weights, one a lane; -1 and 0 where the pair is dropped (its row is then
// a buffer of no size: it loads as zeros and stores nothing).
struct Pairs {
  int pos;
  float w;
};
__device__ __forceinline__ Pairs load_pairs(const TokenRows& p, int t, int lane) {
  Pairs q{-1, 0.f};
  if (lane < p.k) {
    const int64_t i = (int64_t)t * p.k + lane;
    const int r = p.pos[i];
    const float w = p.weights ? p.weights[i] : 1.f;
    if ((unsigned)r < (unsigned)p.n_rows) q = {r, w};
  }
  return q;
}
__device__ __forceinline__ int pos_of(const Pairs& q, int j) {
  return __builtin_amdgcn_readlane(q.pos, j);
}
__device__ __forceinline__ float weight_of(const Pairs& q, int j) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(q.w), j));
}

// A wave's unit: 512 columns of one token.
struct Unit {
  int t, lane;
  uint32_t col;   // the lane's first column; past the row's end for the last lanes
  __device__ __forceinline__ Unit(const TokenRows& p, int64_t unit) {
    const int nseg = (p.D + kSeg - 1) / kSeg;
    lane = threadIdx.x & 63;
    t = (int)(unit / nseg);
    col = (uint32_t)(unit - (int64_t)t * nseg) * kSeg + lane * 8;
  }
};
__device__ __forceinline__ int64_t unit_of_wave() {
  return (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// A wave stores its columns to every row of the token: each row is read once, and nothing waits for
// the stores. STREAM: they go past the caches (past_cache below).
template <Elt T, bool WEIGHTED, bool STREAM>
__global__ __launch_bounds__(256) void spread_kernel(TokenRows p, const void* in, void* out) {
  const Unit u(p, unit_of_wave());
  if (u.t >= p.T) return;
  const Pairs pr = load_pairs(p, u.t, u.lane);
  Raw8<T> r = RowBuffer<T>(in, u.t, 1, p.D).load(u.col);
  float v[8];
  if constexpr (WEIGHTED) unpack8<T>(r, v);
  for (int j = 0; j < p.k; ++j) {
    const int row = pos_of(pr, j);
    if constexpr (WEIGHTED) {
      const float w = weight_of(pr, j);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = w * v[i];
      r = pack8<T>(x);
    }
    RowBuffer<T>(out, row, row >= 0, p.D).template store<STREAM>(u.col, r);
  }
}

// Positions from the dispatch's chunk counts [nch][E] (dispatch_count): a workgroup per chunk of CH
// tokens adds up, for every expert, the chunks before its own and all of them, which takes the place
// of a launch that scans them; the rest is a chunk's own masks. Latency bound (8192 tokens, 6 of 128:
// count 4.7 us, place 4.9; with the scan 4.7 + 6.0 + 5.8).
constexpr int kPlaceThreads = 1024;
template <int CH>
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(const int32_t* __restrict__ idx, int T,
                                                              int E, int k,
                                                              const int32_t* __restrict__ ccount,
                                                              int nch, int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ pos) {
  extern __shared__ uint32_t mask[];   // [CH / 32][E]
  __shared__ int32_t total[1024], start[1024];   // start: pairs of lower chunks, then first row
  __shared__ int32_t sums[kPlaceThreads / 64];
  __shared__ uint64_t valid[CH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, chunk = blockIdx.x;
  for (int e = tid; e < 1024; e += kPlaceThreads) total[e] = start[e] = 0;
  for (int i = tid; i < E * (CH / 32); i += kPlaceThreads) mask[i] = 0;
  __syncthreads();
  // several groups of threads share an expert's chunks (whole numbers: their order is free)
  const int lg = 32 - __clz(max(E - 1, 1));   // log2 of the experts rounded up
  const int e0 = tid & ((1 << lg) - 1), group = tid >> lg, groups = kPlaceThreads >> lg;
  if (e0 < E) {
    int all = 0, before = 0;
    for (int c0 = group; c0 < nch; c0 += 8 * groups) {
      int v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * groups;
        v[i] = c < nch ? ccount[(int64_t)c * E + e0] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        all += v[i];
        if (c0 + i * groups < chunk) before += v[i];
      }
    }
    atomicAdd(&total[e0], all);
    atomicAdd(&start[e0], before);
  }
  // the chunk's masks, a token a thread: a repeated expert of a token is dropped
  if (tid < CH) {
    const int t = chunk * CH + tid;
    uint64_t kept = 0;
    if (t < T) {
      const uint32_t bit = 1u << (tid & 31);
      for (int j0 = 0; j0 < k; j0 += 8) {
        int ev[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) ev[i] = j0 + i < k ? idx[(int64_t)t * k + j0 + i] : -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if ((unsigned)ev[i] >= (unsigned)E) continue;
          const uint32_t old = atomicOr(&mask[(tid >> 5) * E + ev[i]], bit);
          if (!(old & bit)) kept |= 1ull << (j0 + i);
        }
      }
    }
    valid[tid] = kept;
  }
  __syncthreads();
  // the running sum over the experts (kPlaceThreads >= 1024 >= E)
  const int mine = total[tid];
  int up = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(up, d);
    if (lane >= d) up += o;
  }
  if (lane == 63) sums[wave] = up;
  __syncthreads();
  int base = up - mine;
  for (int w = 0; w < wave; ++w) base += sums[w];
  start[tid] += base;
  if (chunk == 0) {
    if (tid < E) offsets[tid] = base;
    if (tid == E - 1) offsets[E] = base + mine;
  }
  __syncthreads();
  const int pairs = min(CH, T - chunk * CH) * k;
  for (int i = tid; i < pairs; i += kPlaceThreads) {
    const int t = i / k, j = i - t * k;
    const int64_t at = (int64_t)chunk * CH * k + i;
    int row = -1;
    if (valid[t] >> j & 1) {
      const int e = idx[at], w = t >> 5;
      row = start[e] + __popc(mask[w * E + e] & ((1u << (t & 31)) - 1));
      for (int q = 0; q < w; ++q) row += __popc(mask[q * E + e]);
    }
    pos[at] = row;
  }
}

// The rows of the pairs [j0, j0 + B), and acc += their weights times them.
template <Elt ROWS, int B, bool STREAM>
__device__ __forceinline__ void load_batch(const TokenRows& p, const Pairs& pr, const void* rows,
                                           int j0, uint32_t col, Raw8<ROWS> (&r)[B]) {
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int row = pos_of(pr, j0 + b);   // (j0 + b < 64; lanes past k hold -1 and 0)
    r[b] = RowBuffer<ROWS>(rows, row, row >= 0, p.D).template load<STREAM>(col);
  }
}
template <Elt ROWS, int B>
__device__ __forceinline__ void add_rows(const Pairs& pr, int j0, const Raw8<ROWS> (&r)[B],
                                         float (&acc)[8]) {
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const float w = weight_of(pr, j0 + b);
    float v[8];
    unpack8<ROWS>(r[b], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
  }
}

// The gated sum where units fill the chip: batches of B rows, fp32 sums in slot order, one rounding. As
// compiled a batch's loads are in flight together where the result is fp32 and for eight bf16 rows to
// bf16; two or four of them, and fp32 rows to bf16 (22 registers for any B), are waited for one row after
// another, which the eight waves of a SIMD hide where tokens are many. Microseconds (TB/s), bf16, 2688
// columns: 8192 tokens, 6 slots 52 (6.0), 12288, 4 59 (5.7), 16384, 2 50 (5.4); fp32 rows to bf16, 4096, 24,
// 1024 columns 73 (5.8).
template <Elt IN, Elt OUT, int B, bool STREAM>
__global__ __launch_bounds__(256) void gather_kernel(TokenRows p, const void* in, const void* add,
                                                     void* out) {
  const Unit u(p, unit_of_wave());
  if (u.t >= p.T) return;
  const Pairs pr = load_pairs(p, u.t, u.lane);
  float acc[8];
  unpack8<OUT>(RowBuffer<OUT>(add, u.t, 1, p.D).load(u.col), acc);
  for (int j0 = 0; j0 < p.k; j0 += B) {
    Raw8<IN> r[B];
    load_batch<IN, B, STREAM>(p, pr, in, j0, u.col, r);
    add_rows<IN, B>(pr, j0, r, acc);
  }
  RowBuffer<OUT>(out, u.t, 1, p.D).store(u.col, pack8<OUT>(acc));
}

// Few pairs: positions and the spread in one launch. Every workgroup finds its own token's positions
// from all the pairs (a pair's place is the number of kept pairs of lower experts, and of its own
// expert before it); the workgroup behind the last token counts the offsets. Latency bound: one
// token to 6 experts 4.5 us, of which the launch is about two.
template <Elt T, bool WEIGHTED>
__global__ __launch_bounds__(256) void sort_small_kernel(const int32_t* __restrict__ idx,
                                                         const float* __restrict__ weights, int Tn,
                                                         int D, int E, int k,
                                                         const void* __restrict__ in,
                                                         void* __restrict__ out,
                                                         int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ pos) {
  __shared__ int16_t ex[kSortSmallPairs];
  __shared__ int32_t part[4][64];
  __shared__ int32_t hist[1024];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int P = Tn * k, t = blockIdx.x;
  constexpr int kSlots = kSortSmallPairs / 256;
  // the token's first columns are on their way meanwhile
  const int first_c = (blockIdx.y * 256 + tid) * 8;
  Raw8<T> r0 = zero8<T>();
  if (t < Tn && first_c < D) r0 = load8<T>(in, (int64_t)t * D + first_c);
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int p = q * 256 + tid;
    const int e = p < P ? idx[p] : -1;
    ex[p] = (int16_t)((unsigned)e < (unsigned)E ? e : -1);
  }
  __syncthreads();
  int keep[kSlots];
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int p = q * 256 + tid;
    int e = ex[p];
    if (p < P && e >= 0) {
      const int first = p / k * k;
      bool repeated = false;
      for (int j = first; j < p; ++j) repeated |= ex[j] == e;
      if (repeated) e = -1;
    }
    keep[q] = e;
  }
  if (t == Tn) {
    if (blockIdx.y) return;
    // offsets: a count per expert, then their running sum
    for (int e = tid; e < 1024; e += 256) hist[e] = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSlots; ++q)
      if (keep[q] >= 0) atomicAdd(&hist[keep[q]], 1);   // whole numbers: any order
    __syncthreads();
    int c[4], s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) { c[i] = s; s += hist[tid * 4 + i]; }
    int up = s;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(up, d);
      if (lane >= d) up += o;
    }
    if (lane == 63) part[0][wave] = up;
    __syncthreads();
    int base = up - s;
    for (int w = 0; w < wave; ++w) base += part[0][w];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (tid * 4 + i < E) offsets[tid * 4 + i] = base + c[i];
    if (tid == 255) offsets[E] = base + s;
    return;
  }
  // counts of this token's slots: wave by wave, then over the waves
  for (int j = 0; j < k; ++j) {
    const int me = t * k + j, e = ex[me];
    int n = 0;
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      if (q * 256 >= P) break;
      const int p = q * 256 + tid, v = keep[q];
      n += __popcll(__ballot(v >= 0 && (v < e || (v == e && p < me))));
    }
    if (lane == 0) part[wave][j] = n;
  }
  __shared__ int32_t at[64];
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {   // which of the token's pairs are kept
    const int p = q * 256 + tid;
    if (p >= t * k && p < t * k + k) at[p - t * k] = keep[q];
  }
  __syncthreads();
  if (tid < k) {
    const int place = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
    const int row = at[tid] >= 0 ? place : -1;
    if (blockIdx.y == 0) pos[(int64_t)t * k + tid] = row;
    at[tid] = row;
  }
  __syncthreads();
  for (int c = first_c; c < D; c += gridDim.y * (256 * 8)) {
    Raw8<T> r = c == first_c ? r0 : load8<T>(in, (int64_t)t * D + c);
    float v[8];
    if constexpr (WEIGHTED) unpack8<T>(r, v);
    for (int j = 0; j < k; ++j) {
      const int row = at[j];
      if (row < 0) continue;
      if constexpr (WEIGHTED) {
        const float w = weights[(int64_t)t * k + j];
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = w * v[i];
        r = pack8<T>(u);
      }
      store8<T>(out, (int64_t)row * D + c, r);
    }
  }
}

// A workgroup per token: `segs` waves share its columns (wave v takes v * 512 + n * segs * 512), and
// `cuts` of each share its pairs (eight at a time in turn), where tokens are too few to fill the chip.
// What the cuts of a column add up to, and the waves' shares of a dot product, are joined through
// LDS in wave order. As compiled Gather and SpreadDot have a batch's loads in flight; GatherDot, whose
// dot products are reduced meanwhile, two or three of eight bf16 rows and four of six, fp32 rows two or
// three.
// Microseconds with cuts / without (24 slots, 1024 columns, two units a token; gated sum, the sort's
// gradients, its own): bf16, 250 tokens 3.5 / 4.1, 4.5 / 5.7, 6.1 / 7.4; 500 4.6 / 4.4, 6.0 / 7.9,
// 9.3 / 10.0; 1001 9.8 / 9.2, 10.8 / 10.5, 16.9 / 17.1; 2000 17.4 / 17.4, 19.6 / 18.1, 32.5 / 31.7; 4000
// 32.5 / 33.0, 33.4 / 34.4, 65 / 66. A quarter of the pairs kept: bf16, 1001 5.6 / 5.0, 7.1 / 7.5, 8.0 / 8.9;
// 4000 15.6 / 11.8, 21.9 / 18.2, 28.3 / 24.7; fp32 rows, 1001 6.4 / 6.2, 7.6 / 8.2, 11.8 / 11.3; 4000
// 19.5 / 30.6, 34.9 / 33.0, 49 / 50.
enum class Pass { Gather, GatherDot, SpreadDot, Spread };
constexpr int kMostWaves = 16;
// Gather, GatherDot: out[t] = add[t] + sum_j w rows[pos] (add, out: IN). SpreadDot: out[pos] = w a[t]
// (a: IN, out: ROWS). Dots: dweights[t, j] = <a[t], rows[pos]> (a: ROWS in GatherDot).
template <Elt IN, Elt ROWS, Pass PASS, int B, bool STREAM>
__global__ __launch_bounds__(kMostWaves * 64) void token_kernel(TokenRows p, int segs, int cuts,
                                                                const void* a, const void* rows,
                                                                const void* add, void* out,
                                                                float* dweights) {
  constexpr bool kDot = PASS != Pass::Gather, kSpread = PASS == Pass::SpreadDot;
  constexpr Elt AT = kSpread ? IN : ROWS;
  __shared__ float part[kDot ? kMostWaves : 1][64];
  extern __shared__ float4 sums[];   // [waves][2][64], where pairs are cut
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int seg = wave % segs, cut = wave / segs;
  const int t = blockIdx.x;
  const Pairs pr = load_pairs(p, t, lane);
  float dot = 0.f;   // of pair `lane`
  for (int c0 = 0; c0 < p.D; c0 += segs * kSeg) {
    const uint32_t col = c0 + seg * kSeg + lane * 8;   // past the row's end: zeros
    float av[8], acc[8] = {};
    if constexpr (kDot) unpack8<AT>(RowBuffer<AT>(a, t, 1, p.D).load(col), av);
    for (int j0 = cut * B; j0 < p.k; j0 += cuts * B) {
      Raw8<ROWS> r[B];
      load_batch<ROWS, B, STREAM>(p, pr, rows, j0, col, r);
      if constexpr (!kSpread) add_rows<ROWS, B>(pr, j0, r, acc);
      if constexpr (kDot) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
          float v[8], d = 0.f;
          unpack8<ROWS>(r[b], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) d = fmaf(av[i], v[i], d);
          d = wave_sum(d);
          if (lane == j0 + b) dot += d;
        }
      }
      if constexpr (kSpread) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int row = pos_of(pr, j0 + b);
          const float w = weight_of(pr, j0 + b);
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = w * av[i];
          RowBuffer<ROWS>(out, row, row >= 0, p.D).store(col, pack8<ROWS>(v));
        }
      }
    }
    if constexpr (!kSpread) {
      if (cuts > 1) {
        if (cut) {
          sums[wave * 128 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
          sums[wave * 128 + 64 + lane] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        }
        __syncthreads();
        if (cut == 0)
          for (int q = 1; q < cuts; ++q) {
            const int from = (seg + q * segs) * 128 + lane;
            const float4 x = sums[from], y = sums[from + 64];
            acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
            acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
          }
        __syncthreads();
      }
      if (cut == 0) {
        float v[8];
        unpack8<IN>(RowBuffer<IN>(add, t, 1, p.D).load(col), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[i];
        RowBuffer<IN>(out, t, 1, p.D).store(col, pack8<IN>(acc));
      }
    }
  }
  if constexpr (kDot) {
    part[wave][lane] = dot;
    __syncthreads();
    if (wave == 0 && lane < p.k) {
      float d = 0.f;
      for (int v = 0; v < segs * cuts; ++v) d += part[v][lane];
      dweights[(int64_t)t * p.k + lane] = pr.pos >= 0 ? d : 0.f;
    }
  }
}

// Many tokens of short rows: L lanes hold a token's row (8 L columns at most), 64 / L tokens a wave, so
// that no lane idles; four pairs in flight, nothing to join.
constexpr int kNarrowBatch = 4;
template <Elt IN, Elt ROWS, Pass PASS, int L>
__global__ __launch_bounds__(256) void narrow_kernel(TokenRows p, const void* a, const void* rows,
                                                     const void* add, void* out, float* dweights) {
  constexpr bool kSpread = PASS == Pass::Spread || PASS == Pass::SpreadDot;
  constexpr bool kDot = PASS == Pass::GatherDot || PASS == Pass::SpreadDot;
  constexpr Elt AT = kSpread ? IN : ROWS;
  constexpr int B = kNarrowBatch;
  const int lane = threadIdx.x & (L - 1), col = lane * 8;
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  if (t >= p.T) return;   // whole groups of lanes
  const bool in_row = col < p.D;
  Raw8<AT> ar = zero8<AT>();
  if ((kSpread || kDot) && in_row) ar = load8<AT>(a, t * p.D + col);
  float av[8], acc[8] = {};
  unpack8<AT>(ar, av);
  if (!kSpread && add && in_row) unpack8<IN>(load8<IN>(add, t * p.D + col), acc);
  for (int j0 = 0; j0 < p.k; j0 += B) {
    int r[B];
    float w[B];
    Raw8<ROWS> x[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      r[b] = j0 + b < p.k ? p.pos[t * p.k + j0 + b] : -1;
      w[b] = j0 + b < p.k && p.weights ? p.weights[t * p.k + j0 + b] : 1.f;
      if ((unsigned)r[b] >= (unsigned)p.n_rows) r[b] = -1;
      x[b] = zero8<ROWS>();
    }
    if constexpr (PASS != Pass::Spread) {
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (r[b] >= 0 && in_row) x[b] = load8<ROWS>(rows, (int64_t)r[b] * p.D + col);
    }
    float dots = 0.f;
#pragma unroll
    for (int b = 0; b < B; ++b) {
      float v[8];
      unpack8<ROWS>(x[b], v);
      if constexpr (kDot) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) d = fmaf(av[i], v[i], d);
        d = group_sum<L>(d);
        if (lane == b) dots = r[b] >= 0 ? d : 0.f;
      }
      if constexpr (kSpread) {
        if (r[b] >= 0 && in_row) {
          if (PASS == Pass::Spread && !p.weights) {   // IN is ROWS: the bits as they are
            store8<IN>(out, (int64_t)r[b] * p.D + col, ar);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = w[b] * av[i];
            store8<ROWS>(out, (int64_t)r[b] * p.D + col, pack8<ROWS>(v));
          }
        }
      } else {
        const float u = r[b] >= 0 ? w[b] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(u, v[i], acc[i]);
      }
    }
    if (kDot && lane < B && j0 + lane < p.k) dweights[t * p.k + j0 + lane] = dots;
  }
  if (!kSpread && in_row) store8<IN>(out, t * p.D + col, pack8<IN>(acc));
}

int64_t units_of(const TokenRows& p) { return (int64_t)p.T * ((p.D + kSeg - 1) / kSeg); }
dim3 seg_grid(const TokenRows& p) { return dim3((unsigned)((units_of(p) + 3) / 4)); }
// Rows of a batch: absent ones cost their instructions, so few slots take a smaller one.
// Microseconds of the code as compiled (2688 columns; gated sum, the sort's gradients, the gated sum's): 2
// slots, 16384 tokens, eight / two 62 / 53, 103 / 77 and 107 / 76; 6 slots, 8192 tokens, eight / six 55 / 59,
// 62 / 58 and 115 / 118; the sort's gradients of 5 slots 62 / 59, of fp32 113 / 111.
int batch_of(int k, Pass pass) {
  if (pass == Pass::GatherDot && (k == 5 || k == 6)) return 6;
  return k <= 2 ? 2 : k <= 4 ? 4 : kMostBatch;
}
// What together passes the last-level cache (256 MB) is read, or for the sort written, past it: sort of
// 8192 tokens to 6 experts, 2688 columns (308 MB) 60 / 69 us, back 55 / 63, the sort's gradients 60 / 71. Smaller results are left to
// the call that reads them next.
bool past_cache(const TokenRows& p, Elt a, Elt rows, int row_passes) {
  auto bytes = [](Elt t) { return t == Elt::BF16 ? 2 : 4; };
  return (int64_t)p.T * p.D * (bytes(a) + (int64_t)p.k * bytes(rows) * row_passes) > (int64_t)256 << 20;
}
// Units that fill the chip with eight waves a SIMD: with as many, pairs are not cut. From about 2000 units
// on (token_kernel's figures) cutting pays for the gated sum of fp32 rows alone, most where few pairs are
// kept (half as long again without), while bf16 rows then lose up to a third by it.
constexpr int64_t kFull = 8192;
struct Waves {
  int segs, cuts;
};
Waves token_waves(const TokenRows& p) {
  const int nseg = (p.D + kSeg - 1) / kSeg, nbatch = (p.k + kMostBatch - 1) / kMostBatch;
  const int segs = std::min(nseg, 8);
  return {segs, units_of(p) >= kFull ? 1 : std::min(nbatch, kMostWaves / segs)};
}

}  // namespace token_rows
}  // namespace

using namespace token_rows;

namespace {
// Short rows of many tokens go to narrow_kernel: with fewer tokens, cutting their pairs over waves gives
// more of them. Microseconds of the gated sum and of the return's gradients, here / there: 16384
// tokens, 24 slots, 64 columns 13.6 / 22.8 and 21.7 / 38.4; 16384, 2, 256 8.7 / 10.4 and 11.5 / 12.3; 4096, 6,
// 128 7.4 / 7.4 and 7.8 / 8.9; 1024, 24, 256 8.2 / 5.8 and 11.7 / 8.3.
constexpr int kNarrowD = 256, kNarrowT = 4096;
bool is_narrow(const TokenRows& p) { return p.D <= kNarrowD && p.T >= kNarrowT; }
template <Pass PASS>
void run_narrow(const TokenRows& p, Elt in_t, Elt rows_t, const void* a, const void* rows,
                const void* add, void* out, float* dweights, hipStream_t s) {
#define MOE_NARROW(I, R, L)                                                                        \
  hipLaunchKernelGGL((narrow_kernel<I, R, PASS, L>),                                               \
                     dim3((unsigned)(((int64_t)p.T * L + 255) / 256)), dim3(256), 0, s, p, a, rows, \
                     add, out, dweights)
#define MOE_NARROW_L(I, R)                       \
  {                                              \
    if (p.D <= 64) MOE_NARROW(I, R, 8);          \
    else if (p.D <= 128) MOE_NARROW(I, R, 16);   \
    else MOE_NARROW(I, R, 32);                   \
  }
  if (PASS == Pass::Spread || in_t == rows_t) {
    if (in_t == Elt::BF16) MOE_NARROW_L(Elt::BF16, Elt::BF16) else MOE_NARROW_L(Elt::F32, Elt::F32)
  } else if constexpr (PASS != Pass::Spread) {
    if (in_t == Elt::BF16) MOE_NARROW_L(Elt::BF16, Elt::F32) else MOE_NARROW_L(Elt::F32, Elt::BF16)
  }
#undef MOE_NARROW_L
#undef MOE_NARROW
}
}  // namespace

hipError_t launch_spread_rows(const TokenRows& p, Elt t, const void* in, void* out, hipStream_t s) {
  if (p.T <= 0) return hipSuccess;
  if (is_narrow(p)) {
    run_narrow<Pass::Spread>(p, t, t, in, nullptr, nullptr, out, nullptr, s);
    return hipGetLastError();
  }
#define MOE_SPREAD(X, W, S) \
  hipLaunchKernelGGL((spread_kernel<X, W, S>), seg_grid(p), dim3(256), 0, s, p, in, out)
#define MOE_SPREAD_W(X, S) \
  if (p.weights) MOE_SPREAD(X, true, S); else MOE_SPREAD(X, false, S)
  const bool bf = t == Elt::BF16;
  if (past_cache(p, t, t, 1)) {
    if (bf) { MOE_SPREAD_W(Elt::BF16, true); } else { MOE_SPREAD_W(Elt::F32, true); }
  } else {
    if (bf) { MOE_SPREAD_W(Elt::BF16, false); } else { MOE_SPREAD_W(Elt::F32, false); }
  }
#undef MOE_SPREAD_W
#undef MOE_SPREAD
  return hipGetLastError();
}

hipError_t launch_positions(const int32_t* idx, int T, int E, int k, int32_t* scratch,
                            int32_t* offsets, int32_t* pos, hipStream_t s) {
  if (T <= 0 || E > 1024 || k > 64) return hipErrorInvalidValue;
  const int ch = dispatch_chunk(T, k), nch = (int)(((int64_t)T + ch - 1) / ch);
  const size_t lds = (size_t)E * (ch / 32) * sizeof(uint32_t);
  auto run = [&](auto count, auto place) {
    hipLaunchKernelGGL(count, dim3(nch), dim3(ch), lds, s, idx, T, E, k, scratch);
    hipLaunchKernelGGL(place, dim3(nch), dim3(kPlaceThreads), lds, s, idx, T, E, k, scratch, nch,
                       offsets, pos);
  };
  if (ch == 64) run(dispatch_count<64>, place_kernel<64>);
  else if (ch == 128) run(dispatch_count<128>, place_kernel<128>);
  else run(dispatch_count<256>, place_kernel<256>);
  return hipGetLastError();
}

hipError_t launch_sort_small(const int32_t* idx, const float* weights, int T, int D, int E, int k,
                             Elt t, const void* in, void* out, int32_t* offsets, int32_t* pos,
                             hipStream_t s) {
  if (!sort_is_small(T, k) || E > 1024 || k > 64) return hipErrorInvalidValue;
  const dim3 grid(T + 1, T < 512 ? (D + 2047) / 2048 : 1);   // a long row is shared by workgroups
#define MOE_SORT(X, W)                                                                            \
  hipLaunchKernelGGL((sort_small_kernel<X, W>), grid, dim3(256), 0, s, idx, weights, T, D, E, \
                     k, in, out, offsets, pos)
  if (t == Elt::BF16) {
    if (weights) MOE_SORT(Elt::BF16, true); else MOE_SORT(Elt::BF16, false);
  } else {
    if (weights) MOE_SORT(Elt::F32, true); else MOE_SORT(Elt::F32, false);
  }
#undef MOE_SORT
  return hipGetLastError();
}

#define MOE_TOKEN(I, R, B)                                                                         \
  hipLaunchKernelGGL((token_kernel<I, R, PASS, B, STREAM>), dim3(p.T), dim3(64 * w.segs * w.cuts),         \
                     PASS != Pass::SpreadDot && w.cuts > 1 ? w.segs * w.cuts * 128 * sizeof(float4) : 0, \
                     s, p, w.segs, w.cuts, a, rows, add, out, dweights)
#define MOE_BATCHED(LAUNCH, I, R)                                         \
  {                                                                       \
    const int batch = batch_of(p.k, PASS);                                \
    if (batch == 2) LAUNCH(I, R, 2);                                      \
    else if (batch == 4) LAUNCH(I, R, 4);                                 \
    else if (batch == kMostBatch) LAUNCH(I, R, kMostBatch);               \
    else if constexpr (PASS == Pass::GatherDot) LAUNCH(I, R, 6);          \
  }
#define MOE_TYPED(LAUNCH)                                                 \
  if (in_t == Elt::BF16) {                                                \
    if (rows_t == Elt::BF16) MOE_BATCHED(LAUNCH, Elt::BF16, Elt::BF16)    \
    else MOE_BATCHED(LAUNCH, Elt::BF16, Elt::F32)                         \
  } else {                                                                \
    if (rows_t == Elt::BF16) MOE_BATCHED(LAUNCH, Elt::F32, Elt::BF16)     \
    else MOE_BATCHED(LAUNCH, Elt::F32, Elt::F32)                          \
  }

namespace {
template <bool STREAM>
void run_gather(const TokenRows& p, Elt in_t, Elt rows_t, const void* rows, const void* add,
                void* out, hipStream_t s) {
  constexpr Pass PASS = Pass::Gather;
#define MOE_GATHER(O, I, B)                                                                       \
  hipLaunchKernelGGL((gather_kernel<I, O, B, STREAM>), seg_grid(p), dim3(256), 0, s, p, rows, add, \
                     out)
  MOE_TYPED(MOE_GATHER)
#undef MOE_GATHER
}
template <Pass PASS, bool STREAM>
void run_tokens(const TokenRows& p, Waves w, Elt in_t, Elt rows_t, const void* a, const void* rows,
                const void* add, void* out, float* dweights, hipStream_t s) {
  MOE_TYPED(MOE_TOKEN)
}
}  // namespace

hipError_t launch_gather_rows(const TokenRows& p, Elt rows_t, const void* rows, const void* add,
                              Elt in_t, void* out, const void* a, float* dweights, hipStream_t s) {
  if (p.T <= 0) return hipSuccess;
  if (is_narrow(p)) {
    if (dweights) run_narrow<Pass::GatherDot>(p, in_t, rows_t, a, rows, add, out, dweights, s);
    else run_narrow<Pass::Gather>(p, in_t, rows_t, a, rows, add, out, dweights, s);
    return hipGetLastError();
  }
  const bool stream = past_cache(p, in_t, rows_t, 1);
  const Waves w = token_waves(p);
  if (dweights) {
    if (stream) run_tokens<Pass::GatherDot, true>(p, w, in_t, rows_t, a, rows, add, out, dweights, s);
    else run_tokens<Pass::GatherDot, false>(p, w, in_t, rows_t, a, rows, add, out, dweights, s);
  } else if (w.cuts > 1) {   // (few tokens)
    run_tokens<Pass::Gather, false>(p, w, in_t, rows_t, a, rows, add, out, dweights, s);
  } else if (stream) {
    run_gather<true>(p, in_t, rows_t, rows, add, out, s);
  } else {
    run_gather<false>(p, in_t, rows_t, rows, add, out, s);
  }
  return hipGetLastError();
}

hipError_t launch_spread_dot(const TokenRows& p, Elt in_t, const void* a, Elt rows_t,
                             const void* rows, void* out, float* dweights, hipStream_t s) {
  if (p.T <= 0) return hipSuccess;
  if (is_narrow(p)) {
    run_narrow<Pass::SpreadDot>(p, in_t, rows_t, a, rows, nullptr, out, dweights, s);
    return hipGetLastError();
  }
  const Waves w = token_waves(p);
  if (past_cache(p, in_t, rows_t, 2))
    run_tokens<Pass::SpreadDot, true>(p, w, in_t, rows_t, a, rows, nullptr, out, dweights, s);
  else
    run_tokens<Pass::SpreadDot, false>(p, w, in_t, rows_t, a, rows, nullptr, out, dweights, s);
  return hipGetLastError();
}
#undef MOE_TYPED
#undef MOE_BATCHED
#undef MOE_TOKEN

}  // namespace moe
