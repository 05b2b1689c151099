// The global norm of many gradients, and their clipping by it (gfx950).
//
//   norm = sqrt(sum over every tensor of g^2), coef = min(1, max_norm / (norm + 1e-6)),
//   out = coef g (rounded once)
//
// Two launches, whatever the number of tensors: a table on the device cuts them into chunks of 16 KB,
// which the workgroups take in turn, one chunk's loads in flight while the one before is worked on.
// The second launch's workgroups each add the first one's partial sums, in order, so no atomics and
// no third launch are needed and the result does not depend on timing. Squares are summed in fp64:
// the conversion hides under the loads, and no gradient over- or underflows on the way to the root.
// Bound by HBM: the norm is needed before the first value can be written, so gradients are read
// twice and written once, the second reading, last chunk first, from the last-level cache (256 MB)
// where they fit. Measured: 2.19 GB of fp32 312 us (7.1 TB/s read) and 793 us (5.5 TB/s), 192 tensors of
// 113 MB, bf16 and fp32, 21 and 36 us (5.5 and 6.2 TB/s); one launch on 4 MB about 3 us. The table costs
// the caller's host time, about 1.4 us a tensor, once for all calls.
// Included once, by backward.hip.
#pragma once

#include "common.hpp"
#include "grad_clip.hpp"
#include "row8.hpp"

namespace moe {
namespace {
namespace grad_clip {

constexpr int kClipThreads = 256;
constexpr int kUnroll = kClipChunkBytes / 16 / kClipThreads;   // 4 vectors a thread

// A thread per chunk: the tensor that holds it is the last whose first chunk is not behind it.
__global__ __launch_bounds__(256) void clip_table_kernel(ClipBatch b, int n, int64_t chunks,
                                                         ClipChunk* table) {
  const int64_t c = b.t[0].first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= b.t[0].first + chunks) return;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (b.t[mid].first <= c) lo = mid; else hi = mid;
  }
  const ClipTensor& t = b.t[lo];
  const int per = kClipChunkBytes / (t.bf16 ? 2 : 4);
  const int64_t k = c - t.first;
  ClipChunk o;
  o.grad = t.grad + k * kClipChunkBytes;
  o.out = t.out + k * kClipChunkBytes;
  o.n = (int)min((int64_t)per, t.n - k * per);
  o.bf16 = t.bf16;
  table[c] = o;
}

// A chunk's elements as its threads hold them: whole 16-byte vectors, and the few elements before and
// behind them, one a thread (at most 7 each). Loads past the vectors give zeros.
struct Held {
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  u32x4 v[kUnroll];
  float one;
  int head, vecs, single;   // single: this thread's element; -1: none

  // LAST: nobody reads the chunk soon again, so its lines are marked as the first to leave the caches.
  template <bool LAST>
  __device__ __forceinline__ void load(const ClipChunk& c, bool present) {
    const int lg = c.bf16 ? 1 : 2, per = 16 >> lg;
    head = min(c.n, (int)((16 - ((uintptr_t)c.grad & 15)) & 15) >> lg);
    vecs = (c.n - head) / per;
    const auto r = __builtin_amdgcn_make_buffer_rsrc((char*)c.grad + (head << lg), (short)0,
                                                     present ? vecs * 16 : 0, 0x00020000);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      v[u] = __builtin_amdgcn_raw_buffer_load_b128(r, (u * kClipThreads + threadIdx.x) * 16, 0,
                                                   LAST ? 2 : 0);
    const int i = threadIdx.x < head ? threadIdx.x : vecs * per + threadIdx.x;
    single = threadIdx.x < 16 && i < c.n && present ? i : -1;
    one = 0.f;
    if (single >= 0)
      one = c.bf16 ? bf16_bits_to_f32(((const uint16_t*)c.grad)[i]) : ((const float*)c.grad)[i];
  }
};

template <bool BF16>
__device__ __forceinline__ void unpack16(Held::u32x4 q, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    } else {
      v[i] = __uint_as_float(q[i]);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ double squares(const Held& h) {
  constexpr int V = BF16 ? 8 : 4;
  double s[2] = {(double)h.one * h.one, 0.0};
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float x[V];
    unpack16<BF16>(h.v[u], x);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i & 1] = fma((double)x[i], (double)x[i], s[i & 1]);
  }
  return s[0] + s[1];
}

template <bool BF16>
__device__ __forceinline__ void scale(const Held& h, char* out, float coef) {
  constexpr int V = BF16 ? 8 : 4, B = BF16 ? 2 : 4;
  auto put = [&](int i, float x) {
    if constexpr (BF16) ((uint16_t*)out)[i] = (uint16_t)f32_to_bf16_bits(x);
    else ((float*)out)[i] = x;
  };
  if (h.single >= 0) put(h.single, coef * h.one);
  char* const body = out + h.head * B;
  const bool aligned = ((uintptr_t)body & 15) == 0;   // the same in every thread
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = u * kClipThreads + threadIdx.x;
    if (i >= h.vecs) continue;
    float x[V];
    unpack16<BF16>(h.v[u], x);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] *= coef;
    if (aligned) {
      Held::u32x4 r;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        r[j] = BF16 ? pack_bf16x2(x[2 * j % V], x[(2 * j + 1) % V]) : __float_as_uint(x[j]);
      __builtin_nontemporal_store(r, (Held::u32x4*)body + i);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) put(h.head + i * V + e, x[e]);
    }
  }
}

// fn(chunk, what is held of it) for the chunks blockIdx.x, blockIdx.x + gridDim.x, .. (counted from
// the last with BACK); the next chunk is loaded first. The second reading starts with the last chunks:
// kKeep of them (240 MB) are read into the caches the first time, all others past them, as are the
// second reading and the results. Microseconds with 0 / 128 / 192 / 240 MB kept: 268 MB of fp32 152 / 144 /
// 138 / 135, 134 MB 77 / 70 / 71 / 70, 2.19 GB 1094 / 1091 / 1089 / 1089 (all through the caches: 166, 85 and 1172).
constexpr int64_t kKeep = 15360;
template <bool BACK, typename F>
__device__ __forceinline__ void walk(const ClipChunk* table, int64_t chunks, F&& fn) {
  int64_t c = blockIdx.x;
  if (c >= chunks) return;
  auto load = [&](Held& h, int64_t i, bool present) {
    const ClipChunk k = table[BACK ? chunks - 1 - i : i];
    if (BACK || i < chunks - kKeep) h.load<true>(k, present);
    else h.load<false>(k, present);
    return k;
  };
  Held a, b;
  ClipChunk now = load(a, c, true);
  while (true) {
    const int64_t n = c + gridDim.x;
    const ClipChunk next = load(b, n < chunks ? n : c, n < chunks);
    fn(now, a);
    if (n >= chunks) return;
    now = next;
    a = b;
    c = n;
  }
}

// Sum over the workgroup, in every thread.
__device__ __forceinline__ double all_sum(double s) {
  __shared__ double part[kClipThreads / 64];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(kClipThreads) void clip_squares_kernel(const ClipChunk* table,
                                                                    int64_t chunks,
                                                                    double* partial) {
  double s = 0.0;
  walk<false>(table, chunks, [&](const ClipChunk& c, const Held& h) {
    s += c.bf16 ? squares<true>(h) : squares<false>(h);
  });
  s = all_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(const ClipChunk* table,
                                                                  int64_t chunks, int parts,
                                                                  bool in_place, float max_norm,
                                                                  const double* partial,
                                                                  float* norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) s += partial[i];
  const double root = sqrt(all_sum(s));
  const double ratio = (double)max_norm / (root + 1e-6);
  const float coef = root < __builtin_inf() && ratio < 1.0 ? (float)ratio : 1.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = (float)root;
    norm[1] = coef;
  }
  if (in_place && coef == 1.f) return;
  walk<true>(table, chunks, [&](const ClipChunk& c, const Held& h) {
    if (c.bf16) scale<true>(h, c.out, coef);
    else scale<false>(h, c.out, coef);
  });
}

}  // namespace grad_clip
}  // namespace

using namespace grad_clip;

hipError_t launch_clip_table(const ClipBatch& b, int n, int64_t chunks, ClipChunk* table,
                             hipStream_t s) {
  hipLaunchKernelGGL(clip_table_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, s, b,
                     n, chunks, table);
  return hipGetLastError();
}

hipError_t launch_clip(const ClipChunk* table, int64_t chunks, bool in_place, float max_norm,
                       double* partial, float* norm, hipStream_t s) {
  const int groups = clip_groups(chunks);
  if (groups)
    hipLaunchKernelGGL(clip_squares_kernel, dim3(groups), dim3(kClipThreads), 0, s, table, chunks,
                       partial);
  hipLaunchKernelGGL(clip_scale_kernel, dim3(groups ? groups : 1), dim3(kClipThreads), 0, s, table,
                     chunks, groups, in_place, max_norm, partial, norm);
  return hipGetLastError();
}

}  // namespace moe
