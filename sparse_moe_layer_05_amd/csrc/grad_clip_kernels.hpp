// The global norm of many gradients, and their clipping by it (gfx950).
//
//   norm = sqrt(sum over every tensor of g^2), coef = min(1, max_norm / (norm + 1e-6)),
//   out = coef g (rounded once)
//
// Two launches, whatever the number of tensors: their table is on the device, cut into chunks of
// 32 KB, and every workgroup walks one contiguous range of chunks. The second launch's workgroups
// each add the first one's partial sums, in order, so no atomics and no third launch are needed and
// the result does not depend on timing. Squares are summed in fp64: the conversion hides under the
// loads, and no gradient over- or underflows on the way to the root.
// Bound by HBM: the norm is needed before the first value can be written, so gradients are read
// twice and written once, the second reading from the last-level cache (256 MB) where they fit.
// Included once, by backward.hip.
#pragma once

#include "common.hpp"
#include "grad_clip.hpp"
#include "row8.hpp"

namespace moe {
namespace {
namespace grad_clip {

constexpr int kClipThreads = 256;

__global__ __launch_bounds__(kClipPerLaunch) void clip_table_kernel(ClipBatch b, int n,
                                                                    ClipTensor* table, int at) {
  const int i = threadIdx.x;
  if (i < n) table[at + i] = b.t[i];
}

// Elements of one chunk: a head up to the first 16-byte border, whole vectors, a tail.
template <Elt T>
struct Span {
  static constexpr int kElt = T == Elt::BF16 ? 2 : 4, kVec = 16 / kElt;
  const char* p;     // the chunk's first element
  int n, head, vecs;
  __device__ Span(const ClipTensor& t, int64_t chunk) {
    constexpr int64_t per = kClipChunkBytes / kElt;
    const int64_t at = chunk * per;
    p = (const char*)t.grad + at * kElt;
    n = (int)min(per, t.n - at);
    head = min(n, (int)((16 - ((uintptr_t)p & 15)) & 15) / kElt);
    vecs = (n - head) / kVec;
  }
  // index of a single element: head first, then the tail; -1 past them
  __device__ int single(int i) const {
    if (i < head) return i;
    const int j = head + vecs * kVec + (i - head);
    return j < n ? j : -1;
  }
};

template <Elt T>
__device__ __forceinline__ float load1(const void* p, int i) {
  if constexpr (T == Elt::BF16) return bf16_bits_to_f32(((const uint16_t*)p)[i]);
  else return ((const float*)p)[i];
}
template <Elt T>
__device__ __forceinline__ void store1(void* p, int i, float v) {
  if constexpr (T == Elt::BF16) ((uint16_t*)p)[i] = (uint16_t)f32_to_bf16_bits(v);
  else ((float*)p)[i] = v;
}

constexpr int kUnroll = kClipChunkBytes / 16 / kClipThreads;   // 8 vectors a thread

template <Elt T>
__device__ __forceinline__ void unpack16(uint4 q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (T == Elt::BF16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}

template <Elt T>
__device__ __forceinline__ double chunk_squares(const ClipTensor& t, int64_t chunk) {
  const Span<T> sp(t, chunk);
  const uint4* v = (const uint4*)(sp.p + sp.head * Span<T>::kElt);
  uint4 q[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = u * kClipThreads + threadIdx.x;
    q[u] = i < sp.vecs ? v[i] : make_uint4(0, 0, 0, 0);
  }
  double s = 0.0;
  const int one = sp.single(threadIdx.x);   // at most 7 before and 7 behind the vectors
  if (threadIdx.x < 16 && one >= 0) {
    const double x = load1<T>(sp.p, one);
    s = x * x;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float x[Span<T>::kVec];
    unpack16<T>(q[u], x);
#pragma unroll
    for (int i = 0; i < Span<T>::kVec; ++i) s = fma((double)x[i], (double)x[i], s);
  }
  return s;
}

template <Elt T>
__device__ __forceinline__ void chunk_scale(const ClipTensor& t, int64_t chunk, float coef) {
  const Span<T> sp(t, chunk);
  constexpr int V = Span<T>::kVec, B = Span<T>::kElt;
  const uint4* v = (const uint4*)(sp.p + sp.head * B);
  char* out = (char*)t.out + (sp.p - (const char*)t.grad);
  const bool aligned = (((uintptr_t)out ^ (uintptr_t)sp.p) & 15) == 0;
  uint4 q[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = u * kClipThreads + threadIdx.x;
    if (i < sp.vecs) q[u] = v[i];
  }
  const int one = sp.single(threadIdx.x);
  if (threadIdx.x < 16 && one >= 0) store1<T>(out, one, coef * load1<T>(sp.p, one));
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = u * kClipThreads + threadIdx.x;
    if (i >= sp.vecs) continue;
    float x[V];
    unpack16<T>(q[u], x);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] *= coef;
    if (aligned) {
      uint4 r;
      if constexpr (T == Elt::BF16)
        r = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
      else
        r = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                       __float_as_uint(x[3]));
      ((uint4*)(out + sp.head * B))[i] = r;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) store1<T>(out, sp.head + i * V + e, x[e]);
    }
  }
}

// The entry that holds a chunk: the last whose first chunk is not behind it (entries are in order of
// their first chunk; empty tensors are not in the table). 64 candidates a step.
__device__ __forceinline__ int find_entry(const ClipTensor* table, int count, int64_t chunk) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = count;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int i = lo + lane * step;
    const bool le = lane * step < n && (table[i].first & ~kClipBf16) <= chunk;
    const int k = __popcll(__ballot(le)) - 1;   // entry lo is never behind it
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// fn(entry, chunk within its tensor) for the chunks of this workgroup, forwards or backwards.
template <bool BACK, typename F>
__device__ __forceinline__ void walk(const ClipTensor* table, int count, int64_t chunks, F&& fn) {
  const int64_t per = chunks / gridDim.x, more = chunks % gridDim.x, b = blockIdx.x;
  const int64_t lo = b * per + min(b, more), hi = lo + per + (b < more ? 1 : 0);
  if (lo >= hi) return;
  int i = find_entry(table, count, BACK ? hi - 1 : lo);
  ClipTensor t = table[i];
  for (int64_t s = 0; s < hi - lo; ++s) {
    const int64_t c = BACK ? hi - 1 - s : lo + s;
    if (BACK) {
      if (c < (t.first & ~kClipBf16)) t = table[--i];
    } else {
      while (i + 1 < count && (table[i + 1].first & ~kClipBf16) <= c) t = table[++i];
    }
    fn(t, c - (t.first & ~kClipBf16));
  }
}

// Sum over the workgroup, in every thread.
__device__ __forceinline__ double group_sum(double s) {
  __shared__ double part[kClipThreads / 64];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(kClipThreads) void clip_squares_kernel(const ClipTensor* table, int count,
                                                                int64_t chunks, double* partial) {
  double s = 0.0;
  walk<false>(table, count, chunks, [&](const ClipTensor& t, int64_t c) {
    s += (t.first & kClipBf16) ? chunk_squares<Elt::BF16>(t, c) : chunk_squares<Elt::F32>(t, c);
  });
  s = group_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(const ClipTensor* table, int count,
                                                              int64_t chunks, int parts,
                                                              bool in_place, float max_norm,
                                                              const double* partial, float* norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) s += partial[i];
  const double root = sqrt(group_sum(s));
  const double ratio = (double)max_norm / (root + 1e-6);
  const float coef = root < __builtin_inf() && ratio < 1.0 ? (float)ratio : 1.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = (float)root;
    norm[1] = coef;
  }
  if (in_place && coef == 1.f) return;
  walk<true>(table, count, chunks, [&](const ClipTensor& t, int64_t c) {
    if (t.first & kClipBf16) chunk_scale<Elt::BF16>(t, c, coef);
    else chunk_scale<Elt::F32>(t, c, coef);
  });
}

}  // namespace grad_clip
}  // namespace

using namespace grad_clip;

hipError_t launch_clip_table(const ClipBatch& b, int n, ClipTensor* table, int at, hipStream_t s) {
  hipLaunchKernelGGL(clip_table_kernel, dim3(1), dim3(kClipPerLaunch), 0, s, b, n, table, at);
  return hipGetLastError();
}

hipError_t launch_clip(const ClipTensor* table, int count, int64_t chunks, bool in_place,
                       float max_norm, double* partial, float* norm, hipStream_t s) {
  const int groups = clip_groups(chunks);
  if (groups)
    hipLaunchKernelGGL(clip_squares_kernel, dim3(groups), dim3(kClipThreads), 0, s, table, count,
                       chunks, partial);
  hipLaunchKernelGGL(clip_scale_kernel, dim3(groups ? groups : 1), dim3(kClipThreads), 0, s, table,
                     count, chunks, groups, in_place, max_norm, partial, norm);
  return hipGetLastError();
}

}  // namespace moe
