// Launchers of the global gradient norm over many tensors and clipping by it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstddef>

#include "gemm.hpp"

namespace moe {

constexpr int kClipChunkBytes = 16384;
// Most workgroups of a pass, and partial sums: four a CU (1024 / 2048: 2.19 GB 1089 / 1088 us, 134 MB
// 70.5 / 71.9, 134 MB read alone 30 / 32).
constexpr int kClipGroups = 1024;
constexpr int kClipPerLaunch = 80;     // tensors passed with one launch (3.2 KB)

// One tensor: n elements at `grad`, the clipped values go to `out` (may be grad); its chunks are
// [first, first + clip_chunks(n)) of all tensors' chunks.
struct ClipTensor {
  const char* grad;
  char* out;
  int64_t n;
  int64_t first;
  int32_t bf16;
};
// One chunk of a tensor, on the device.
struct alignas(32) ClipChunk {
  const char* grad;
  char* out;
  int32_t n;       // elements
  int32_t bf16;
};

inline int64_t clip_chunks(int64_t n, bool bf16) {
  const int64_t e = kClipChunkBytes / (bf16 ? 2 : 4);
  return (n + e - 1) / e;
}
inline int clip_groups(int64_t chunks) {
  return chunks < kClipGroups ? (int)chunks : kClipGroups;
}

// Writes the chunks of n tensors, `chunks` in all, to the table on the device.
struct ClipBatch {
  ClipTensor t[kClipPerLaunch];
};
hipError_t launch_clip_table(const ClipBatch& b, int n, int64_t chunks, ClipChunk* table,
                             hipStream_t s);

// norm[0] = sqrt(sum of squares over all chunks), norm[1] = coef = min(1, max_norm / (norm + 1e-6))
// (1 where the norm is not finite); out = coef * grad. in_place: every out is its grad, so nothing is
// written where coef is 1. partial: kClipGroups doubles.
hipError_t launch_clip(const ClipChunk* table, int64_t chunks, bool in_place, float max_norm,
                       double* partial, float* norm, hipStream_t s);

}  // namespace moe
