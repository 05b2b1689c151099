// Launchers of the global gradient norm over many tensors and clipping by it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstddef>

#include "gemm.hpp"

namespace moe {

// One tensor: n elements (fp32, or bf16) at `grad`; the clipped values go to `out` (may be grad).
// first: its first chunk among all tensors' chunks.
struct ClipTensor {
  const void* grad;
  void* out;
  int64_t n;
  int64_t first;   // bit 62: bf16
};
constexpr int64_t kClipBf16 = (int64_t)1 << 62;
constexpr int kClipChunkBytes = 32768;
constexpr int kClipGroups = 1024;      // workgroups of a pass, and partial sums
constexpr int kClipPerLaunch = 96;     // table entries passed with one launch (3 KB)

inline int64_t clip_chunks(int64_t n, Elt t) {
  const int64_t e = kClipChunkBytes / (t == Elt::BF16 ? 2 : 4);
  return (n + e - 1) / e;
}
inline int clip_groups(int64_t chunks) {
  return chunks < kClipGroups ? (int)chunks : kClipGroups;
}

// Writes entries [at, at + n) of the table on the device.
struct ClipBatch {
  ClipTensor t[kClipPerLaunch];
};
hipError_t launch_clip_table(const ClipBatch& b, int n, ClipTensor* table, int at, hipStream_t s);

// norm[0] = sqrt(sum of squares over all tensors), norm[1] = coef = min(1, max_norm / (norm + 1e-6))
// (1 where the norm is not finite); with write: out = coef * grad. in_place: every out is its grad,
// so nothing is written where coef is 1. partial: kClipGroups doubles.
hipError_t launch_clip(const ClipTensor* table, int count, int64_t chunks, bool in_place,
                       float max_norm, double* partial, float* norm, hipStream_t s);

}  // namespace moe
