// Launchers of the kernels that move token rows into expert order and back.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.hpp"
#include "kernels.hpp"

namespace moe {

// pos [T, k]: the row of pair (t, j); a value outside [0, n_rows) marks a dropped pair. weights
// [T, k] fp32 or nullptr (1). D is a multiple of 8, k at most 64.
struct TokenRows {
  const int32_t* pos = nullptr;
  const float* weights = nullptr;
  int T = 0, D = 0, k = 0, n_rows = 0;
};

// out[pos[t, j]] = weights[t, j] * in[t], both of type t.
hipError_t launch_spread_rows(const TokenRows& p, Elt t, const void* in, void* out, hipStream_t s);

// Positions, offsets and the spread of few pairs in one launch (E <= 1024). Every workgroup looks at
// all pairs for each of its token's slots, so the limit is on pairs times slots as well. Microseconds,
// one launch / the dispatch and a spread: 64 tokens, 6 slots (2304) 6.4 / 8.8; 1000, 2 (4000) 9.2 / 12.1;
// 256, 6 (9216) 11.5 / 11.0; 64, 24 (36864) 19.6 / 12.6.
constexpr int kSortSmallPairs = 2048, kSortSmallWork = 8192;
inline bool sort_is_small(int64_t T, int k) {
  return T * k <= kSortSmallPairs && T * k * k <= kSortSmallWork;
}
hipError_t launch_sort_small(const int32_t* idx, const float* weights, int T, int D, int E, int k,
                             Elt t, const void* in, void* out, int32_t* offsets, int32_t* pos,
                             hipStream_t s);

// Positions and offsets alone, in two launches (T >= 1, E <= 1024). scratch: ceil(T / chunk) * E ints,
// chunk as the dispatch cuts the tokens. Every chunk's workgroup reads all chunks' counts: for many of
// both the dispatch, which scans them once in a launch of its own, is faster. Microseconds here / there
// (16 columns): 65536 tokens, 6 of 128 22 / 46; 262144, 6 of 128 (2^27) 64 / 135; 131072, 24 of 512 (2^27)
// 102 / 166; 262144, 6 of 1024 (2^30) 291 / 216.
inline bool positions_by_chunks(int T, int E, int k) {
  const int ch = dispatch_chunk(T, k);
  const int64_t n = ((int64_t)T + ch - 1) / ch;
  return n <= 16384 && n * n * E <= (int64_t)1 << 28;
}
hipError_t launch_positions(const int32_t* idx, int T, int E, int k, int32_t* scratch,
                            int32_t* offsets, int32_t* pos, hipStream_t s);

// out[t] = add[t] + sum_j weights[t, j] * rows[pos[t, j]], rounded once (add, of out's type, may be
// nullptr). With dweights: dweights[t, j] = <a[t], rows[pos[t, j]]>, a of the rows' type (0 for dropped
// pairs).
hipError_t launch_gather_rows(const TokenRows& p, Elt rows_t, const void* rows, const void* add,
                              Elt out_t, void* out, const void* a, float* dweights, hipStream_t s);

// out[pos[t, j]] = weights[t, j] * a[t] and dweights[t, j] = <a[t], rows[pos[t, j]]>; rows and out of
// type rows_t (out may be rows).
hipError_t launch_spread_dot(const TokenRows& p, Elt a_t, const void* a, Elt rows_t,
                             const void* rows, void* out, float* dweights, hipStream_t s);

}  // namespace moe
