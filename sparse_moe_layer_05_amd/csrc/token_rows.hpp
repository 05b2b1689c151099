// Launchers of the kernels that move token rows into expert order and back.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.hpp"

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

// out[t] = add[t] + sum_j weights[t, j] * in[pos[t, j]] in j order, rounded once (add, of out's
// type, may be nullptr). With dot: dweights[t, j] = <other[t], in[pos[t, j]]>, other of in's type
// (0 for dropped pairs).
hipError_t launch_gather_rows(const TokenRows& p, Elt in_t, const void* in, const void* add,
                              Elt out_t, void* out, const void* other, float* dweights,
                              hipStream_t s);

// out[pos[t, j]] = weights[t, j] * in[t] and dweights[t, j] = <in[t], rows[pos[t, j]]>; rows and
// out of type rows_t (out may be rows).
hipError_t launch_spread_dot(const TokenRows& p, Elt in_t, const void* in, Elt rows_t,
                             const void* rows, void* out, float* dweights, hipStream_t s);

}  // namespace moe
