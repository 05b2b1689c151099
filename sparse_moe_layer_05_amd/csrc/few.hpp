// Launchers of the few-token layer (at most kFewTokens tokens): the whole layer in three launches
// (four for LatentMoE).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.hpp"

namespace moe {

constexpr int kFewTokens = 16;          // one matrix-core block of tokens
// 8- and 4-bit experts: T * D and T * I in whole steps of 128, whose rows stay in LDS as bf16.
constexpr int kFewNarrowElts = 65536;

struct FewParams {
  int T = 0, H = 0, E = 0, k = 0, I = 0, Is = 0, L = 0, D = 0;
  Elt ex = Elt::BF16;
  bool given = false;                   // idx_in / gates_in instead of the router
  const uint16_t* x = nullptr;          // [T][H]
  const uint16_t* W_r = nullptr;
  const float* b = nullptr;
  const uint8_t* W_up = nullptr;        // [E][I][D], stored format
  const uint8_t* W_down = nullptr;      // [E][D][I]
  const void* s_up = nullptr;           // e4m3: fp32 [E][I]; MX: uint8 [E][I][D / 32]
  const void* s_down = nullptr;
  const uint16_t* Ws_up = nullptr;      // [Is][H]
  const uint16_t* Ws_down = nullptr;    // [H][Is]
  const uint16_t* W_in = nullptr;       // [L][H]
  const uint16_t* W_out = nullptr;      // [H][L]
  uint16_t* y = nullptr;                // [T][H]
  const int32_t* idx_in = nullptr;
  const float* gates_in = nullptr;
  // routing record and scratch
  float* logits = nullptr;              // [T][E]
  float* score = nullptr;               // [T][E] sigmoid(logit)
  int32_t* idx = nullptr;               // [T][k]
  float* gates = nullptr;               // [T][k]
  int32_t* n_slots = nullptr;           // [1]
  int32_t* slot_e = nullptr;            // [slots] touched experts, ascending
  float* gate_m = nullptr;              // [slots][kFewTokens] gate of a token, 0 where not selected
  uint32_t* slot_mask = nullptr;        // [slots] bit t: token t selected the expert
  uint32_t* hmax = nullptr;             // [slots][kFewTokens] bits of max h (8- and 4-bit experts)
  float* slabs = nullptr;               // [D / 16][parts][kFewTokens][16] (parts > 1)
  int32_t* joined = nullptr;            // [D / 16] parts of a column block that have ended
  uint16_t* h = nullptr;                // [slots][T][I] bf16
  uint16_t* h_lo = nullptr;             // what h's rounding left over (bf16 experts)
  uint16_t* hs = nullptr;               // [T][Is] bf16, and what its rounding left over
  uint16_t* hs_lo = nullptr;
  uint16_t* u = nullptr;                // [T][L] bf16
  uint16_t* z = nullptr;                // [T][L] bf16, and what its rounding left over
  uint16_t* z_lo = nullptr;
};

__host__ __device__ inline int few_slots(int T, int E, int k) { return E < T * k ? E : T * k; }

// Parts that the down projection's column blocks of 16 are cut into: about two workgroups of
// eight waves per CU.
inline int few_parts(int D) {
  const int n = 512 / (D / 16);
  return n < 1 ? 1 : (n > 8 ? 8 : n);
}

// The launches, in order; launch_few_out is LatentMoE's.
hipError_t launch_few_front(const FewParams& p, hipStream_t s);
hipError_t launch_few_up(const FewParams& p, hipStream_t s);
hipError_t launch_few_down(const FewParams& p, hipStream_t s);
hipError_t launch_few_out(const FewParams& p, hipStream_t s);

}  // namespace moe
