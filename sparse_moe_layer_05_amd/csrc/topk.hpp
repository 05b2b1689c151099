// Selection of the k largest keys of one token by one wave, shared by the router kernels and the
// few-token layer.
#pragma once

#include "common.hpp"

namespace moe {

// Order-preserving map of a float's bits to an unsigned integer (larger float, larger integer).
__device__ __forceinline__ uint32_t okey(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// Wave-wide maximum of a 64-bit value by DPP row shifts and row broadcasts (lane 63 ends with
// the result over all 64 lanes), then read back from lane 63 as a wave-uniform value. A lane
// whose DPP source is outside its row (or whose row is masked off) combines with 0, the
// identity.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_max_step_u64(uint64_t v) {
  const uint32_t lo =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
  const uint64_t o = ((uint64_t)hi << 32) | lo;
  return o > v ? o : v;
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  v = dpp_max_step_u64<0x111, 0xf>(v);  // row_shr:1
  v = dpp_max_step_u64<0x112, 0xf>(v);  // row_shr:2
  v = dpp_max_step_u64<0x114, 0xf>(v);  // row_shr:4
  v = dpp_max_step_u64<0x118, 0xf>(v);  // row_shr:8: lane 15 of each row holds the row's max
  v = dpp_max_step_u64<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_max_step_u64<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, 63);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63);
  return ((uint64_t)hi << 32) | lo;
}

// k rounds of selection over the keys of one token; lane l holds experts l, l + 64, ... Each
// expert carries one 64-bit value, its key's order-preserving bits above its inverted index, so
// that one wave-wide maximum per round yields the largest key and, among equal keys, the lowest
// expert (a float maximum followed by an index minimum took two reductions a round). The values
// are distinct, so round j retires the largest value below round j-1's: nothing is cleared and
// no score is read inside a round, whose cost is one dependent chain. Lane j keeps round j's
// winner; the scores are fetched afterwards and summed in round order on every lane.
// TREE: each lane's largest value below the last winner as a tree over its slots (shorter chain;
// faster with one token per workgroup, slower with four waves of tokens per workgroup).
// Writes the k experts (descending key) and their gates (scores renormalised over the
// selection).
template <int NPER, bool TREE>
__device__ __forceinline__ void select_topk(const float* key, const float* sc, int lane, int E,
                                            int k, int32_t* __restrict__ idx_t,
                                            float* __restrict__ gates_t) {
  uint64_t c[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 64 * i;
    c[i] = e < E ? ((uint64_t)okey(key[i]) << 32) | (uint32_t)~e : 0;
  }
  uint64_t prev = ~0ull, mine = 0;
  for (int j = 0; j < k; ++j) {
    uint64_t m = 0;
    if constexpr (TREE) {
      uint64_t a[NPER];
#pragma unroll
      for (int i = 0; i < NPER; ++i) a[i] = c[i] < prev ? c[i] : 0;
#pragma unroll
      for (int w = 1; w < NPER; w *= 2)
#pragma unroll
        for (int i = 0; i + w < NPER; i += 2 * w) a[i] = a[i + w] > a[i] ? a[i + w] : a[i];
      m = a[0];
    } else {
#pragma unroll
      for (int i = 0; i < NPER; ++i) m = c[i] < prev && c[i] > m ? c[i] : m;
    }
    prev = wave_max_u64(m);
    if (lane == j) mine = prev;
  }
  const int be = (int)~(uint32_t)mine;
  const int slot = lane < k ? be >> 6 : 0, owner = lane < k ? be & 63 : 0;
  float bs = 0.f;  // the score lane `owner` holds in slot `slot`
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const float t = __int_as_float(__builtin_amdgcn_ds_bpermute(owner << 2, __float_as_int(sc[i])));
    bs = slot == i ? t : bs;
  }
  float sum = 0.f;  // the same order j = 0..k-1 on every lane: deterministic
  for (int j = 0; j < k; ++j) sum += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bs), j));
  if (lane < k) {
    idx_t[lane] = be;
    gates_t[lane] = bs / sum;
  }
}

}  // namespace moe
