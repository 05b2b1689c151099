// Launchers of the norms before and after a block, with its gate, residual and the next norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstddef>

#include "gemm.hpp"

namespace moe {

constexpr int kBlockMaxH = 16384;   // row width the kernels hold in registers

enum class Gate : int { None = 0, Token = 1, Element = 2 };

// One block's description, the same for its forward and its backward pass. T rows of H elements
// (a multiple of 8, at most kBlockMaxH) of type t; w and w_next [H] of type w_t or nullptr (1).
struct BlockShape {
  int T = 0, H = 0;
  Elt t = Elt::BF16, w_t = Elt::BF16;
  Gate gate_kind = Gate::None;   // Token: [T] fp32, Element: [T, H] of type t
  bool sigmoid = false;          // the gate is given before its sigmoid
  bool norm = false;             // f is normalised
  float scale = 1.f, eps = 0.f;
};

// y = x + scale * gate * (n(f) or f) * w, h = n(y) * w_next (nullptr: not wanted).
// f == nullptr: h = n(x) * w_next alone.
struct BlockForward {
  const void *x = nullptr, *f = nullptr, *w = nullptr, *gate = nullptr, *w_next = nullptr;
  void *y = nullptr, *h = nullptr;
  bool stream = false;   // set by the launcher: operands are read past the caches
};
hipError_t launch_block_forward(const BlockShape& b, const BlockForward& p, hipStream_t s);

// Gradients of the same: d = dy + (gradient of h at y); dx = d; df, dw, dgate from d; dw_next.
// f == nullptr: dx = dy + gradient of h at y, and dw_next. dy, or y and dh together, may be
// nullptr; dh has type dh_t. dw, dw_next: [H] fp32 or nullptr. part: block_parts(...) fp32.
struct BlockBackward {
  const void *dy = nullptr, *f = nullptr, *w = nullptr, *gate = nullptr, *y = nullptr,
             *dh = nullptr, *w_next = nullptr;
  Elt dh_t = Elt::BF16;
  void *dx = nullptr, *df = nullptr, *dgate = nullptr;
  float *dw = nullptr, *dw_next = nullptr;
  float* part = nullptr;
  bool stream = false;   // as above
};
hipError_t launch_block_backward(const BlockShape& b, const BlockBackward& p, hipStream_t s);
// fp32 partial sums of dw and dw_next.
size_t block_part_floats(int T, int H);

}  // namespace moe
