// Launchers of the block-scaled (OCP microscaling, MX v1.0) kernels: conversion of rows to and
// from MXFP4 / MXFP8, and products of block-scaled matrices.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.hpp"

namespace moe {

constexpr int kMxBlockElts = 32;  // elements that share one E8M0 scale
// Elements one conversion launch takes: a grid's threads (16 elements or more each) stay at or
// below 2^32.
constexpr int64_t kMxMaxElts = (int64_t)1 << 35;

// n elements (whole blocks, contiguous) of bf16 / fp32 -> codes and one E8M0 scale per block.
hipError_t launch_mx_quantize(const void* x, Elt xt, int64_t n, Elt fmt, uint8_t* codes,
                              uint8_t* scales, hipStream_t s);
// The values that n stored elements stand for, as bf16 / fp32.
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, Elt fmt, int64_t n,
                                void* x, Elt xt, hipStream_t s);

// C[m, n] = act( a_row[m] * sum_k A[m, k] W[n, k] ). A: MXFP4 or MXFP8 with block scales a_mx, or
// FP8 (e4m3 codes with one fp32 scale a_row per source row). W: MXFP4 or MXFP8 with block scales
// w_mx. Grouped launches (mt_start set) walk M-tiles of bm rows per group, as GemmParams.
struct MxGemmParams {
  const uint8_t* A = nullptr;        // [a_rows][K] elements, contiguous rows
  const uint8_t* a_mx = nullptr;     // [a_rows][K / 32]
  const float* a_row = nullptr;      // [a_rows]
  int a_rows = 0;
  const int32_t* a_gather = nullptr; // source row of row r (nullptr: r)
  const uint8_t* W = nullptr;        // [G][N][K]
  const uint8_t* w_mx = nullptr;     // [G][N][K / 32]
  void* C = nullptr;                 // [M][N]
  int M = 0, N = 0, K = 0;
  int out_f32 = 0;                   // C element type: fp32, else bf16
  int sqrelu = 0;                    // C = relu(acc)^2
  const int32_t* offs = nullptr;     // grouped: [G + 1] row offsets
  const int32_t* mt_start = nullptr; // grouped: [G + 1] prefix of ceil(rows_g / bm)
  int G = 0;
  int bm = 0;                        // grouped: 64 or 128 (mx_group_bm)
};
// Rows of the grouped launches' M-tiles: 64 where experts hold few rows on average (every expert's
// last tile is partly empty), else 128, which read the weights half as often; and 64 where tiles of
// 128 are fewer than CUs. Microseconds per layer, 64 / 128: Nano (128 experts) MXFP4 at 38 rows an
// expert 397 / 395, 48 408 / 407, 56 449 / 418, 96 562 / 502, 384 1637 / 1355; MXFP8 at 48 rows 491 /
// 540, 80 581 / 617, 112 692 / 703, 131 761 / 738, 384 1812 / 1589. LatentMoE (512 experts) MXFP4 at
// 47 rows 257 / 261, 56 287 / 282, 96 391 / 372; MXFP8 at 47 rows 296 / 317, 112 476 / 490, 131 542 /
// 541. H 288, I 160, 24 experts of 125 rows: MXFP4 49 / 61, MXFP8 50 / 54.
inline int mx_group_bm(int P, int E, int D, int I, bool mxfp4) {
  const int64_t tiles = ((int64_t)P / 128 + E / 2) * (((D < I ? D : I) + 255) / 256);
  return P <= (mxfp4 ? 48 : 112) * (int64_t)E || tiles < 256 ? 64 : 128;
}
// The gated sum of the experts' fp32 rows, out[t] + out_lo[t] = sum_j gates[t, j] Y[pos[t, j]] (all
// of D columns): rounded to bf16, and what that left over, in bf16 too.
hipError_t launch_combine_pair(const float* Y, const int32_t* pos, const float* gates, int T,
                               int D, int k, uint16_t* out, uint16_t* out_lo, hipStream_t s);
hipError_t launch_mx_gemm(Elt a, Elt w, const MxGemmParams& p, int max_mtiles, hipStream_t s);

}  // namespace moe
