// Products of block-scaled (OCP microscaling) matrices on the gfx950 matrix cores:
//   C[m, n] = act( sum over blocks b of 2^(sa[m, b] + sw[n, b] - 254) sum_{i in b} A[m, i] W[n, i] )
// through v_mfma_scale_f32_*_f8f6f4, which takes E2M1 or E4M3 elements and one E8M0 scale per 32
// of them for each operand and accumulates in fp32. A may instead be e4m3 codes with one fp32
// scale per row (unit block scales; the row scale multiplies the result), which is how the MoE
// layer's expert rows meet block-scaled expert weights.
//
// What the instruction rounds (measured with two nonzero products at chosen distances): of each
// eight consecutive k, products are cut toward zero to multiples of 2^(e - 13), e the exponent of
// the largest of them; the groups of eight are then added in fp32. Two E2M1 operands lose nothing
// (products are multiples of 1/4 up to 36). With an E4M3 operand a group loses up to 7 * 2^-13 of its
// largest product: random data ends 4.5e-6 (E2M1 on the other side) or 1.5e-5 off, inside a bf16
// result's half step, but where large products cancel it can be all of the result. fp32 results
// are offered for two E2M1 operands alone.
//
// Three kernels:
//  - mx_rows_kernel, few rows: the weights are the matrix core's first operand, 16 weight rows
//    against 16, 32 or 64 rows of A, and the workgroup's waves split K and join in LDS, so that
//    the launch is one pass over W by N / 16 workgroups.
//  - mx_tile_kernel, many rows: BM x BN tiles staged through LDS, dense or grouped by expert.
//  - mx_persist_kernel, expert products over longer K: the same tiles as one pipeline per CU.
//
// Order of k (32x32x64 / 16x16x128): lane group g holds, of an E4M3 operand, k 16g .. 16g + 15
// and KS/2 + 16g .. KS/2 + 16g + 15 (KS = 64 or 128: the two 16-byte halves of its 32 bytes), of
// an E2M1 operand k 32g .. 32g + 31, and the scale byte it passes covers k 32g .. 32g + 31.
// Included once, by backward.hip: these kernels are part of that object, so that the library stays the
// objects that its parts are linked from elsewhere (host code under the sanitizers).
#pragma once

#include <algorithm>

#include "common.hpp"
#include "mx.hpp"

namespace moe {
namespace {
namespace mx_tiles {

// Operand formats of the kernels: E4M3 with block scales, E2M1 with block scales, E4M3 with a
// row scale (A only).
enum Fmt : int { kE4 = 0, kE2 = 1, kE4Row = 2 };
template <int F> constexpr int kBits = F == kE2 ? 4 : 8;
template <int F> constexpr int kCode = F == kE2 ? 4 : 0;  // the instruction's format field

__device__ __forceinline__ i32x8_t frag(uint4 lo, uint4 hi) {
  return i32x8_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z,
                 (int)hi.w};
}
constexpr uint4 kZero4 = {0, 0, 0, 0};

__device__ __forceinline__ void store8(const MxGemmParams& p, int64_t row, int col, const float* v) {
  if (p.out_f32) {
    float* o = (float*)p.C + row * p.N + col;
    *(float4*)o = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {  // one rounding, to nearest even, at the end
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
    *(uint4*)((uint16_t*)p.C + row * p.N + col) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------------------- few rows
// Workgroup (x, y): weight rows 16x .. 16x + 15 against rows 16*TB*y .. of A. Wave w takes the
// K-steps of 128 in its contiguous share; loads of U steps are in flight together. Bound by round
// trips: 1 x 2688 x 1856 (8 x 4 bits) 4.6 us, 64 x 1856 x 2688 (4 bits, every workgroup reads all of
// A from L2) 7.0 us. Eight waves give each 2 or 3 K-steps there, one batch of loads.
template <int FA, int FW, int TB, int NW>
__global__ __launch_bounds__(64 * NW) void mx_rows_kernel(MxGemmParams p) {
  constexpr int U = TB >= 4 ? 2 : 4;
  constexpr int CA = kBits<FA> == 8 ? 2 : 1, CW = kBits<FW> == 8 ? 2 : 1;  // 16-byte chunks
  __shared__ float part[NW][TB][16][17];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int n0 = blockIdx.x * 16;
  const int m0 = blockIdx.y * 16 * TB;
  const int nb = p.K / kMxBlockElts;        // blocks of a row
  const int nk = cdiv(p.K, 128);
  const int per = cdiv(nk, NW);
  const int k_lo = wave * per, k_hi = min(nk, k_lo + per);
  const int64_t kbw = (int64_t)p.K * kBits<FW> / 8, kba = (int64_t)p.K * kBits<FA> / 8;
  const uint8_t* w = p.W + (int64_t)(n0 + r) * kbw;
  const uint8_t* wx = p.w_mx + (int64_t)(n0 + r) * nb;
  const uint8_t* a[TB];
  const uint8_t* ax[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int64_t row = min(m0 + 16 * t + r, p.M - 1);
    a[t] = p.A + row * kba;
    ax[t] = p.a_mx + row * nb;
  }
  f32x4_t acc[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // Chunks past this wave's share are read from the row's start and zeroed on the weights' side;
  // no branch on them: loads whose use is conditional are moved to it, one by one, instead of
  // being in flight together.
  const int kend = min(p.K, k_hi * 128);
  auto el_of = [&](int ks, int c, int chunks) {
    return ks * 128 + (chunks == 2 ? 64 * c + 16 * g : 32 * g);
  };
  for (int k0 = k_lo; k0 < k_hi; k0 += U) {
    uint4 wf[U][CW], af[U][TB][CA];
    int ws[U], as[U][TB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int blk = min((k0 + u) * 4 + g, nb - 1);
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        const int el = el_of(k0 + u, c, CW);
        wf[u][c] = *(const uint4*)(w + (int64_t)(el < kend ? el : 0) * kBits<FW> / 8);
      }
      ws[u] = wx[blk];
#pragma unroll
      for (int t = 0; t < TB; ++t) {
#pragma unroll
        for (int c = 0; c < CA; ++c) {
          const int el = el_of(k0 + u, c, CA);
          af[u][t][c] = *(const uint4*)(a[t] + (int64_t)(el < kend ? el : 0) * kBits<FA> / 8);
        }
        as[u][t] = ax[t][blk];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int c = 0; c < CW; ++c)
        if (el_of(k0 + u, c, CW) >= kend) wf[u][c] = kZero4;
#pragma unroll
      for (int t = 0; t < TB; ++t)
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            frag(wf[u][0], CW == 2 ? wf[u][CW - 1] : kZero4),
            frag(af[u][t][0], CA == 2 ? af[u][t][CA - 1] : kZero4), acc[t], kCode<FW>, kCode<FA>,
            0, ws[u], 0, as[u][t]);
    }
  }
  // lane: C[row m0 + 16 t + lane % 16][column n0 + 4 g + i]
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][t][r][4 * g + i] = acc[t][i];
  __syncthreads();
  // the waves' shares of K added in wave order, 8 columns per thread
  const int item = threadIdx.x;
  if (item < TB * 32) {
    const int t = item >> 5, row = (item >> 1) & 15, c = (item & 1) * 8;
    const int m = m0 + 16 * t + row;
    if (m < p.M) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float s = part[0][t][row][c + q];
#pragma unroll
        for (int x = 1; x < NW; ++x) s += part[x][t][row][c + q];
        v[q] = p.sqrelu ? sqrelu(s) : s;
      }
      store8(p, m, n0 + c, v);
    }
  }
}

// ------------------------------------------------------------------------------- many rows
// A workgroup of WGM x WGN waves owns a BM x BN tile of C. Each K-step stages 128 elements of
// every A and W row in LDS (128 bytes of E4M3, 64 of E2M1) by buffer loads straight to LDS, 1 KB
// an instruction; the 16-byte chunks of a row are XOR-swizzled by choosing which global chunk a
// lane fetches, so that 16 consecutive rows at one chunk index fall on distinct banks. Block
// scales go through LDS too, 16 bytes (512 elements) of every row at a time, loaded one such
// super-step ahead through registers: read directly by the lanes that need them, scattered dwords
// per K-step and wave would take as many address cycles as the operands. The first half of the
// waves load the operands, the other half the scales: a wave's wait for its scales would wait for
// its operand loads in flight too. All waves multiply.
// 8192 x 3712 x 2688 (4 bits, 256 x 256): 61 us, 2.7 PFLOP/s, where the products alone reach 5.2: the
// matrix cores are busy a third of the time, the rest is fragment reads from LDS between barriers
// and 8 us of first loads and epilogue a round. 1999 x 1040 x 4096 (8 bits, 64 x 128): 23 us.
template <int SL> __device__ __forceinline__ int swz(int row) {
  return SL == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}
template <int SL> __device__ __forceinline__ int slot(int row, int chunk) {
  return row * SL + ((chunk ^ swz<SL>(row)) << 4);
}
// A raw buffer resource over [base, base + bytes) in scalar registers: accesses at offsets beyond
// it are skipped.
__device__ __forceinline__ i32x4_t rsrc(const void* base, int64_t bytes) {
  const uint64_t b = (uint64_t)base;
  return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                 __builtin_amdgcn_readfirstlane((int)((b >> 32) & 0xFFFF)),
                 __builtin_amdgcn_readfirstlane((int)(uint32_t)bytes), 0x00020000};
}
// 16 bytes per lane from buffer offset voff + soff to LDS byte lds + 16 * lane. Written as an
// instruction, not through the builtin: for every LDS read after the builtin the compiler waits
// until all such loads have landed (it cannot tell the stages apart), which leaves one K-step in
// flight however many stages there are. The load has no register result; its landing is awaited by
// the explicit vmcnt waits of the main loop. The nop is the wait state between a write of m0 and a
// load that uses it.
__device__ __forceinline__ void dma16(i32x4_t r, uint32_t lds, uint32_t voff, int soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_of(const void* q) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)q;
}

// A barrier of the workgroup for LDS alone: it does not wait for loads in flight. The fences are what
// tells the compiler that other waves' LDS writes become visible here; to a clobber on an asm
// statement it need not react for arrays whose address never leaves the kernel.
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The 16 bytes v shifted down by `by` bytes, and those from byte `valid` on set to 0x7F (scale 1).
__device__ __forceinline__ uint4 trim_scales(uint4 v, int by, int valid) {
  uint32_t w[8] = {v.x, v.y, v.z, v.w, 0, 0, 0, 0};
  const int d = by >> 2, b = 8 * (by & 3);
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t lo = w[j], hi = w[j + 1];
#pragma unroll
    for (int q = 1; q < 4; ++q) {
      lo = d == q ? w[j + q] : lo;
      hi = d == q ? w[j + q + 1] : hi;
    }
    o[j] = (uint32_t)((((uint64_t)hi << 32) | lo) >> b);
    const int n = min(max(valid - 4 * j, 0), 4);
    const uint32_t keep = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
    o[j] = (o[j] & keep) | (0x7F7F7F7Fu & ~keep);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Scales are kept as one array of dwords per K-step: read as dwords of 16-byte entries, a wave's 32
// rows meet 16 banks and take 8 clocks instead of 2.3.
template <int ROWS>
__device__ __forceinline__ void put4(uint32_t (&sc)[4][ROWS], int row, uint4 v) {
  sc[0][row] = v.x; sc[1][row] = v.y; sc[2][row] = v.z; sc[3][row] = v.w;
}

// The local-th tile of a group of mt_g M-tiles: bands of 8 M-tiles, M fastest inside.
template <int BN>
__device__ __forceinline__ void place_tile(int local, int mt_g, int nN, int& mt, int& n0) {
  constexpr int GB = 8;
  const int first = (local / (GB * nN)) * GB;
  const int gm = min(GB, mt_g - first);
  const int within = local - first * nN;
  n0 = (within / gm) * BN;
  mt = first + within % gm;
}
// Logical tile L -> group, first row, rows, first column.
template <int BM, int BN>
__device__ __forceinline__ bool tile_of(const MxGemmParams& p, int L, int& g, int& row0, int& rows,
                                        int& n0) {
  const int nN = cdiv(p.N, BN);
  int local, mt_g;
  if (p.mt_start) {
    if (L >= p.mt_start[p.G] * nN) return false;
    // the last group whose first M-tile is at or before this one: counted by the wave's lanes, one
    // round trip to the list where a search would take a chain of them
    const int key = L / nN, lane = threadIdx.x & 63;
    int below = 0;
    for (int i = 0; i < p.G; i += 64)
      below += __popcll(__ballot(i + lane < p.G && p.mt_start[min(i + lane, p.G - 1)] <= key));
    g = __builtin_amdgcn_readfirstlane(below) - 1;
    mt_g = p.mt_start[g + 1] - p.mt_start[g];
    local = L - p.mt_start[g] * nN;
  } else {
    g = 0;
    mt_g = cdiv(p.M, BM);
    local = L;
    if (L >= mt_g * nN) return false;
  }
  int mt;
  place_tile<BN>(local, mt_g, nN, mt, n0);
  row0 = (p.mt_start ? p.offs[g] : 0) + mt * BM;
  rows = min(BM, (p.mt_start ? p.offs[g + 1] : p.M) - row0);
  return rows > 0;
}

// One K-step (128 elements) of a BM x BN tile from the stage at st (A rows, then W rows) and its
// scales, a dword per row. mid() is what a wave issues for later (the loads of a stage ahead): between
// the two halves of K, where it goes out while the matrix core works on the first (with the scales'
// layout: 8192 tokens of 128 MXFP4 experts 1218 -> 1202 us, 512 x 3712 x 2688 in 4 bits 15.0 -> 13.5
// to 14.5), but before them where both halves' fragments would not fit beside the accumulators
// (256 x 256 in 8 bits: spills).
template <int B>
__device__ __forceinline__ i32x8_t read_frag(const uint8_t* base, int row, int s, int lg) {
  constexpr int SL = B * 16;
  if constexpr (B == 8)
    return frag(*(const uint4*)(base + slot<SL>(row, 4 * s + lg)),
                *(const uint4*)(base + slot<SL>(row, 4 * s + 2 + lg)));
  else
    return frag(*(const uint4*)(base + slot<SL>(row, 2 * s + lg)), kZero4);
}
template <int BM, int BN, int WGM, int WGN, int FA, int FW, class Mid>
__device__ __forceinline__ void mma_step(f32x16_t (&acc)[BM / WGM / 32][BN / WGN / 32],
                                         const uint8_t* st, const uint32_t* sc, int lane, int wm,
                                         int wn, Mid&& mid) {
  constexpr int SA = kBits<FA> * 16, WM = BM / WGM, WN = BN / WGN, MB = WM / 32, NB = WN / 32;
  constexpr int W0 = FA == kE4Row ? 0 : BM;   // first W row among the staged scales
  constexpr bool kMidway = 16 * MB * NB + 2 * (MB * kBits<FA> + NB * kBits<FW>) <= 160;  // registers
  const int lg = lane >> 5, lr = lane & 31;
  if constexpr (!kMidway) mid();
  int xa[MB], xw[NB];   // this lane's scale bytes at bits 0 and 16 (k-sub 0 and 1)
#pragma unroll
  for (int i = 0; i < MB; ++i)
    xa[i] = FA == kE4Row ? 0x7F7F7F7F : (int)(sc[wm * WM + i * 32 + lr] >> (8 * lg));
#pragma unroll
  for (int j = 0; j < NB; ++j)
    xw[j] = (int)(sc[W0 + wn * WN + j * 32 + lr] >> (8 * lg));
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    i32x8_t a[MB], b[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) a[i] = read_frag<kBits<FA>>(st, wm * WM + i * 32 + lr, s, lg);
#pragma unroll
    for (int j = 0; j < NB; ++j)
      b[j] = read_frag<kBits<FW>>(st + BM * SA, wn * WN + j * 32 + lr, s, lg);
    if (kMidway && s == 1) mid();
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[i][j] = s == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                 a[i], b[j], acc[i][j], kCode<FA>, kCode<FW>, 0, xa[i], 0, xw[j])
                           : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                 a[i], b[j], acc[i][j], kCode<FA>, kCode<FW>, 2, xa[i], 2, xw[j]);
  }
}

template <int BM, int BN, int WGM, int WGN, int NS, int FA, int FW>
__global__ __launch_bounds__(64 * WGM * WGN, 2)
void mx_tile_kernel(MxGemmParams p) {
  constexpr int NW = WGM * WGN, DW = NW / 2;                // waves, waves that load operands
  constexpr int SA = kBits<FA> * 16, SW = kBits<FW> * 16;   // bytes of a row's K-step
  constexpr int WM = BM / WGM, WN = BN / WGN, MB = WM / 32, NB = WN / 32;
  constexpr int RA = 1024 / SA, RW = 1024 / SW;             // rows per 1-KB load
  constexpr int LA = SA / 16, LW = SW / 16;                 // lanes per row
  constexpr int GA = BM / (RA * DW), GW = BN / (RW * DW);   // 1-KB loads per loading wave
  constexpr int STAGE = BM * SA + BN * SW;
  constexpr int SROWS = (FA == kE4Row ? 0 : BM) + BN;       // rows whose scales are staged
  constexpr int ST = 64 * (NW - DW), SR = (SROWS + ST - 1) / ST;
  constexpr int EPW = WN + 4;
  static_assert(GA >= 1 && GW >= 1 && BM % (RA * DW) == 0 && BN % (RW * DW) == 0, "1-KB loads");
  static_assert(WM % 32 == 0 && WN % 32 == 0 && DW % 2 == 0 && NS >= 2, "tile shape");
  static_assert(NW * 16 * EPW * 4 <= NS * STAGE, "epilogue strips fit in the stages");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * STAGE];
  __shared__ uint32_t sc[2][4][SROWS];   // of K-step q of a super-step: [q]

  int g, row0, rows, n0;
  if (!tile_of<BM, BN>(p, xcd_logical_block(blockIdx.x, gridDim.x), g, row0, rows, n0)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN, lg = lane >> 5, lr = lane & 31;
  const bool loads = wave < DW;
  const int kba = p.K * kBits<FA> / 8, kbw = p.K * kBits<FW> / 8;   // bytes of a row
  const int nb = p.K / kMxBlockElts, nk = cdiv(p.K, 128);
  const int tail_a = kba % SA, tail_w = kbw % SW;   // bytes of a partial last K-step

  const i32x4_t ra = rsrc(p.A, (int64_t)p.a_rows * kba);
  const i32x4_t rw = rsrc(p.W + (int64_t)g * p.N * kbw, (int64_t)p.N * kbw);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_of(smem)) + wave * 1024;
  const int ca = ((lane % LA) ^ swz<SA>(wave * RA + lane / LA)) << 4;
  const int cw = ((lane % LW) ^ swz<SW>(wave * RW + lane / LW)) << 4;
  constexpr uint32_t kOut = 0xFFFFFFF0u;   // an offset past every buffer: the load is skipped
  uint32_t oa[GA], ow[GW];
  if (loads) {
#pragma unroll
    for (int i = 0; i < GA; ++i) {
      const int r = (wave + DW * i) * RA + lane / LA;
      const int src = r < rows ? (p.a_gather ? p.a_gather[row0 + r] : row0 + r) : 0;
      oa[i] = r < rows ? (uint32_t)src * (uint32_t)kba + ca : kOut;
    }
#pragma unroll
    for (int i = 0; i < GW; ++i)
      ow[i] = (uint32_t)min(n0 + (wave + DW * i) * RW + lane / LW, p.N - 1) * (uint32_t)kbw + cw;
  }

  auto issue = [&](int ks, int stage) {
    if (!loads) return;
    const bool last = ks == nk - 1;
    const bool la = !(last && tail_a) || ca < tail_a, lw = !(last && tail_w) || cw < tail_w;
    const uint32_t st = lds0 + stage * STAGE;
#pragma unroll
    for (int i = 0; i < GA; ++i) dma16(ra, st + DW * i * 1024, la ? oa[i] : kOut, ks * SA);
#pragma unroll
    for (int i = 0; i < GW; ++i)
      dma16(rw, st + BM * SA + DW * i * 1024, lw ? ow[i] : kOut, ks * SW);
  };
  // the chunks of a partial last K-step that lie past K, zeroed once the stage has landed
  auto fix_tail = [&](uint8_t* st) {
    if (loads) {
      if (tail_a && ca >= tail_a)
#pragma unroll
        for (int i = 0; i < GA; ++i) *(uint4*)(st + (wave + DW * i) * 1024 + lane * 16) = kZero4;
      if (tail_w && cw >= tail_w)
#pragma unroll
        for (int i = 0; i < GW; ++i)
          *(uint4*)(st + BM * SA + (wave + DW * i) * 1024 + lane * 16) = kZero4;
    }
    barrier();
  };

  // scales: thread t of the other waves carries rows t, t + ST, ... of (A rows, W rows). A row's
  // 16 bytes are loaded from where they start, or from the array's last 16 (the array is longer
  // than that) and moved down.
  const int st0 = tid - 64 * DW;
  const uint8_t* sp[SR];
  int64_t sleft[SR];   // bytes of the array from the row's first scale on
  uint4 sv[SR];
  if (!loads) {
#pragma unroll
    for (int i = 0; i < SR; ++i) {
      const int r = min(st0 + ST * i, SROWS - 1);
      if (FA != kE4Row && r < BM) {
        const int rr = min(r, rows - 1);
        const int64_t src = p.a_gather ? p.a_gather[row0 + rr] : row0 + rr;
        sp[i] = p.a_mx + src * nb;
        sleft[i] = ((int64_t)p.a_rows - src) * nb;
      } else {
        const int64_t n = min(n0 + r - (SROWS - BN), p.N - 1);
        sp[i] = p.w_mx + ((int64_t)g * p.N + n) * nb;
        sleft[i] = ((int64_t)(p.mt_start ? p.G - g : 1) * p.N - n) * nb;
      }
    }
  }
  auto fetch_scales = [&](int ss) {
    if (loads) return;
#pragma unroll
    for (int i = 0; i < SR; ++i) {
      typedef uint32_t u32x4a1 __attribute__((ext_vector_type(4), aligned(1)));
      const u32x4a1 x = *(const u32x4a1*)(sp[i] + min((int64_t)16 * ss, sleft[i] - 16));
      sv[i] = make_uint4(x.x, x.y, x.z, x.w);
    }
  };
  auto put_scales = [&](int ss) {
    if (loads) return;
#pragma unroll
    for (int i = 0; i < SR; ++i)
      if (st0 + ST * i < SROWS)
        put4(sc[ss & 1], st0 + ST * i,
             trim_scales(sv[i], (int)max((int64_t)0, 16 * ss + 16 - sleft[i]), nb - 16 * ss));
  };

  f32x16_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // K-step ks + NS - 1 is in flight while K-step ks is multiplied; before ks a wave waits until
  // at most the loads of the stages after ks are outstanding, then the barrier publishes the
  // stage (and the scales of the super-step) and frees the stage before.
  constexpr int PER = GA + GW;
  static_assert((NS - 1) * PER < 64, "vmcnt range");
  auto wait_ahead = [&](int ahead) {
#define MOE_VMCNT(n) __builtin_amdgcn_s_waitcnt((((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8)))
    if constexpr (NS >= 4) { if (ahead >= 2) { MOE_VMCNT(2 * PER); return; } }
    if constexpr (NS >= 3) { if (ahead >= 1) { MOE_VMCNT(PER); return; } }
    MOE_VMCNT(0);
#undef MOE_VMCNT
  };
  fetch_scales(0);
#pragma unroll
  for (int q = 0; q < NS - 1; ++q)
    if (q < nk) issue(q, q);
  put_scales(0);
  const int nss = cdiv(nk, 4);
  int cur = 0, ahead = NS - 1;   // stages of K-step ks and of the one issued next
  for (int ss = 0; ss < nss; ++ss) {
    if (ss + 1 < nss) fetch_scales(ss + 1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int ks = 4 * ss + q;
      if (ks >= nk) break;
      wait_ahead(min(NS - 2, nk - 1 - ks));
      barrier();
      uint8_t* st = smem + cur * STAGE;
      if (ks == nk - 1 && (tail_a || tail_w)) fix_tail(st);
      mma_step<BM, BN, WGM, WGN, FA, FW>(acc, st, sc[ss & 1][q], lane, wm, wn, [&]() {
        if (ks + NS - 1 < nk) issue(ks + NS - 1, ahead);
      });
      cur = cur + 1 == NS ? 0 : cur + 1;
      ahead = ahead + 1 == NS ? 0 : ahead + 1;
    }
    // the other buffer was last read a whole super-step ago
    if (ss + 1 < nss) put_scales(ss + 1);
  }
  barrier();   // every wave is done with the stages: the epilogue reuses them

  // acc[i][j][r] is C[wm*WM + i*32 + (r/4)*8 + lg*4 + r%4][wn*WN + j*32 + lr]; strips of 16 rows
  // go through this wave's own LDS so that a lane stores 8 consecutive columns
  float* ep = (float*)smem + wave * 16 * EPW;
  constexpr int CG = WN / 8, ITEMS = 16 * CG / 64;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int rr = 0; rr < 8; ++rr)
          ep[((rr >> 2) * 8 + lg * 4 + (rr & 3)) * EPW + j * 32 + lr] = acc[i][j][8 * h + rr];
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        const int item = it * 64 + lane, srow = item / CG, cg = item % CG;
        const int rl = wm * WM + i * 32 + h * 16 + srow, col = n0 + wn * WN + cg * 8;
        const float4 lo = *(const float4*)(ep + srow * EPW + cg * 8);
        const float4 hi = *(const float4*)(ep + srow * EPW + cg * 8 + 4);
        float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        if (rl < rows && col < p.N) {
          const int row = row0 + rl;
          if constexpr (FA == kE4Row) {
            const float rs = p.a_row[p.a_gather ? p.a_gather[row] : row];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= rs;
          }
          if (p.sqrelu)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = sqrelu(v[q]);
          store8(p, row, col, v);
        }
      }
    }
}

// ---------------------------------------------------------------------- experts, persistent
// Expert products (A: e4m3 rows with a scale each) by one workgroup of 8 waves per CU that walks
// BM x 256 tiles: workgroup b runs on die b % 8 and takes every (grid / 8)-th tile of that die's
// contiguous range. The K-steps of all its tiles form one pipeline: while a tile's last K-steps are
// multiplied and its result is stored, the next tile's first ones are landing, so that neither the
// first loads nor the epilogue are waited for. What the loading waves need of the next tile (group,
// rows and their sources) is looked up by the other waves, one load's round trip per K-step, and
// passed through LDS, so that a loading wave waits for no load but the operands; so are the row
// scales that the epilogue reads. Without the products a launch over 49152 rows of 128 MXFP4
// experts (K 2688, N 1856) takes 269 of its 365 us, without the loads 285: operands come through
// the L1 at 15 to 17 B per clock and CU, in 64-byte requests of which 82% hit the L2 and the rest
// is each expert read once; lines fetched into L2 ahead of use change nothing.
constexpr int kStripRows = 8;   // rows of a wave's epilogue strip
constexpr int kLookups = 5;     // phases of a tile's lookup
constexpr int kPersistSteps = 8;   // least K-steps of a tile

template <int BM, int NS, int FW>
__global__ __launch_bounds__(512, 2) void mx_persist_kernel(MxGemmParams p) {
  constexpr int BN = 256, WGM = 2, WGN = 4, DW = 4;         // waves; the first DW load operands
  constexpr int SA = 128, SW = kBits<FW> * 16;              // bytes of a row's K-step
  constexpr int WM = BM / WGM, WN = BN / WGN, MB = WM / 32, NB = WN / 32;
  constexpr int RA = 1024 / SA, RW = 1024 / SW;             // rows per 1-KB load
  constexpr int LA = SA / 16, LW = SW / 16;                 // lanes per row
  constexpr int GA = BM / (RA * DW), GW = BN / (RW * DW);   // 1-KB loads per loading wave
  constexpr int STAGE = BM * SA + BN * SW;
  constexpr int EPW = WN + 4, CG = WN / 8, ITEMS = kStripRows * CG / 64;
  static_assert(GA >= 1 && GW >= 1 && BM % (RA * DW) == 0 && BN % (RW * DW) == 0, "1-KB loads");
  static_assert(WM % 32 == 0 && NS >= 2 && BM <= 64 * DW && BN == 64 * DW, "tile shape");
  static_assert(kStripRows * CG % 64 == 0, "whole strips");
  // a tile's description is written by its predecessor's K-step 3 and read from K-step nk - NS + 1
  static_assert(kPersistSteps - NS + 1 >= kLookups - 1, "lookups end before the loads need them");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * STAGE];
  __shared__ uint32_t sc[2][4][BN];   // of K-step q of a super-step: [q]
  __shared__ __attribute__((aligned(16))) float strips[8][kStripRows][EPW];
  __shared__ int tinfo[2][4];      // group, first row, rows, first column of a tile
  __shared__ int tsrc[2][BM];      // source row of each of its rows, -1 past the last
  __shared__ float trow[2][BM];    // and its scale

  const int nN = cdiv(p.N, BN), total = p.mt_start[p.G] * nN;
  const int die = blockIdx.x % kXcds, step = gridDim.x / kXcds, share = cdiv(total, kXcds);
  const int hi = min(total, (die + 1) * share);
  int L = die * share + (int)blockIdx.x / kXcds;
  if (L >= hi) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN, lg = lane >> 5, lr = lane & 31;
  const bool loads = wave < DW;
  const int kba = p.K, kbw = p.K * kBits<FW> / 8;   // bytes of a row
  const int nb = p.K / kMxBlockElts, nk = cdiv(p.K, 128), nss = cdiv(nk, 4);
  const int tail_a = kba % SA, tail_w = kbw % SW;   // bytes of a partial last K-step

  // The other waves: tile Lt's description to LDS buffer b, by phases whose loads are used in the
  // next one; then its scales, a thread a row.
  const int st0 = tid - 64 * DW;
  int near0 = 0, near1 = 0, ng = 0, first_mt = 0, end_mt = 0, off0 = 0, off1 = 0, nrows = 0, nn0 = 0;
  int src = 0;
  float row_scale = 0.f;
  auto lookup = [&](int phase, int Lt, int b) {
    if (loads) return;
    const int key = Lt / nN;
    if (phase == 0) {
      near0 = p.mt_start[min(lane, p.G - 1)];
      near1 = p.mt_start[min(64 + lane, p.G - 1)];
    } else if (phase == 1) {   // the last group that starts at or before this M-tile
      int below = __popcll(__ballot(lane < p.G && near0 <= key)) +
                  __popcll(__ballot(64 + lane < p.G && near1 <= key));
      for (int i = 128; i < p.G; i += 64)
        below += __popcll(__ballot(i + lane < p.G && p.mt_start[min(i + lane, p.G - 1)] <= key));
      ng = __builtin_amdgcn_readfirstlane(below) - 1;
      first_mt = p.mt_start[ng];
      end_mt = p.mt_start[ng + 1];
      off0 = p.offs[ng];
      off1 = p.offs[ng + 1];
    } else if (phase == 2) {
      int mt;
      place_tile<BN>(Lt - first_mt * nN, end_mt - first_mt, nN, mt, nn0);
      const int row0 = off0 + mt * BM;
      nrows = min(BM, off1 - row0);
      if (st0 < 4) tinfo[b][st0] = st0 == 0 ? ng : st0 == 1 ? row0 : st0 == 2 ? nrows : nn0;
      src = row0 + min(min(st0, BM - 1), nrows - 1);
      if (p.a_gather) src = p.a_gather[src];
    } else if (phase == 3) {
      if (st0 < BM) tsrc[b][st0] = st0 < nrows ? src : -1;
      row_scale = p.a_row[src];
    } else if (st0 < BM) {
      trow[b][st0] = row_scale;
    }
  };
  const uint8_t* sp = p.w_mx;   // this thread's row of scales, and the array's bytes from it on
  int64_t sleft = 16;
  uint4 sv = kZero4;
  auto scales_of = [&]() {      // the looked-up tile's
    const int64_t n = min(nn0 + st0, p.N - 1);
    sp = p.w_mx + ((int64_t)ng * p.N + n) * nb;
    sleft = ((int64_t)(p.G - ng) * p.N - n) * nb;
  };
  auto fetch_scales = [&](int ss) {
    if (loads) return;
    typedef uint32_t u32x4a1 __attribute__((ext_vector_type(4), aligned(1)));
    const u32x4a1 x = *(const u32x4a1*)(sp + min((int64_t)16 * ss, sleft - 16));
    sv = make_uint4(x.x, x.y, x.z, x.w);
  };
  auto put_scales = [&](int ss, int b) {
    if (loads) return;
    put4(sc[b], st0, trim_scales(sv, (int)max((int64_t)0, 16 * ss + 16 - sleft), nb - 16 * ss));
  };

  // the loading waves: sources of the tile whose K-steps are being issued
  const i32x4_t ra = rsrc(p.A, (int64_t)p.a_rows * kba);
  i32x4_t rw = ra;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_of(smem)) + wave * 1024;
  const int ca = ((lane % LA) ^ swz<SA>(wave * RA + lane / LA)) << 4;
  const int cw = ((lane % LW) ^ swz<SW>(wave * RW + lane / LW)) << 4;
  constexpr uint32_t kOut = 0xFFFFFFF0u;   // an offset past every buffer: the load is skipped
  uint32_t oa[GA], ow[GW];
  auto sources = [&](int b) {
    if (!loads) return;
    const int g = __builtin_amdgcn_readfirstlane(tinfo[b][0]);
    const int n0 = __builtin_amdgcn_readfirstlane(tinfo[b][3]);
    rw = rsrc(p.W + (int64_t)g * p.N * kbw, (int64_t)p.N * kbw);
#pragma unroll
    for (int i = 0; i < GA; ++i) {
      const int s = tsrc[b][(wave + DW * i) * RA + lane / LA];
      oa[i] = s >= 0 ? (uint32_t)s * (uint32_t)kba + ca : kOut;
    }
#pragma unroll
    for (int i = 0; i < GW; ++i)
      ow[i] = (uint32_t)min(n0 + (wave + DW * i) * RW + lane / LW, p.N - 1) * (uint32_t)kbw + cw;
  };
  int islot = 0, cslot = 0;    // stages issued into next, multiplied next
  int flying = 0, iks = 0;     // stages issued and not yet multiplied; the next K-step to issue ...
  bool inext = false;          // ... of the next tile instead of the current one
  auto issue = [&]() {
    if (loads) {
      const bool last = iks == nk - 1;
      const bool la = !(last && tail_a) || ca < tail_a, lw = !(last && tail_w) || cw < tail_w;
      const uint32_t st = lds0 + islot * STAGE;
#pragma unroll
      for (int i = 0; i < GA; ++i) dma16(ra, st + DW * i * 1024, la ? oa[i] : kOut, iks * SA);
#pragma unroll
      for (int i = 0; i < GW; ++i)
        dma16(rw, st + BM * SA + DW * i * 1024, lw ? ow[i] : kOut, iks * SW);
    }
    ++iks;
    ++flying;
    islot = islot + 1 == NS ? 0 : islot + 1;
  };
  constexpr int PER = GA + GW;
  static_assert((NS - 2) * PER < 64 && NS <= 4, "vmcnt range");
  // until at most `ahead` later stages are outstanding (result stores in between wait longer)
  auto wait_ahead = [&](int ahead) {
    if (!loads) return;
#define MOE_VMCNT(n) __builtin_amdgcn_s_waitcnt((((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8)))
    if constexpr (NS >= 4) { if (ahead >= 2) { MOE_VMCNT(2 * PER); return; } }
    if constexpr (NS >= 3) { if (ahead >= 1) { MOE_VMCNT(PER); return; } }
    MOE_VMCNT(0);
#undef MOE_VMCNT
  };
  // the missing part of a partial last K-step reads as zero elements
  auto fix_tail = [&](uint8_t* st) {
    if (loads) {
      if (tail_a && ca >= tail_a)
#pragma unroll
        for (int i = 0; i < GA; ++i) *(uint4*)(st + (wave + DW * i) * 1024 + lane * 16) = kZero4;
      if (tail_w && cw >= tail_w)
#pragma unroll
        for (int i = 0; i < GW; ++i)
          *(uint4*)(st + BM * SA + (wave + DW * i) * 1024 + lane * 16) = kZero4;
    }
    barrier();
  };

  for (int ph = 0; ph < kLookups; ++ph) lookup(ph, L, 0);
  scales_of();
  fetch_scales(0);
  put_scales(0, 0);
  barrier();
  sources(0);
  while (flying < NS - 1) issue();
  const int last_ss = (nk - 1) / 4 * 4;   // K-step that starts the last super-step
  for (int tb = 0, sb = 0;; tb ^= 1) {    // LDS buffers of the tile, the super-step
    const bool more = L + step < hi;
    const int row0 = __builtin_amdgcn_readfirstlane(tinfo[tb][1]);
    const int rows = __builtin_amdgcn_readfirstlane(tinfo[tb][2]);
    const int n0 = __builtin_amdgcn_readfirstlane(tinfo[tb][3]);
    f32x16_t acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    for (int ks = 0; ks < nk; ++ks) {
      const int q = ks & 3, ss = ks >> 2;
      wait_ahead(flying - 1);
      barrier();               // publishes the stage (and its scales), frees the one before
      uint8_t* st = smem + cslot * STAGE;
      if (ks == nk - 1 && (tail_a || tail_w)) fix_tail(st);
      mma_step<BM, BN, WGM, WGN, kE4Row, FW>(acc, st, sc[sb][q], lane, wm, wn, [&]() {
        // the stage NS - 1 ahead, the next tile's first ones after this one's last
        if (iks == nk && !inext && more) {
          sources(tb ^ 1);
          inext = true;
          iks = 0;
        }
        if (iks < nk) issue();
        if (q == 0 && ss + 1 < nss) fetch_scales(ss + 1);
        if (more && ks < kLookups) lookup(ks, L + step, tb ^ 1);
        if (more && ks == last_ss) {
          scales_of();
          fetch_scales(0);
        }
      });
      --flying;
      cslot = cslot + 1 == NS ? 0 : cslot + 1;
      if (q == 3 && ss + 1 < nss) {   // the other buffer was last read before this step's barrier
        put_scales(ss + 1, sb ^ 1);
        sb ^= 1;
      }
    }
    if (more) {
      put_scales(0, sb ^ 1);
      sb ^= 1;
    }
    // acc[i][j][r] is C[wm*WM + i*32 + (r/4)*8 + lg*4 + r%4][wn*WN + j*32 + lr]; strips of 8 rows
    // go through this wave's own LDS so that a lane stores 8 consecutive columns
    float (*ep)[EPW] = strips[wave];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int rr = 0; rr < 4; ++rr) ep[lg * 4 + rr][j * 32 + lr] = acc[i][j][4 * h + rr];
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
          const int srow = (it * 64 + lane) / CG, cg = lane % CG;
          const int rl = wm * WM + i * 32 + h * 8 + srow, col = n0 + wn * WN + cg * 8;
          const float4 x = *(const float4*)&ep[srow][cg * 8];
          const float4 y = *(const float4*)&ep[srow][cg * 8 + 4];
          const float rs = trow[tb][rl];
          float v[8] = {x.x * rs, x.y * rs, x.z * rs, x.w * rs, y.x * rs, y.y * rs, y.z * rs, y.w * rs};
          if (p.sqrelu)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = sqrelu(v[e]);
          if (rl < rows && col < p.N) store8(p, row0 + rl, col, v);
        }
      }
    if (!more) break;
    L += step;
    inext = false;
  }
}

template <int BM, int NS, int FW>
hipError_t run_persist(const MxGemmParams& p, int mtiles, hipStream_t s) {
  const int64_t tiles = (int64_t)mtiles * cdiv(p.N, 256);
  if (tiles <= 0) return hipSuccess;
  if (tiles > INT32_MAX / 512) return hipErrorInvalidValue;
  const int grid = std::min(cdiv((int)tiles, kXcds) * kXcds, std::max(kXcds, persist_grid() / 2 / kXcds * kXcds));
  hipLaunchKernelGGL((mx_persist_kernel<BM, NS, FW>), dim3(grid), dim3(512), 0, s, p);
  return hipGetLastError();
}

template <int BM, int BN, int WGM, int WGN, int NS, int FA, int FW>
hipError_t run_tile(const MxGemmParams& p, int mtiles, hipStream_t s) {
  const int64_t tiles = (int64_t)mtiles * cdiv(p.N, BN);
  if (tiles <= 0) return hipSuccess;
  if (tiles > INT32_MAX / 512) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WGM, WGN, NS, FA, FW>),
                     dim3(cdiv((int)tiles, kXcds) * kXcds), dim3(64 * WGM * WGN), 0, s, p);
  return hipGetLastError();
}

// Tile shapes by their BM: 256 x 256 on 8 waves, one workgroup per CU; 128 x 256 (128 x 128 where
// W has 8 bits) and 64 x 128 on 4 waves, two per CU. A K-step's loads take over a microsecond to
// land, so as many stages as LDS holds are in flight.
template <int FA, int FW>
constexpr int stages(int BM, int BN, int lds) {
  const int stage = (BM * kBits<FA> + BN * kBits<FW>) * 16;
  const int n = (lds - 32 * ((FA == kE4Row ? 0 : BM) + BN)) / stage;
  return n > 4 ? 4 : n;
}
constexpr int kLds = 160 * 1024;
constexpr int tile_bn(int bm, int w_bits) { return bm == 256 ? 256 : (bm == 128 && w_bits == 4 ? 256 : 128); }
template <int FA, int FW, int BM>
hipError_t run_shape(const MxGemmParams& p, int mtiles, hipStream_t s) {
  constexpr int BN = tile_bn(BM, kBits<FW>);
  // Workgroups of a CU: one of 8 waves, two, or, for the short K of expert products on 64 rows (few
  // steps to wait for between a tile's first loads and its result), three of fewer stages: 24024
  // rows of 512 MXFP8 experts, K 512, N 1024: 106 us with 2 stages each, 114 as two with 3.
  constexpr int CU = BM == 256 ? 1 : FA == kE4Row && BM == 64 ? 3 : 2;
  constexpr int NS = stages<FA, FW>(BM, BN, kLds / CU);
  return run_tile<BM, BN, 2, BM == 256 ? 4 : 2, NS, FA, FW>(p, mtiles, s);
}

template <int FA, int FW, int TB>
hipError_t run_rows(const MxGemmParams& p, hipStream_t s) {
  hipLaunchKernelGGL((mx_rows_kernel<FA, FW, TB, 8>), dim3(p.N / 16, cdiv(p.M, 16 * TB)), dim3(512),
                     0, s, p);
  return hipGetLastError();
}

// Estimated microseconds of a dense product on tiles of BM rows: rounds over the CUs of K-steps
// and a fixed part (first loads and epilogue). Measured on 4096 x 4096 outputs, K of 512 to 4096:
// 1.1 / 1.37 / 0.57 us per K-step and 8 / 7 / 3 us fixed; a CU that holds one workgroup of the
// smaller shapes instead of two takes about 0.55 of their step. 8192 x 3712 x 2688 (4 bits): 67 us
// on 256 rows, 69 on 128, 116 on 64; 512 x 3712 x 2688: 27, 21.5 and 14.
double tile_time(int bm, int w_bits, int M, int N, int K) {
  const int tiles = cdiv(M, bm) * cdiv(N, tile_bn(bm, w_bits)), cap = bm == 256 ? 256 : 512;
  const double c = bm == 256 ? 1.1 : (bm == 128 ? 1.37 : 0.57) * (tiles <= 256 ? 0.55 : 1.0);
  return cdiv(tiles, cap) * (cdiv(K, 128) * c + (bm == 256 ? 8 : bm == 128 ? 7 : 3));
}

template <int FA, int FW>
hipError_t run_dense(const MxGemmParams& p, hipStream_t s) {
  if (p.M <= 16) return run_rows<FA, FW, 1>(p, s);
  if (p.M <= 32) return run_rows<FA, FW, 2>(p, s);
  // Few rows: every 16 weight rows meet 64 rows of A, which re-read each other's operands from L2
  // (about 10 TB/s over the chip) but fill it where tiles would leave CUs idle.
  const double re_read = (double)cdiv(p.M, 64) * (p.N / 16) * p.K * (64 * kBits<FA> + 16 * kBits<FW>) / 8;
  double best_t = p.M <= 512 ? 4 + re_read / 10e6 : 1e30;
  int best = 0;
  for (int bm = 64; bm <= 256; bm *= 2) {
    const double t = tile_time(bm, kBits<FW>, p.M, p.N, p.K);
    if (p.M > 64 && t < best_t) { best_t = t; best = bm; }
  }
  switch (best) {
    case 256: return run_shape<FA, FW, 256>(p, cdiv(p.M, 256), s);
    case 128: return run_shape<FA, FW, 128>(p, cdiv(p.M, 128), s);
    case 64: return run_shape<FA, FW, 64>(p, cdiv(p.M, 64), s);
    default: return run_rows<FA, FW, 4>(p, s);
  }
}

// Stages of the persistent tiles, beside the scales, strips and descriptions.
template <int FW>
constexpr int persist_stages(int BM) {
  const int n = (kLds - 2 * 256 * 16 - 8 * kStripRows * 68 * 4 - 16 * BM - 64) /
                ((8 * BM + kBits<FW> * 256) * 16);
  return n > 4 ? 4 : n;
}
// Expert products: the persistent tiles where K fills their pipeline (8 steps, which the lookup of
// the next tile needs too). Microseconds, persistent / a workgroup per tile: 49152 rows of 128
// MXFP4 experts, K 2688, N 1856 365 / 393 and K 1856, N 2688 404 / 433; 24024 rows of 512 MXFP8
// experts, K 1024, N 512 81 / 90, but K 512, N 1024 (4 steps, with the lookups after the last) 115
// / 106. (Nano's figures with bf16 results; its second product with the fp32 rows it stores: 461 under
// the profiler.)
template <int FW>
hipError_t run_grouped(const MxGemmParams& p, int mtiles, hipStream_t s) {
  const bool walk = cdiv(p.K, 128) >= kPersistSteps;
  if (p.bm == 64)
    return walk ? run_persist<64, persist_stages<FW>(64), FW>(p, mtiles, s)
                : run_shape<kE4Row, FW, 64>(p, mtiles, s);
  if (p.bm == 128)
    return walk ? run_persist<128, persist_stages<FW>(128), FW>(p, mtiles, s)
                : run_shape<kE4Row, FW, 128>(p, mtiles, s);
  return hipErrorInvalidValue;
}

}  // namespace mx_tiles
}  // namespace

using namespace mx_tiles;

hipError_t launch_mx_gemm(Elt a, Elt w, const MxGemmParams& p, int max_mtiles, hipStream_t s) {
  if (p.K < 32 || p.K % 32 || p.N < 16 || p.N % 16 || !p.w_mx) return hipErrorInvalidValue;
  // 32-bit operand offsets
  constexpr int64_t kLim = ((int64_t)1 << 31) - 1;
  const int ab = a == Elt::MXFP4 ? 4 : 8, wb = w == Elt::MXFP4 ? 4 : 8;
  if ((int64_t)p.a_rows * p.K * ab / 8 > kLim || (int64_t)p.N * p.K * wb / 8 > kLim)
    return hipErrorInvalidValue;
  if (w != Elt::MXFP4 && w != Elt::MXFP8) return hipErrorInvalidValue;
  const bool w4 = w == Elt::MXFP4;
  if (p.mt_start) {  // grouped: e4m3 rows with a row scale against block-scaled experts
    if (a != Elt::FP8 || !p.a_row || !p.offs) return hipErrorInvalidValue;
    return w4 ? run_grouped<kE2>(p, max_mtiles, s) : run_grouped<kE4>(p, max_mtiles, s);
  }
  if (p.M <= 0) return hipSuccess;
  if (!p.a_mx || p.a_gather || p.a_rows != p.M) return hipErrorInvalidValue;
  if (a == Elt::MXFP4) return w4 ? run_dense<kE2, kE2>(p, s) : run_dense<kE2, kE4>(p, s);
  if (a == Elt::MXFP8) return w4 ? run_dense<kE4, kE2>(p, s) : run_dense<kE4, kE4>(p, s);
  return hipErrorInvalidValue;
}

}  // namespace moe
