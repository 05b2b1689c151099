// Entry points of the operators around the layer: token rows into expert order and back, the norms
// before and after a block, and gradient clipping. Argument checks and launches only; nothing here
// allocates or waits. Included once, by moe_api.cpp, after its helpers.
#pragma once

#include <initializer_list>

namespace {

bool float_type(moe_dtype_t t) { return t == MOE_F32 || t == MOE_BF16; }
Elt elt_of(moe_dtype_t t) { return t == MOE_F32 ? Elt::F32 : Elt::BF16; }
bool aligned32(const void* p) { return ((uintptr_t)p & 31u) == 0; }
bool absent_or_aligned(const void* p) { return !p || aligned16(p); }
// Arrays of 32-bit values, or absent ones.
bool words(std::initializer_list<const void*> all) {
  for (const void* p : all)
    if ((uintptr_t)p & 3u) return false;
  return true;
}

// ---- token rows
constexpr int kRowsMaxD = 1 << 20;
constexpr int64_t kRowsMaxUnits = (int64_t)1 << 25;   // waves of a launch: fewer than 2^32 lanes

int32_t rows_shape(int32_t T, int32_t D, int32_t k) {
  if (T < 0 || D < 16 || D % 16 || D > kRowsMaxD || k < 1 || k > kMaxK) return MOE_ERR_INVALID_ARG;
  if ((int64_t)T * ((D + 511) / 512) > kRowsMaxUnits || (int64_t)T * k > INT32_MAX)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

TokenRows token_rows_of(const int32_t* pos, const float* weights, int32_t T, int32_t D, int32_t k,
                        int32_t n_rows) {
  TokenRows r;
  r.pos = pos; r.weights = weights; r.T = T; r.D = D; r.k = k; r.n_rows = n_rows;
  return r;
}

// The sort's scratch: none for few pairs; the chunk counts; where chunks are too many for each
// workgroup to add them up, what the dispatch needs.
struct SortPlan {
  size_t counts = 0, perm = 0, scratch = 0, total = 0;
  bool chunked = false;
};
int32_t make_sort_plan(int32_t T, int32_t E, int32_t k, SortPlan* out) {
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > kMaxK || (int64_t)T * k > INT32_MAX)
    return MOE_ERR_INVALID_ARG;
  SortPlan pl;
  auto take = [&](size_t ints) {
    const size_t at = pl.total;
    pl.total += (ints * sizeof(int32_t) + kAlign - 1) / kAlign * kAlign;
    return at;
  };
  if (!sort_is_small(T, k)) {
    pl.chunked = positions_by_chunks(T, E, k);
    pl.scratch = take(dispatch_scratch_ints(T, E, k) / (pl.chunked ? 2 : 1));
    if (!pl.chunked) {
      pl.counts = take((size_t)E);
      pl.perm = take((size_t)T * k);
    }
  }
  *out = pl;
  return MOE_OK;
}

// ---- the block's norms
constexpr int kBlockMaxT = 1 << 23;
constexpr uint32_t kBlockFlags = MOE_BLOCK_NORM | MOE_GATE_TOKEN | MOE_GATE_ELEMENT | MOE_GATE_SIGMOID;

int32_t block_shape(int32_t T, int32_t H, moe_dtype_t dt, moe_dtype_t w_dt, uint32_t flags,
                    float scale, float eps, BlockShape* out) {
  if (T < 0 || T >= kBlockMaxT || H < 16 || H % 16 || H > kBlockMaxH) return MOE_ERR_INVALID_ARG;
  if (flags & ~kBlockFlags) return MOE_ERR_INVALID_ARG;
  if ((flags & MOE_GATE_TOKEN) && (flags & MOE_GATE_ELEMENT)) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 1e-30f) || !(eps < __builtin_inff()) || !(scale - scale == 0.f)) return MOE_ERR_INVALID_ARG;
  if (!float_type(dt) || !float_type(w_dt)) return MOE_ERR_UNSUPPORTED;
  BlockShape b;
  b.T = T; b.H = H; b.t = elt_of(dt); b.w_t = elt_of(w_dt);
  b.gate_kind = flags & MOE_GATE_TOKEN ? Gate::Token
                : flags & MOE_GATE_ELEMENT ? Gate::Element : Gate::None;
  b.sigmoid = flags & MOE_GATE_SIGMOID;
  b.norm = flags & MOE_BLOCK_NORM;
  b.scale = scale;
  b.eps = eps;
  *out = b;
  return MOE_OK;
}

int32_t block_workspace(const BlockShape& b, bool sums, const void* ws, size_t ws_bytes) {
  if (!sums || b.T == 0) return MOE_OK;
  return ws && ws_bytes >= block_part_floats(b.T, b.H) * sizeof(float) && aligned16(ws)
             ? MOE_OK : MOE_ERR_WORKSPACE;
}

// ---- clipping
constexpr int kClipMaxTensors = 1 << 16;
constexpr int64_t kClipMaxChunks = (int64_t)1 << 30;            // 16 TB
constexpr size_t kClipPartial = kClipGroups * sizeof(double);   // at the start of the plan

int32_t clip_check(const moe_clip_tensor_t* t, int32_t count, int64_t* chunks) {
  if (count < 0 || count > kClipMaxTensors || (count && !t)) return MOE_ERR_INVALID_ARG;
  int64_t c = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].n > (int64_t)1 << 43) return MOE_ERR_INVALID_ARG;
    if (!float_type(t[i].dt)) return MOE_ERR_UNSUPPORTED;
    if (t[i].n == 0) continue;
    const uintptr_t mask = t[i].dt == MOE_BF16 ? 1 : 3;
    if (!t[i].grad || ((uintptr_t)t[i].grad & mask) || ((uintptr_t)t[i].out & mask))
      return MOE_ERR_INVALID_ARG;
    c += clip_chunks(t[i].n, t[i].dt == MOE_BF16);
    if (c > kClipMaxChunks) return MOE_ERR_INVALID_ARG;
  }
  *chunks = c;
  return MOE_OK;
}

// Which capture the stream is in: 0 for none, else its number with the sign bit set.
int32_t capture_of(hipStream_t s, int32_t* capture) {
  hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (hipStreamGetCaptureInfo(s, &status, &id) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ERR_HIP;
  }
  *capture = status == hipStreamCaptureStatusActive ? (int32_t)((uint32_t)id | 0x80000000u) : 0;
  return MOE_OK;
}

}  // namespace

extern "C" {

int32_t moe_sort_tokens_workspace_size(int32_t T, int32_t E, int32_t k, size_t* bytes) {
  SortPlan pl;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int32_t rc = make_sort_plan(T, E, k, &pl);
  if (rc == MOE_OK) *bytes = pl.total;
  return rc;
}

int32_t moe_sort_tokens(const void* x, moe_dtype_t dt, const int32_t* idx, const float* weights,
                        int32_t T, int32_t D, int32_t E, int32_t k, void* rows, int32_t* offsets,
                        int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
  SortPlan pl;
  int32_t rc = rows_shape(T, D, k);
  if (rc == MOE_OK) rc = make_sort_plan(T, E, k, &pl);
  if (rc) return rc;
  if (!float_type(dt)) return MOE_ERR_UNSUPPORTED;
  if (!offsets || (T && (!x || !idx || !rows || !pos)) || !absent_or_aligned(x) ||
      !absent_or_aligned(rows) || !words({idx, weights, offsets, pos}))
    return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (pl.total == 0)
    return hip_status(launch_sort_small(idx, weights, T, D, E, k, elt_of(dt), x, rows, offsets, pos, s));
  if (!ws || ws_bytes < pl.total || !aligned16(ws)) return MOE_ERR_WORKSPACE;
  int32_t* const scratch = (int32_t*)((char*)ws + pl.scratch);
  if (pl.chunked)
    MOE_TRY(launch_positions(idx, T, E, k, scratch, offsets, pos, s));
  else
    MOE_TRY(launch_dispatch(idx, T, E, k, (int32_t*)((char*)ws + pl.counts), offsets,
                            (int32_t*)((char*)ws + pl.perm), pos, scratch, 0, nullptr,
                            DispatchExtras(), s));
  return hip_status(launch_spread_rows(token_rows_of(pos, weights, T, D, k, T * k), elt_of(dt), x,
                                       rows, s));
}

int32_t moe_sort_tokens_backward(const void* drows, const void* x, moe_dtype_t dt,
                                 const int32_t* pos, const float* weights, int32_t T, int32_t D,
                                 int32_t k, int32_t n_rows, void* dx, moe_dtype_t dx_dt,
                                 float* dweights, void* stream) {
  const int32_t rc = rows_shape(T, D, k);
  if (rc) return rc;
  if (n_rows < 0) return MOE_ERR_INVALID_ARG;
  if (!float_type(dt) || !float_type(dx_dt)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if ((n_rows && !drows) || !pos || !dx || (dweights && !x) || !absent_or_aligned(drows) ||
      !absent_or_aligned(x) || !aligned16(dx) || !words({pos, weights, dweights}))
    return MOE_ERR_INVALID_ARG;
  return hip_status(launch_gather_rows(token_rows_of(pos, weights, T, D, k, n_rows), elt_of(dt),
                                       drows, nullptr, elt_of(dx_dt), dx, x, dweights,
                                       (hipStream_t)stream));
}

int32_t moe_unsort_tokens(const void* rows, moe_dtype_t dt, const int32_t* pos,
                          const float* weights, const void* add, int32_t T, int32_t D, int32_t k,
                          int32_t n_rows, void* y, moe_dtype_t y_dt, void* stream) {
  const int32_t rc = rows_shape(T, D, k);
  if (rc) return rc;
  if (n_rows < 0) return MOE_ERR_INVALID_ARG;
  if (!float_type(dt) || !float_type(y_dt)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if ((n_rows && !rows) || !pos || !y || !absent_or_aligned(rows) || !absent_or_aligned(add) ||
      !aligned16(y) || !words({pos, weights}))
    return MOE_ERR_INVALID_ARG;
  return hip_status(launch_gather_rows(token_rows_of(pos, weights, T, D, k, n_rows), elt_of(dt),
                                       rows, add, elt_of(y_dt), y, nullptr, nullptr,
                                       (hipStream_t)stream));
}

int32_t moe_unsort_tokens_backward(const void* dy, moe_dtype_t dy_dt, const void* rows,
                                   moe_dtype_t dt, const int32_t* pos, const float* weights,
                                   int32_t T, int32_t D, int32_t k, int32_t n_rows, void* drows,
                                   float* dweights, void* stream) {
  const int32_t rc = rows_shape(T, D, k);
  if (rc) return rc;
  if (n_rows < 0) return MOE_ERR_INVALID_ARG;
  if (!float_type(dt) || !float_type(dy_dt)) return MOE_ERR_UNSUPPORTED;
  if (!dweights && dt != dy_dt) return MOE_ERR_UNSUPPORTED;   // rows of dy's type alone
  if (T == 0) return MOE_OK;
  if (!dy || !pos || (n_rows && !drows) || (dweights && n_rows && !rows) || !aligned16(dy) ||
      !absent_or_aligned(rows) || !absent_or_aligned(drows) || !words({pos, weights, dweights}))
    return MOE_ERR_INVALID_ARG;
  const TokenRows r = token_rows_of(pos, weights, T, D, k, n_rows);
  hipStream_t s = (hipStream_t)stream;
  if (!dweights) return hip_status(launch_spread_rows(r, elt_of(dt), dy, drows, s));
  return hip_status(launch_spread_dot(r, elt_of(dy_dt), dy, elt_of(dt), rows, drows, dweights, s));
}

int32_t moe_block_norm(const void* x, const void* w, void* h, int32_t T, int32_t H, moe_dtype_t dt,
                       moe_dtype_t w_dt, float eps, void* stream) {
  BlockShape b;
  const int32_t rc = block_shape(T, H, dt, w_dt, 0, 1.f, eps, &b);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!x || !h || !aligned16(x) || !aligned16(h) || !absent_or_aligned(w)) return MOE_ERR_INVALID_ARG;
  BlockForward p;
  p.x = x; p.w_next = w; p.h = h;
  return hip_status(launch_block_forward(b, p, (hipStream_t)stream));
}

int32_t moe_block_residual(const void* x, const void* f, const void* w, const void* gate,
                           const void* w_next, void* y, void* h, int32_t T, int32_t H,
                           moe_dtype_t dt, moe_dtype_t w_dt, uint32_t flags, float scale, float eps,
                           void* stream) {
  BlockShape b;
  const int32_t rc = block_shape(T, H, dt, w_dt, flags, scale, eps, &b);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!x || !f || !y || ((b.gate_kind == Gate::None) != (gate == nullptr)) || !aligned16(x) ||
      !aligned16(f) || !aligned16(y) || !absent_or_aligned(w) || !absent_or_aligned(w_next) ||
      !absent_or_aligned(h) || !absent_or_aligned(gate))
    return MOE_ERR_INVALID_ARG;
  BlockForward p;
  p.x = x; p.f = f; p.w = w; p.gate = gate; p.w_next = w_next; p.y = y; p.h = h;
  return hip_status(launch_block_forward(b, p, (hipStream_t)stream));
}

int32_t moe_block_backward_workspace_size(int32_t T, int32_t H, size_t* bytes) {
  BlockShape b;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int32_t rc = block_shape(T, H, MOE_BF16, MOE_BF16, 0, 1.f, 1.f, &b);
  if (rc == MOE_OK) *bytes = block_part_floats(T, H) * sizeof(float);
  return rc;
}

int32_t moe_block_norm_backward(const void* dh, moe_dtype_t dh_dt, const void* x, const void* w,
                                const void* dres, void* dx, float* dw, int32_t T, int32_t H,
                                moe_dtype_t dt, moe_dtype_t w_dt, float eps, void* ws,
                                size_t ws_bytes, void* stream) {
  BlockShape b;
  int32_t rc = block_shape(T, H, dt, w_dt, 0, 1.f, eps, &b);
  if (rc) return rc;
  if (dh_dt != dt && dh_dt != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (T && (!dh || !x || !dx)) return MOE_ERR_INVALID_ARG;
  if (!absent_or_aligned(dh) || !absent_or_aligned(x) || !absent_or_aligned(w) ||
      !absent_or_aligned(dres) || !absent_or_aligned(dx) || !words({dw}))
    return MOE_ERR_INVALID_ARG;
  if ((rc = block_workspace(b, dw != nullptr, ws, ws_bytes))) return rc;
  BlockBackward p;
  p.dy = dres; p.y = x; p.dh = dh; p.dh_t = elt_of(dh_dt); p.w_next = w; p.dx = dx; p.dw_next = dw;
  p.part = (float*)ws;
  return hip_status(launch_block_backward(b, p, (hipStream_t)stream));
}

int32_t moe_block_residual_backward(const void* dy, const void* f, const void* w, const void* gate,
                                    const void* y, const void* dh, moe_dtype_t dh_dt,
                                    const void* w_next, void* dx, void* df, float* dw, void* dgate,
                                    float* dw_next, int32_t T, int32_t H, moe_dtype_t dt,
                                    moe_dtype_t w_dt, uint32_t flags, float scale, float eps,
                                    void* ws, size_t ws_bytes, void* stream) {
  BlockShape b;
  int32_t rc = block_shape(T, H, dt, w_dt, flags, scale, eps, &b);
  if (rc) return rc;
  if (dh && dh_dt != dt && dh_dt != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if ((dw_next && T && !dh) || (dw && T && !f)) return MOE_ERR_INVALID_ARG;
  if (T && (!f || !dx || !df || (!dy && !dh) || (dh && !y) ||
            ((b.gate_kind == Gate::None) != (gate == nullptr)) || (dgate && !gate)))
    return MOE_ERR_INVALID_ARG;
  const void* all[] = {dy, f, w, gate, y, dh, w_next, dx, df, dgate};
  for (const void* q : all)
    if (!absent_or_aligned(q)) return MOE_ERR_INVALID_ARG;
  if (!words({dw, dw_next})) return MOE_ERR_INVALID_ARG;
  if ((rc = block_workspace(b, dw || dw_next, ws, ws_bytes))) return rc;
  BlockBackward p;
  p.dy = dy; p.f = f; p.w = w; p.gate = gate; p.y = y; p.dh = dh; p.dh_t = elt_of(dh_dt);
  p.w_next = dh ? w_next : nullptr;   // (without dh nothing may meet it)
  p.dx = dx; p.df = df; p.dw = dw; p.dgate = dgate; p.dw_next = dw_next;
  p.part = (float*)ws;
  return hip_status(launch_block_backward(b, p, (hipStream_t)stream));
}

int32_t moe_clip_plan_size(const moe_clip_tensor_t* tensors, int32_t count, size_t* bytes) {
  int64_t chunks = 0;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int32_t rc = clip_check(tensors, count, &chunks);
  if (rc == MOE_OK) *bytes = kClipPartial + (size_t)chunks * sizeof(ClipChunk);
  return rc;
}

int32_t moe_clip_plan(const moe_clip_tensor_t* tensors, int32_t count, void* plan,
                      size_t plan_bytes, moe_clip_t* clip, void* stream) {
  int64_t chunks = 0;
  const int32_t rc = clip_check(tensors, count, &chunks);
  if (rc) return rc;
  if (!clip) return MOE_ERR_INVALID_ARG;
  if (!plan || !aligned32(plan) || plan_bytes < kClipPartial + (size_t)chunks * sizeof(ClipChunk))
    return MOE_ERR_WORKSPACE;
  int32_t capture = 0;
  const int32_t e = capture_of((hipStream_t)stream, &capture);
  if (e && chunks) return e;   // (nothing to write: nothing that a GPU is needed for)
  ClipChunk* table = (ClipChunk*)((char*)plan + kClipPartial);
  ClipBatch batch;
  memset(&batch, 0, sizeof(batch));
  int32_t in_place = 1;
  int held = 0;
  int64_t first = 0;
  for (int32_t i = 0; i < count; ++i) {
    const moe_clip_tensor_t& t = tensors[i];
    if (t.n == 0) continue;
    void* out = t.out ? t.out : t.grad;
    if (out != t.grad) in_place = 0;
    const bool bf16 = t.dt == MOE_BF16;
    batch.t[held++] = {(const char*)t.grad, (char*)out, t.n, first, bf16};
    first += clip_chunks(t.n, bf16);
    if (held == kClipPerLaunch) {
      MOE_TRY(launch_clip_table(batch, held, first - batch.t[0].first, table, (hipStream_t)stream));
      held = 0;
    }
  }
  if (held)
    MOE_TRY(launch_clip_table(batch, held, first - batch.t[0].first, table, (hipStream_t)stream));
  clip->plan = plan;
  clip->chunks = chunks;
  clip->in_place = in_place;
  clip->capture = capture;
  return MOE_OK;
}

int32_t moe_clip_grads(const moe_clip_t* clip, float max_norm, float* norm, void* stream) {
  if (!clip || !clip->plan || !aligned32(clip->plan) || clip->chunks < 0 ||
      clip->chunks > kClipMaxChunks || !norm || ((uintptr_t)norm & 3) || !(max_norm >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (clip->capture) {
    int32_t now = 0;
    const int32_t e = capture_of((hipStream_t)stream, &now);
    if (e) return e;
    if (now != clip->capture) return MOE_ERR_INVALID_ARG;
  }
  return hip_status(launch_clip((const ClipChunk*)((const char*)clip->plan + kClipPartial),
                                clip->chunks, clip->in_place != 0, max_norm, (double*)clip->plan,
                                norm, (hipStream_t)stream));
}

}  // extern "C"
