"""ctypes binding of libmoe_mi355x.so (the gfx950 MoE layer library).

Argument marshalling only: torch tensors supply device memory and the current stream; every step
of the layer runs in the library's HIP kernels. The library must have been built
(``python -m sparse_moe_layer_05_amd.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mi355x.so")

MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_MXFP4, MOE_MXFP8 = 0, 1, 2, 3, 4
_EXPERT_DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "e4m3": MOE_FP8_E4M3, "mxfp4": MOE_MXFP4,
                  "mxfp8": MOE_MXFP8}
MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
PATH_AUTO, PATH_GROUPED, PATH_STREAM, ROUTING_GIVEN, SAVED_IN_WORKSPACE = 0, 1, 2, 4, 8
WGRAD_BF16, MX_GROUPED = 16, 32
# "grouped_mx": matrix-core tiles for MXFP4 / MXFP8 experts (many tokens); "few": the few-token
# layer (an entry point of its own)
_PATHS = {"auto": PATH_AUTO, "grouped": PATH_GROUPED, "stream": PATH_STREAM,
          "grouped_mx": MX_GROUPED, "few": PATH_AUTO}
FEW_TOKENS = 16
_MX_FORMATS = {"mxfp4": MOE_MXFP4, "mxfp8": MOE_MXFP8}
MX_BLOCK = 32

EXPORTS = ("moe_workspace_size", "moe_layer_forward", "latent_moe_forward", "moe_route",
           "moe_dispatch_workspace_size", "moe_dispatch", "moe_bias_update",
           "moe_backward_workspace_size", "moe_layer_forward_train", "moe_layer_backward",
           "moe_layer_forward_static", "moe_few_workspace_size", "moe_few_forward",
           "moe_mx_quantize", "moe_mx_dequantize", "moe_mx_gemm",
           "moe_sort_tokens_workspace_size", "moe_sort_tokens", "moe_sort_tokens_backward",
           "moe_unsort_tokens", "moe_unsort_tokens_backward",
           "moe_block_norm", "moe_block_residual", "moe_block_backward_workspace_size",
           "moe_block_norm_backward", "moe_block_residual_backward",
           "moe_clip_plan_size", "moe_clip_plan", "moe_clip_grads",
           "moe_status_str",
           "moe_trace_enable",
           "moe_trace_count", "moe_trace_read", "moe_trace_reset")


class MoeDesc(C.Structure):
    _fields_ = [("T", C.c_int32), ("H", C.c_int32), ("E", C.c_int32), ("k", C.c_int32),
                ("I", C.c_int32), ("I_shared", C.c_int32), ("latent", C.c_int32),
                ("act_dtype", C.c_int32), ("expert_dtype", C.c_int32), ("flags", C.c_uint32)]


class MoeWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("x", "W_r", "b", "W_up", "W_down", "s_up", "s_down",
                                          "Ws_up", "Ws_down", "W_in", "W_out")]


class MoeRouting(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("idx", "gates", "counts", "offsets", "perm", "pos",
                                          "logits")]


class MoeGrads(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("dx", "dW_r", "dW_up", "dW_down", "dWs_up",
                                          "dWs_down", "dW_in", "dW_out")]


class MoeClipTensor(C.Structure):
    _fields_ = [("grad", C.c_void_p), ("out", C.c_void_p), ("n", C.c_int64), ("dt", C.c_int32)]


class MoeClip(C.Structure):
    _fields_ = [("plan", C.c_void_p), ("chunks", C.c_int64), ("in_place", C.c_int32),
                ("capture", C.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_str(code)} ({code})")
        self.code = code


_lock = threading.Lock()
_lib = None


def lib() -> C.CDLL:
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing "
                                   "(run python -m sparse_moe_layer_05_amd.build)")
            L = C.CDLL(LIB_PATH)
            vp, i32, sz = C.c_void_p, C.c_int32, C.c_size_t
            L.moe_workspace_size.argtypes = [C.POINTER(MoeDesc), C.POINTER(sz)]
            L.moe_few_workspace_size.argtypes = [C.POINTER(MoeDesc), C.POINTER(sz)]
            for fn in (L.moe_layer_forward, L.latent_moe_forward, L.moe_few_forward):
                fn.argtypes = [C.POINTER(MoeDesc), C.POINTER(MoeWeights), vp, vp, sz,
                               C.POINTER(MoeRouting), vp]
            L.moe_layer_forward_static.argtypes = [C.POINTER(MoeDesc), C.POINTER(MoeWeights),
                                                   vp, C.POINTER(MoeRouting), vp]
            L.moe_route.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
            L.moe_dispatch_workspace_size.argtypes = [i32, i32, i32, C.POINTER(sz)]
            L.moe_dispatch.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
            L.moe_bias_update.argtypes = [vp, vp, i32, C.c_float, vp, vp]
            L.moe_backward_workspace_size.argtypes = [C.POINTER(MoeDesc), C.POINTER(sz)]
            L.moe_layer_backward.argtypes = [C.POINTER(MoeDesc), C.POINTER(MoeWeights), vp,
                                             C.POINTER(MoeGrads), vp, sz, vp]
            L.moe_layer_forward_train.argtypes = [C.POINTER(MoeDesc), C.POINTER(MoeWeights), vp,
                                                  vp, sz, vp]
            L.moe_mx_quantize.argtypes = [vp, i32, C.c_int64, i32, i32, vp, vp, vp]
            L.moe_mx_dequantize.argtypes = [vp, vp, i32, C.c_int64, i32, vp, i32, vp]
            L.moe_mx_gemm.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, i32, vp]
            f32, u32 = C.c_float, C.c_uint32
            L.moe_sort_tokens_workspace_size.argtypes = [i32, i32, i32, C.POINTER(sz)]
            L.moe_sort_tokens.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
            L.moe_sort_tokens_backward.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, i32,
                                                   vp, vp]
            L.moe_unsort_tokens.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp]
            L.moe_unsort_tokens_backward.argtypes = [vp, i32, vp, i32, vp, vp, i32, i32, i32, i32,
                                                     vp, vp, vp]
            L.moe_block_norm.argtypes = [vp, vp, vp, i32, i32, i32, i32, f32, vp]
            L.moe_block_residual.argtypes = [vp] * 7 + [i32, i32, i32, i32, u32, f32, f32, vp]
            L.moe_block_backward_workspace_size.argtypes = [i32, i32, C.POINTER(sz)]
            L.moe_block_norm_backward.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                                  f32, vp, sz, vp]
            L.moe_block_residual_backward.argtypes = [vp] * 6 + [i32] + [vp] * 6 + [
                i32, i32, i32, i32, u32, f32, f32, vp, sz, vp]
            L.moe_clip_plan_size.argtypes = [C.POINTER(MoeClipTensor), i32, C.POINTER(sz)]
            L.moe_clip_plan.argtypes = [C.POINTER(MoeClipTensor), i32, vp, sz, C.POINTER(MoeClip),
                                        vp]
            L.moe_clip_grads.argtypes = [C.POINTER(MoeClip), f32, vp, vp]
            L.moe_status_str.argtypes = [i32]
            L.moe_trace_enable.argtypes = [i32, C.c_char_p]
            L.moe_trace_count.argtypes = []
            L.moe_trace_read.argtypes = [i32, C.POINTER(C.c_char_p), C.POINTER(C.c_float)]
            L.moe_trace_reset.argtypes = []
            for name in EXPORTS:
                getattr(L, name).restype = C.c_int32
            L.moe_status_str.restype = C.c_char_p
            L.moe_trace_reset.restype = None
            _lib = L
    return _lib


def status_str(code: int) -> str:
    return lib().moe_status_str(code).decode()


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return MOE_FP8_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _used_on(stream, *tensors):
    """Tell the caching allocator that `tensors` (allocated on the current stream) are in use on
    `stream` too, so that their memory is not handed out again before that stream's work ends."""
    if stream is None:
        return
    for t in tensors:
        if t is not None:
            if not isinstance(stream, torch.Stream):   # another library's: see _launch
                stream = torch.cuda.ExternalStream(stream.cuda_stream, device=t.device)
            t.record_stream(stream)


def _raw(stream, device):
    """Raw handle of the stream that _launch takes."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index) if device.type == "cuda" else 0


def _torch_stream(stream, device):
    """The same as a torch stream."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream, device=device)


class _Own:
    """What a prepared call has allocated. Marked as in use on every other stream that the call runs
    on, it is not handed out again before that stream's work ends, though the object be dropped."""

    def __init__(self, device, *tensors):
        self.device, self.tensors = device, tensors
        self.made_on = _raw(None, device)

    def used_on(self, stream):
        if _raw(stream, self.device) != self.made_on:
            _used_on(_torch_stream(stream, self.device), *self.tensors)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def expert_dtype_code(x, W_up, s_up=None, W_in=None, expert_dtype=None) -> int:
    """moe_dtype_t of the expert weights: given by name, or read off the tensors (float / bf16
    weights: their dtype; uint8 codes with fp32 scales: e4m3; with uint8 block scales: MXFP8,
    or MXFP4 when a row holds half as many bytes as the expert input width)."""
    if expert_dtype is not None:
        return _EXPERT_DTYPES[expert_dtype]
    if W_up.dtype in (torch.uint8, torch.float8_e4m3fn) and s_up is not None \
            and s_up.dtype == torch.uint8:
        D = W_in.shape[0] if W_in is not None else x.shape[1]
        return MOE_MXFP4 if 2 * W_up.shape[-1] == D else MOE_MXFP8
    return _dtype_code(W_up)


def _need(t, shape, what, dtype=None, device=None):
    if t is None:
        raise ValueError(f"{what} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")


def check_shapes(desc, x, W_r, b, W_up, W_down, s_up=None, s_down=None, Ws_up=None,
                 Ws_down=None, W_in=None, W_out=None):
    """Every tensor must have the shape, dtype and device the descriptor implies: the library
    only sees pointers, so a mismatch would make it read outside a buffer."""
    T, H, E, I, Is, L = desc.T, desc.H, desc.E, desc.I, desc.I_shared, desc.latent
    D = L or H
    act = x.dtype
    dev = x.device
    _need(W_r, (E, H), "W_r", act, dev)
    _need(b, (E,), "b", torch.float32, dev)
    ed = desc.expert_dtype
    if ed in (MOE_F32, MOE_BF16):
        _need(W_up, (E, I, D), "W_up", act, dev)
        _need(W_down, (E, D, I), "W_down", act, dev)
    elif ed == MOE_FP8_E4M3:
        _need(W_up, (E, I, D), "W_up", W_up.dtype, dev)
        _need(W_down, (E, D, I), "W_down", W_down.dtype, dev)
        _need(s_up, (E, I), "s_up", torch.float32, dev)
        _need(s_down, (E, D), "s_down", torch.float32, dev)
    else:  # MXFP4 packs two elements per byte, MXFP8 one; one uint8 scale per 32 along K
        per = 2 if ed == MOE_MXFP4 else 1
        _need(W_up, (E, I, D // per), "W_up", W_up.dtype, dev)
        _need(W_down, (E, D, I // per), "W_down", W_down.dtype, dev)
        _need(s_up, (E, I, D // 32), "s_up", torch.uint8, dev)
        _need(s_down, (E, D, I // 32), "s_down", torch.uint8, dev)
    if ed not in (MOE_F32, MOE_BF16) and W_up.element_size() != 1:
        raise ValueError("8- and 4-bit expert weights are passed as 1-byte tensors")
    if Is:
        _need(Ws_up, (Is, H), "Ws_up", act, dev)
        _need(Ws_down, (H, Is), "Ws_down", act, dev)
    if L:
        _need(W_in, (L, H), "W_in", act, dev)
        _need(W_out, (H, L), "W_out", act, dev)


def make_desc(x, W_r, W_up, k, Ws_up=None, W_in=None, path="auto", routing_given=False,
              s_up=None, expert_dtype=None):
    T, H = x.shape
    E, I = W_up.shape[0], W_up.shape[1]
    d = MoeDesc()
    d.T, d.H, d.E, d.k, d.I = T, H, E, k, I
    d.I_shared = Ws_up.shape[0] if Ws_up is not None else 0
    d.latent = W_in.shape[0] if W_in is not None else 0
    d.act_dtype = _dtype_code(x)
    d.expert_dtype = expert_dtype_code(x, W_up, s_up, W_in, expert_dtype)
    d.flags = _PATHS[path] | (ROUTING_GIVEN if routing_given else 0)
    return d


def workspace_size(desc: MoeDesc, few: bool = False) -> int:
    n = C.c_size_t(0)
    name = "moe_few_workspace_size" if few else "moe_workspace_size"
    _check(getattr(lib(), name)(C.byref(desc), C.byref(n)), name)
    return n.value


def alloc_routing(T: int, E: int, k: int, device) -> dict:
    i32 = dict(dtype=torch.int32, device=device)
    return dict(idx=torch.empty((T, k), **i32), gates=torch.empty((T, k), dtype=torch.float32,
                                                                  device=device),
                counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                perm=torch.empty(T * k, **i32), pos=torch.empty((T, k), **i32),
                logits=torch.empty((T, E), dtype=torch.float32, device=device))


class Layer:
    """One layer call prepared once (descriptor, weights struct, workspace, outputs), so that a
    benchmark loop or a graph capture can replay ``__call__`` without any allocation."""

    def __init__(self, x, W_r, b, W_up, W_down, k, *, s_up=None, s_down=None, Ws_up=None,
                 Ws_down=None, W_in=None, W_out=None, path="auto", routing=None,
                 routing_given=False, out=None, expert_dtype=None, no_alloc=False):
        self.desc = make_desc(x, W_r, W_up, k, Ws_up, W_in, path, routing_given, s_up,
                              expert_dtype)
        check_shapes(self.desc, x, W_r, b, W_up, W_down, s_up, s_down, Ws_up, Ws_down, W_in,
                     W_out)
        if out is not None:
            _need(out, x.shape, "out", x.dtype, x.device)
        w = MoeWeights()
        w.x, w.W_r, w.b, w.W_up, w.W_down = _p(x), _p(W_r), _p(b), _p(W_up), _p(W_down)
        w.s_up, w.s_down = _p(s_up), _p(s_down)
        w.Ws_up, w.Ws_down, w.W_in, w.W_out = _p(Ws_up), _p(Ws_down), _p(W_in), _p(W_out)
        self.w = w
        self._keep = [x, W_r, b, W_up, W_down, s_up, s_down, Ws_up, Ws_down, W_in, W_out]
        self.y = out if out is not None else torch.empty_like(x)
        self.no_alloc = no_alloc
        few = path == "few"      # moe_few_forward: at most FEW_TOKENS tokens, few launches
        if few and no_alloc:
            raise ValueError("path 'few' takes its own workspace: no_alloc is not offered")
        if no_alloc:          # moe_layer_forward_static: the library's own per-GPU scratch
            self.ws_bytes, self.ws = 0, None
        else:
            self.ws_bytes = workspace_size(self.desc, few)
            self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=x.device)
        self.routing = routing
        self.r = None
        if routing is not None:
            r = MoeRouting()
            for name, _ in MoeRouting._fields_:
                setattr(r, name, _p(routing.get(name)))
            self.r = r
        self.fn_name = "moe_few_forward" if few else \
            "latent_moe_forward" if self.desc.latent else "moe_layer_forward"
        self.fn = getattr(lib(), self.fn_name)
        self._own = _Own(x.device, self.ws, self.y if out is None else None)

    def __call__(self, stream=None):
        r = C.byref(self.r) if self.r is not None else None
        if self.no_alloc:
            rc = lib().moe_layer_forward_static(C.byref(self.desc), C.byref(self.w), _p(self.y),
                                                r, _stream(stream))
            _check(rc, "moe_layer_forward_static")
        else:
            _launch(self.fn, self.fn_name, self.y.device, stream, C.byref(self.desc),
                    C.byref(self.w), _p(self.y), _p(self.ws), self.ws_bytes, r)
        self._own.used_on(stream)
        return self.y


class Backward:
    """One backward call prepared once (descriptor, weights, gradient outputs in fp32,
    workspace): ``__call__(dy)`` writes the gradients of sum(dy * y) into ``self.grads``.
    ``wgrad_bf16``: the expert weight gradients (dW_up, dW_down, dWs_up, dWs_down) in bf16."""

    def __init__(self, x, W_r, b, W_up, W_down, k, *, Ws_up=None, Ws_down=None, W_in=None,
                 W_out=None, wgrad_bf16=False):
        self.desc = make_desc(x, W_r, W_up, k, Ws_up, W_in)
        check_shapes(self.desc, x, W_r, b, W_up, W_down, Ws_up=Ws_up, Ws_down=Ws_down,
                     W_in=W_in, W_out=W_out)
        w = MoeWeights()
        w.x, w.W_r, w.b, w.W_up, w.W_down = _p(x), _p(W_r), _p(b), _p(W_up), _p(W_down)
        w.Ws_up, w.Ws_down, w.W_in, w.W_out = _p(Ws_up), _p(Ws_down), _p(W_in), _p(W_out)
        self.w = w
        self._keep = [x, W_r, b, W_up, W_down, Ws_up, Ws_down, W_in, W_out]
        f32 = dict(dtype=torch.float32, device=x.device)
        wg = dict(dtype=torch.bfloat16 if wgrad_bf16 else torch.float32, device=x.device)
        self.wgrad_bf16 = bool(wgrad_bf16)
        self.grads = {"dx": torch.empty(x.shape, **f32), "dW_r": torch.empty(W_r.shape, **f32),
                      "dW_up": torch.empty(W_up.shape, **wg),
                      "dW_down": torch.empty(W_down.shape, **wg)}
        if Ws_up is not None:
            self.grads["dWs_up"] = torch.empty(Ws_up.shape, **wg)
            self.grads["dWs_down"] = torch.empty(Ws_down.shape, **wg)
        if W_in is not None:
            self.grads["dW_in"] = torch.empty(W_in.shape, **f32)
            self.grads["dW_out"] = torch.empty(W_out.shape, **f32)
        g = MoeGrads()
        for name, _ in MoeGrads._fields_:
            setattr(g, name, _p(self.grads.get(name)))
        self.g = g
        n = C.c_size_t(0)
        _check(lib().moe_backward_workspace_size(C.byref(self.desc), C.byref(n)),
               "moe_backward_workspace_size")
        self.ws_bytes = n.value
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=x.device)
        self._own = _Own(x.device, self.ws, *self.grads.values())
        self._clip = None

    def forward_train(self, y=None, stream=None):
        """y of the layer (grouped path), keeping what the backward pass reads in the workspace:
        later calls with ``saved=True`` skip the recompute."""
        x = self._keep[0]
        own = y is None
        if own:
            y = torch.empty_like(x)
        _need(y, x.shape, "y", x.dtype, x.device)
        rc = lib().moe_layer_forward_train(C.byref(self.desc), C.byref(self.w), _p(y),
                                           _p(self.ws), self.ws_bytes, _stream(stream))
        _check(rc, "moe_layer_forward_train")
        self._own.used_on(stream)
        if own:
            _used_on(stream, y)
        return y

    def __call__(self, dy, stream=None, saved=False):
        x = self._keep[0]
        _need(dy, x.shape, "dy", x.dtype, x.device)
        d = MoeDesc.from_buffer_copy(self.desc)
        if saved:
            d.flags |= SAVED_IN_WORKSPACE
        if self.wgrad_bf16:
            d.flags |= WGRAD_BF16
        rc = lib().moe_layer_backward(C.byref(d), C.byref(self.w), _p(dy), C.byref(self.g),
                                      _p(self.ws), self.ws_bytes, _stream(stream))
        _check(rc, "moe_layer_backward")
        self._own.used_on(stream)
        return self.grads

    def clip(self, max_norm, stream=None):
        """Clips the weight gradients of the last call in place by their global norm, which is
        returned (GradClip over self.grads without dx, made on the first call: outside a capture; see
        there for calls on other streams)."""
        if self._clip is None:
            from .block import GradClip, _is_capturing
            if _is_capturing(_torch_stream(stream, self.ws.device)):
                raise ValueError("the first clip() makes its table: call it once before a capture")
            self._clip = GradClip({n: g for n, g in self.grads.items() if n != "dx"}, stream=stream)
        return self._clip(max_norm, stream)


def backward_from(dev: dict, k: int, **kw) -> Backward:
    """A Backward over a ``to_device`` dict (keywords as for Backward)."""
    return Backward(dev["x"], dev["W_r"], dev["b"], dev["W_up"], dev["W_down"], k,
                    Ws_up=dev.get("Ws_up"), Ws_down=dev.get("Ws_down"), W_in=dev.get("W_in"),
                    W_out=dev.get("W_out"), **kw)


def layer_forward(x, W_r, b, W_up, W_down, k, **kw):
    """y = MoE layer (or LatentMoE when W_in / W_out are given) of x; see moe.h."""
    return Layer(x, W_r, b, W_up, W_down, k, **kw)()


def route(b, k, *, logits=None, x=None, W_r=None, stream=None):
    """Router alone. Returns (idx, gates, logits)."""
    src = logits if logits is not None else x
    T = src.shape[0]
    E = b.shape[0]
    dev = src.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    lo = None
    H, dt = 0, MOE_F32
    if logits is None:
        H = x.shape[1]
        dt = _dtype_code(x)
        lo = torch.empty((T, E), dtype=torch.float32, device=dev)
    rc = lib().moe_route(_p(logits), _p(x), _p(W_r), _p(b), T, H, E, k, dt, _p(idx), _p(gates),
                         _p(lo), _stream(stream))
    _check(rc, "moe_route")
    _used_on(stream, idx, gates, lo)
    return idx, gates, (logits if logits is not None else lo)


def dispatch(idx, E, stream=None):
    """(counts, offsets, perm, pos) of idx [T, k]."""
    T, k = idx.shape
    dev = idx.device
    n = C.c_size_t(0)
    _check(lib().moe_dispatch_workspace_size(T, E, k, C.byref(n)), "moe_dispatch_workspace_size")
    ws = torch.empty(max(n.value, 1), dtype=torch.uint8, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    pos = torch.empty((T, k), dtype=torch.int32, device=dev)
    rc = lib().moe_dispatch(_p(idx), T, E, k, _p(counts), _p(offsets), _p(perm), _p(pos), _p(ws),
                            n.value, _stream(stream))
    _check(rc, "moe_dispatch")
    # the workspace is dropped here while the kernels may still run on `stream`
    _used_on(stream, ws, counts, offsets, perm, pos)
    return counts, offsets, perm, pos


def bias_update(counts, b, gamma: float, target=None, stream=None) -> None:
    """In place: b[e] += gamma * sign(target[e] - counts[e]) (target None: the mean load)."""
    E = b.numel()
    rc = lib().moe_bias_update(_p(counts), _p(target) if target is not None else None, E,
                               float(gamma), _p(b), _stream(stream))
    _check(rc, "moe_bias_update")


def _float_code(dtype: torch.dtype) -> int:
    if dtype is torch.bfloat16:
        return MOE_BF16
    if dtype is torch.float32:
        return MOE_F32
    raise ValueError(f"dtype {dtype} is neither float32 nor bfloat16")


def _launch(fn, name, device, stream, *args):
    """fn(*args, stream) on `device`, whatever device is current, on `stream` (None: the device's
    current stream; else a torch stream, or any object whose `cuda_stream` is the raw handle of a
    stream of that device). The raw handle is read directly: a torch.cuda.Stream object per call
    costs more host time than the launch."""
    if device.type != "cuda":
        raise ValueError(f"{name}: tensors are on {device}, expected a GPU")
    i = device.index
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(i)
    else:
        at = getattr(stream, "device", device)
        if at.index != i:
            raise ValueError(f"{name}: tensors are on {device}, the stream is on {at}")
        raw = stream.cuda_stream
    if torch._C._cuda_getDevice() == i:     # (tensors on a GPU: it is initialised)
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(i):
            rc = fn(*args, raw)
    if rc != MOE_OK:
        raise MoeError(rc, name)


def _mx_format(codes, scales, what):
    """(moe_dtype_t, element columns) of a block-scaled matrix, read off its shapes: one scale per
    32 columns, two MXFP4 elements or one MXFP8 element per byte."""
    cs, ss = codes.shape, scales.shape
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise ValueError(f"{what} and its scales must be uint8 tensors")
    # (two dimensions without slices: a call's time is host time where rows are few)
    same = cs[0] == ss[0] if len(cs) == len(ss) == 2 else cs[:-1] == ss[:-1]
    if not cs or len(cs) != len(ss) or not same or scales.device != codes.device:
        raise ValueError(f"{what} {tuple(cs)} on {codes.device} and its scales {tuple(ss)} on "
                         f"{scales.device} do not belong together")
    n, cols = cs[-1], MX_BLOCK * ss[-1]
    if cols and n * 2 == cols:
        return MOE_MXFP4, cols
    if cols and n == cols:
        return MOE_MXFP8, cols
    raise ValueError(f"{what}: {n} bytes and {ss[-1]} scales a row are neither MXFP4 nor MXFP8")


def mx_quantize(x, fmt="mxfp4", *, codes=None, scales=None, stream=None):
    """(codes, scales) of x [.., cols] (float32 or bfloat16, contiguous) in the OCP microscaling
    format ``fmt``, laid out as block-scaled expert weights are: codes [.., cols / 2] ("mxfp4")
    or [.., cols] ("mxfp8"), scales [.., cols / 32], both uint8. See moe_mx_quantize in moe.h."""
    if fmt not in _MX_FORMATS:
        raise ValueError(f"fmt {fmt!r} is not one of {sorted(_MX_FORMATS)}")
    dt, shape = _float_code(x.dtype), x.shape
    if not shape or shape[-1] % MX_BLOCK or not shape[-1]:
        raise ValueError(f"x {tuple(shape)}: the last dimension is not a multiple of {MX_BLOCK}")
    cols, lead, dev = shape[-1], shape[:-1], x.device
    cshape = lead + (cols // 2 if fmt == "mxfp4" else cols,)
    sshape = lead + (cols // MX_BLOCK,)
    made = []
    if codes is None:
        codes = x.new_empty(cshape, dtype=torch.uint8)
        made.append(codes)
    else:
        _need(codes, cshape, "codes", torch.uint8, dev)
    if scales is None:
        scales = x.new_empty(sshape, dtype=torch.uint8)
        made.append(scales)
    else:
        _need(scales, sshape, "scales", torch.uint8, dev)
    _launch(lib().moe_mx_quantize, "moe_mx_quantize", dev, stream, _p(x), dt, x.numel() // cols,
            cols, _MX_FORMATS[fmt], _p(codes), _p(scales))
    _used_on(stream, *made)
    return codes, scales


def mx_dequantize(codes, scales, *, dtype=torch.float32, out=None, stream=None):
    """The values [.., cols] (float32 or bfloat16) that MXFP4 / MXFP8 codes and scales stand for;
    the format is read off the shapes. See moe_mx_dequantize in moe.h."""
    fmt, cols = _mx_format(codes, scales, "codes")
    dt = _float_code(dtype)
    shape, dev = codes.shape[:-1] + (cols,), codes.device
    made = out is None
    if made:
        out = codes.new_empty(shape, dtype=dtype)
    else:
        _need(out, shape, "out", dtype, dev)
    _launch(lib().moe_mx_dequantize, "moe_mx_dequantize", dev, stream, _p(codes), _p(scales), fmt,
            out.numel() // cols, cols, _p(out), dt)
    if made:
        _used_on(stream, out)
    return out


def mx_gemm(a, a_scales, w, w_scales, *, out_dtype=torch.bfloat16, out=None, stream=None):
    """C [M, N] = A [M, K] W [N, K]^T of two block-scaled matrices (each MXFP4 or MXFP8, read off
    the shapes), fp32 accumulation, as bfloat16, or float32 for two MXFP4 operands. See
    moe_mx_gemm in moe.h."""
    fa, K = _mx_format(a, a_scales, "a")
    fw, kw = _mx_format(w, w_scales, "w")
    dev = a.device
    if a.dim() != 2 or w.dim() != 2 or K != kw or dev != w.device:
        raise ValueError(f"a {tuple(a.shape)} ({K} columns, {dev}) and w {tuple(w.shape)} "
                         f"({kw} columns, {w.device}) do not multiply")
    dt, M, N = _float_code(out_dtype), a.shape[0], w.shape[0]
    made = out is None
    if made:
        out = a.new_empty((M, N), dtype=out_dtype)
    else:
        _need(out, (M, N), "out", out_dtype, dev)
    _launch(lib().moe_mx_gemm, "moe_mx_gemm", dev, stream, _p(a), _p(a_scales), fa, _p(w),
            _p(w_scales), fw, M, N, K, _p(out), dt)
    if made:
        _used_on(stream, out)
    return out


def trace_enable(capacity: int, prefix: str = "") -> None:
    """Record HIP events around every launch whose trace name starts with `prefix`."""
    _check(lib().moe_trace_enable(capacity, prefix.encode()), "moe_trace_enable")


def trace_disable() -> None:
    _check(lib().moe_trace_enable(0, None), "moe_trace_enable")


def trace_reset() -> None:
    lib().moe_trace_reset()


def trace_records() -> list:
    """[(name, ms)] of the recorded launches (synchronise the stream first)."""
    out = []
    for i in range(lib().moe_trace_count()):
        name, ms = C.c_char_p(), C.c_float()
        _check(lib().moe_trace_read(i, C.byref(name), C.byref(ms)), "moe_trace_read")
        out.append((name.value.decode(), ms.value))
    return out


def to_device(inp: dict, device="cuda") -> dict:
    """numpy arrays of a ``moe_inputs.make_layer`` dict -> torch tensors on ``device``
    (uint16 bf16 bit patterns become torch.bfloat16; e4m3, E2M1 and E8M0 codes stay uint8)."""
    import numpy as np
    out = {}
    for name, a in inp.items():
        if isinstance(a, np.ndarray):
            t = torch.from_numpy(a.view(np.int16)).view(torch.bfloat16) if a.dtype == np.uint16 \
                else torch.from_numpy(a)
            out[name] = t.to(device)
    return out


def layer_from(dev: dict, k: int, **kw) -> Layer:
    """A Layer over a ``to_device`` dict."""
    return Layer(dev["x"], dev["W_r"], dev["b"], dev["W_up"], dev["W_down"], k,
                 s_up=dev.get("s_up"), s_down=dev.get("s_down"), Ws_up=dev.get("Ws_up"),
                 Ws_down=dev.get("Ws_down"), W_in=dev.get("W_in"), W_out=dev.get("W_out"), **kw)
