"""The operators around the layer: token rows into expert order and back, the norms before and
after a block with its gate and residual, and gradient clipping, each with its gradients where it
has any. Argument checks and marshalling only, as in binding.py; see include/moe.h for what each
computes."""
from __future__ import annotations

import ctypes as C
import functools
from array import array

import torch

from .binding import (MOE_BF16, Layer, MoeClip, MoeClipTensor, MoeError, _check, _float_code,
                      _launch, _need, _Own, _p, _raw, _torch_stream, _used_on, lib)

BLOCK_NORM, GATE_TOKEN, GATE_ELEMENT, GATE_SIGMOID = 1, 2, 4, 8
_F32, _I32 = torch.float32, torch.int32

# The time of a call on few rows is host time: every tensor is checked and turned into its address
# in one step, and new outputs, which need no check, are made by the cheapest call.


def _ptr(t, shape, what, dtype, device):
    """Address of a contiguous tensor that must have this shape, type and device."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _need(t, shape, what, dtype, device)
    return _p(t)


def _is_capturing(stream):
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _two(t, what):
    s = t.shape
    if len(s) != 2 or max(s) > 0x7FFFFFFF:   # the library takes 32-bit sizes
        raise ValueError(f"{what} has shape {tuple(s)}, expected two dimensions below 2^31")
    return s


# ------------------------------------------------------------------------------- token rows

@functools.lru_cache(maxsize=256)
def _sort_workspace(T, E, k):
    n = C.c_size_t(0)
    _check(lib().moe_sort_tokens_workspace_size(T, E, k, C.byref(n)),
           "moe_sort_tokens_workspace_size")
    return n.value


def _pairs(pos, weights, T, dev, what="pos"):
    """(slots, address of pos, address of weights or None)."""
    k = _two(pos, what)[1]
    shape = pos.shape
    return (k, _ptr(pos, (T, k), what, _I32, dev),
            None if weights is None else _ptr(weights, shape, "weights", _F32, dev))


def sort_tokens(x, idx, E, *, weights=None, out=None, stream=None):
    """(rows, offsets, pos): the rows of x [T, D] (float32 or bfloat16) in expert order, once per
    kept pair of idx [T, k] (int32), rows[pos[t, j]] = weights[t, j] * x[t] (weights float32 or
    None for 1). Expert e's rows are rows[offsets[e]:offsets[e + 1]], tokens ascending; pos is -1
    where a pair is dropped (expert outside [0, E), or repeated in its token). rows has T * k rows;
    those behind offsets[E] are not written. See moe_sort_tokens in moe.h."""
    T, D = _two(x, "x")
    dev, dtype = x.device, x.dtype
    dt = _float_code(dtype)
    k, ip, wp = _pairs(idx, weights, T, dev, "idx")
    if not -1 < E < 0x80000000:              # as _two
        raise ValueError(f"E is {E}, expected the number of experts")
    n = _sort_workspace(T, E, k)
    if out is None:
        rows = x.new_empty((T * k, D))
        rp = rows.data_ptr()
    else:
        rows, rp = out, _ptr(out, (T * k, D), "out", dtype, dev)
    offsets = idx.new_empty(E + 1)
    pos = torch.empty_like(idx)
    ws = x.new_empty(n, dtype=torch.uint8) if n else None
    _launch(lib().moe_sort_tokens, "moe_sort_tokens", dev, stream, _p(x), dt, ip, wp, T, D, E, k, rp,
            offsets.data_ptr(), pos.data_ptr(), ws.data_ptr() if n else None, n)
    if stream is not None:
        _used_on(stream, offsets, pos, ws, rows if out is None else None)
    return rows, offsets, pos


def sort_tokens_backward(drows, pos, *, x=None, weights=None, out_dtype=None, stream=None):
    """(dx, dweights) of sort_tokens given drows [n, D] and its pos [T, k]: dx [T, D] of out_dtype
    (default: that of drows), dweights [T, k] float32 where x (the sorted rows' source, of drows'
    type) is given, else None. See moe_sort_tokens_backward in moe.h."""
    n, D = _two(drows, "drows")
    dev, dtype, T = drows.device, drows.dtype, pos.shape[0]
    dt = odt = _float_code(dtype)
    k, pp, wp = _pairs(pos, weights, T, dev)
    if out_dtype is None:
        dx = drows.new_empty((T, D))
    else:
        odt = _float_code(out_dtype)
        dx = drows.new_empty((T, D), dtype=out_dtype)
    dw = xp = None
    if x is not None:
        xp = _ptr(x, (T, D), "x", dtype, dev)
        dw = torch.empty_like(pos, dtype=_F32)
    _launch(lib().moe_sort_tokens_backward, "moe_sort_tokens_backward", dev, stream, _p(drows), xp,
            dt, pp, wp, T, D, k, n, dx.data_ptr(), odt, None if dw is None else dw.data_ptr())
    if stream is not None:
        _used_on(stream, dx, dw)
    return dx, dw


def unsort_tokens(rows, pos, *, weights=None, add=None, out_dtype=None, out=None, stream=None):
    """y [T, D] of rows [n, D] in expert order: y[t] = add[t] + sum_j weights[t, j] *
    rows[pos[t, j]] (dropped pairs add nothing; weights None: 1). y has out_dtype (default: that
    of out, of add, or of rows), add too; out may be add. See moe_unsort_tokens in moe.h."""
    n, D = _two(rows, "rows")
    dev, T = rows.device, pos.shape[0]
    dt = _float_code(rows.dtype)
    k, pp, wp = _pairs(pos, weights, T, dev)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else add.dtype if add is not None else rows.dtype
    odt = _float_code(out_dtype)
    ap = None if add is None else _ptr(add, (T, D), "add", out_dtype, dev)
    if out is None:
        y = rows.new_empty((T, D), dtype=out_dtype)
        yp = y.data_ptr()
    else:
        y, yp = out, _ptr(out, (T, D), "out", out_dtype, dev)
    _launch(lib().moe_unsort_tokens, "moe_unsort_tokens", dev, stream, _p(rows), dt, pp, wp, ap, T,
            D, k, n, yp, odt)
    if stream is not None and out is None:
        _used_on(stream, y)
    return y


def unsort_tokens_backward(dy, pos, *, rows=None, weights=None, n_rows=None, out=None, stream=None):
    """(drows, dweights) of unsort_tokens given dy [T, D]: drows[pos[t, j]] = weights[t, j] * dy[t],
    and dweights [T, k] float32 where the forward's rows are given, else None. drows is as large and
    of the same type as out or rows (out may be rows), else [n_rows or T * k, D] of dy's type; rows
    that no pair names are not written. See moe_unsort_tokens_backward in moe.h."""
    T, D = _two(dy, "dy")
    dev = dy.device
    dyt = _float_code(dy.dtype)
    k, pp, wp = _pairs(pos, weights, T, dev)
    if rows is not None:
        like, n = rows, _two(rows, "rows")[0]
    elif out is not None:
        like, n = out, _two(out, "out")[0]
    else:
        like, n = None, T * k
    if n_rows is not None:
        n = n_rows
    if not 0 <= n <= 0x7FFFFFFF:             # as _two
        raise ValueError(f"n_rows is {n}, expected 0 to 2^31 - 1")
    dtype = like.dtype if like is not None else dy.dtype
    dt = _float_code(dtype)
    rp = dw = None
    if rows is not None:
        rp = _ptr(rows, (n, D), "rows", dtype, dev)
        dw = torch.empty_like(pos, dtype=_F32)
    elif dt != dyt:
        raise ValueError(f"out has dtype {dtype}: without rows it is dy's, {dy.dtype}")
    if out is None:
        drows = dy.new_empty((n, D), dtype=dtype)
        op = drows.data_ptr()
    else:
        drows, op = out, _ptr(out, (n, D), "out", dtype, dev)
    _launch(lib().moe_unsort_tokens_backward, "moe_unsort_tokens_backward", dev, stream, _p(dy), dyt,
            rp, dt, pp, wp, T, D, k, n, op, None if dw is None else dw.data_ptr())
    if stream is not None:
        _used_on(stream, dw, drows if out is None else None)
    return drows, dw


# --------------------------------------------------------------------------- the block's norms

def _weights(w, w_next, H, dev, dt):
    """(moe_dtype_t of the norms' weights, their addresses): both of one type."""
    wp = nextp = None
    if w is not None:
        dt = _float_code(w.dtype)
        wp = _ptr(w, (H,), "w", w.dtype, dev)
    if w_next is not None:
        if w is not None and w_next.dtype is not w.dtype:
            raise ValueError(f"w_next has dtype {w_next.dtype}, w {w.dtype}")
        dt = _float_code(w_next.dtype)
        nextp = _ptr(w_next, (H,), "w_next", w_next.dtype, dev)
    return dt, wp, nextp


def _gate(gate, gate_act, shape, dtype, dev):
    """(flags, address) of a gate per element or per token."""
    if gate_act not in ("sigmoid", "none"):
        raise ValueError(f"gate_act {gate_act!r} is neither 'sigmoid' nor 'none'")
    if gate is None:
        return 0, None
    sigmoid = GATE_SIGMOID if gate_act == "sigmoid" else 0
    if gate.shape == shape:
        return GATE_ELEMENT | sigmoid, _ptr(gate, shape, "gate", dtype, dev)
    if gate.shape != shape[:1] and gate.shape != (shape[0], 1):
        raise ValueError(f"gate has shape {tuple(gate.shape)}, expected {tuple(shape)}, "
                         f"({shape[0]}, 1) or ({shape[0]},)")
    return GATE_TOKEN | sigmoid, _ptr(gate, gate.shape, "gate", _F32, dev)


@functools.lru_cache(maxsize=256)
def _block_workspace(T, H):
    n = C.c_size_t(0)
    _check(lib().moe_block_backward_workspace_size(T, H, C.byref(n)),
           "moe_block_backward_workspace_size")
    return n.value


def block_norm(x, w=None, *, eps=1e-5, out=None, stream=None):
    """h = x / sqrt(mean(x^2) + eps) * w per row of x [T, H] (float32 or bfloat16); w [H] float32
    or bfloat16, None for 1. out may be x. See moe_block_norm in moe.h."""
    T, H = _two(x, "x")
    dev, dtype = x.device, x.dtype
    dt = _float_code(dtype)
    wdt, wp, _ = _weights(w, None, H, dev, dt)
    xp = _p(x)
    if out is None:
        h = torch.empty_like(x)
        hp = h.data_ptr()
    else:
        h, hp = out, _ptr(out, x.shape, "out", dtype, dev)
    _launch(lib().moe_block_norm, "moe_block_norm", dev, stream, xp, wp, hp, T, H, dt, wdt, eps)
    if stream is not None and out is None:
        _used_on(stream, h)
    return h


def block_norm_backward(dh, x, w=None, *, dres=None, eps=1e-5, out=None, stream=None):
    """(dx, dw) of block_norm given dh [T, H] (x's type, or float32): dx = dres + the norm's
    gradient, of x's type (out may be dres); dw [H] float32, None without w. See
    moe_block_norm_backward in moe.h."""
    T, H = shape = _two(x, "x")
    dev, dtype = x.device, x.dtype
    dt = _float_code(dtype)
    xp = _p(x)
    dhp = _ptr(dh, shape, "dh", dh.dtype, dev)
    wdt, wp, _ = _weights(w, None, H, dev, dt)
    rp = None if dres is None else _ptr(dres, shape, "dres", dtype, dev)
    if out is None:
        dx = torch.empty_like(x)
        dxp = dx.data_ptr()
    else:
        dx, dxp = out, _ptr(out, shape, "out", dtype, dev)
    dw = ws = dwp = wsp = None
    n = 0
    if w is not None:
        dw = torch.empty_like(w, dtype=_F32)
        n = _block_workspace(T, H)
        ws = x.new_empty(n, dtype=torch.uint8)
        dwp, wsp = dw.data_ptr(), ws.data_ptr()
    _launch(lib().moe_block_norm_backward, "moe_block_norm_backward", dev, stream, dhp,
            _float_code(dh.dtype), xp, wp, rp, dxp, dwp, T, H, dt, wdt, eps, wsp, n)
    if stream is not None:
        _used_on(stream, ws, dw, dx if out is None else None)
    return dx, dw


def block_residual(x, f, *, w=None, norm=True, gate=None, gate_act="sigmoid", scale=1.0,
                   next_norm=False, w_next=None, eps=1e-5, out=None, h_out=None, stream=None):
    """(y, h): y = x + scale * a * z for the block's output f (x, f [T, H], float32 or bfloat16),
    z the norm of f times w (norm=False: f * w), a the gate or its sigmoid: per token (float32
    [T] or [T, 1]), per element ([T, H], x's type), or None for 1. With next_norm (or h_out, or
    w_next) h is the next block's norm of y, else None. out may be x or f. See moe_block_residual
    in moe.h."""
    T, H = shape = _two(x, "x")
    dev, dtype = x.device, x.dtype
    dt = _float_code(dtype)
    xp = _p(x)
    fp = _ptr(f, shape, "f", dtype, dev)
    wdt, wp, nextp = _weights(w, w_next, H, dev, dt)
    flags, gp = _gate(gate, gate_act, shape, dtype, dev)
    if norm:
        flags |= BLOCK_NORM
    if out is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        y, yp = out, _ptr(out, shape, "out", dtype, dev)
    h = hp = None
    if h_out is not None:
        h, hp = h_out, _ptr(h_out, shape, "h_out", dtype, dev)
    elif next_norm or w_next is not None:
        h = torch.empty_like(x)
        hp = h.data_ptr()
    _launch(lib().moe_block_residual, "moe_block_residual", dev, stream, xp, fp, wp, gp, nextp, yp, hp,
            T, H, dt, wdt, flags, scale, eps)
    if stream is not None:
        _used_on(stream, y if out is None else None, h if h_out is None else None)
    return y, h


def block_residual_backward(dy, f, *, w=None, norm=True, gate=None, gate_act="sigmoid", scale=1.0,
                            y=None, dh=None, w_next=None, eps=1e-5, stream=None):
    """Gradients of block_residual as a dict: dx, df, and dw, dgate, dw_next where w, gate and
    w_next are given. dy [T, H] (f's type, or None where only h was used) reaches y; dh (f's type or
    float32), with the forward's y, reaches h. dw and dw_next are float32. See
    moe_block_residual_backward in moe.h."""
    T, H = shape = _two(f, "f")
    dev, dtype = f.device, f.dtype
    dt = dh_dt = _float_code(dtype)
    fp = _p(f)
    if dy is None and dh is None:
        raise ValueError("dy or dh is required")
    dyp = None if dy is None else _ptr(dy, shape, "dy", dtype, dev)
    yp = dhp = None
    if dh is not None:
        dh_dt = _float_code(dh.dtype)
        dhp = _ptr(dh, shape, "dh", dh.dtype, dev)
        if y is None:
            raise ValueError("y is required with dh")
        yp = _ptr(y, shape, "y", dtype, dev)
    elif w_next is not None:
        raise ValueError("w_next has no gradient without dh")
    wdt, wp, nextp = _weights(w, w_next, H, dev, dt)
    flags, gp = _gate(gate, gate_act, shape, dtype, dev)
    if norm:
        flags |= BLOCK_NORM
    dx, df = torch.empty_like(f), torch.empty_like(f)
    out = {"dx": dx, "df": df}
    dgp = dwp = dnp = ws = wsp = None
    n = 0
    if gate is not None:
        out["dgate"] = dgate = torch.empty_like(gate)
        dgp = dgate.data_ptr()
    if w is not None:
        out["dw"] = dw = torch.empty_like(w, dtype=_F32)
        dwp = dw.data_ptr()
    if w_next is not None:
        out["dw_next"] = dw = torch.empty_like(w_next, dtype=_F32)
        dnp = dw.data_ptr()
    if dwp is not None or dnp is not None:
        n = _block_workspace(T, H)
        ws = f.new_empty(n, dtype=torch.uint8)
        wsp = ws.data_ptr()
    _launch(lib().moe_block_residual_backward, "moe_block_residual_backward", dev, stream, dyp, fp,
            wp, gp, yp, dhp, dh_dt, nextp, dx.data_ptr(), df.data_ptr(), dwp, dgp, dnp, T, H, dt, wdt,
            flags, scale, eps, wsp, n)
    if stream is not None:
        _used_on(stream, ws, *out.values())
    return out


# ----------------------------------------------------------------------------- gradient clipping

class GradClip:
    """Clipping of a fixed set of gradients (a list, or a dict's values; float32 and bfloat16,
    contiguous, one GPU) by their global norm, prepared once: ``__call__(max_norm)`` writes
    grad * min(1, max_norm / (norm + 1e-6)) into the gradients, or into ``out`` (as many tensors of
    the same shapes and types), and returns the norm (a float32 tensor that the next call
    overwrites; ``coef`` is beside it). A norm that is not finite leaves the values as they are.
    A call on another stream than the constructor's waits for the constructor's work, unless that
    stream is captured: a graph is then replayed after it, and the object kept as long as the graph.
    Calls of one GradClip must not overlap; one that was made while a stream was captured serves
    that capture alone (its table is written by the graph). See moe_clip_plan in moe.h."""

    _one_use = False

    def __init__(self, grads, *, out=None, stream=None):
        grads = list(grads.values()) if isinstance(grads, dict) else list(grads)
        outs = grads if out is None else list(out.values()) if isinstance(out, dict) else list(out)
        if not grads:
            raise ValueError("grads is empty")
        if len(outs) != len(grads):
            raise ValueError(f"{len(outs)} outputs for {len(grads)} gradients")
        dev = grads[0].device
        flat, spans = array("q"), []     # MoeClipTensor: three 64-bit words and the type, padded
        for g, o in zip(grads, outs):
            n, dtype = g.numel(), g.dtype
            dt = _float_code(dtype)
            if g.device != dev:
                raise ValueError(f"a gradient is on {g.device}, another on {dev}")
            gp = op = _p(g)
            if o is not g:
                op = _ptr(o, g.shape, "an output", dtype, dev)
            flat.extend((gp, op, n, dt))
            if n:
                size = n * (2 if dt == MOE_BF16 else 4)
                if op != gp:
                    spans.append((gp, gp + size, False))
                spans.append((op, op + size, True))
        _check_apart(spans)
        table = (MoeClipTensor * len(grads)).from_buffer(flat)
        n = C.c_size_t(0)
        _check(lib().moe_clip_plan_size(table, len(grads), C.byref(n)), "moe_clip_plan_size")
        self._keep = (grads, outs)
        self.device = dev
        self.plan = grads[0].new_empty(n.value, dtype=torch.uint8)
        self.clip = MoeClip()
        _launch(lib().moe_clip_plan, "moe_clip_plan", dev, stream, table, len(grads), _p(self.plan),
                n.value, C.byref(self.clip))
        self._both = both = grads[0].new_empty(2, dtype=torch.float32)
        if stream is not None:
            _used_on(stream, self.plan, both)
        self.norm, self.coef = both[0], both[1]
        self._args = (C.byref(self.clip), both.data_ptr())
        self._made_on, self._ready = _raw(stream, dev), None
        if not (self.clip.capture or self._one_use):
            self._ready = torch.cuda.Event()
            self._ready.record(_torch_stream(stream, dev))

    def __call__(self, max_norm, stream=None):
        clip, norm = self._args
        other = _raw(stream, self.device) != self._made_on
        if other:
            stream = _torch_stream(stream, self.device)
            if self._ready is not None and not _is_capturing(stream):
                stream.wait_event(self._ready)
        try:
            _launch(lib().moe_clip_grads, "moe_clip_grads", self.device, stream, clip, max_norm, norm)
        except MoeError as e:
            if self.clip.capture and max_norm >= 0:
                raise ValueError("this GradClip was made while a stream was captured and serves that "
                                 "capture alone") from e
            raise
        if other:      # the plan holds addresses that the kernels write through
            _used_on(stream, self.plan, self._both)
        return self.norm


def _check_apart(spans):
    """spans: (begin, end, written) of every gradient and output. What is written lies apart from
    everything else."""
    end = written = 0    # ends of what is read or written, and of what is written, so far
    for lo, hi, writes in sorted(spans):
        if lo < written or (writes and lo < end):
            raise ValueError("an output overlaps another output or another gradient")
        end = max(end, hi)
        if writes:
            written = max(written, hi)


class _OneUse(GradClip):
    """Called on its constructor's stream alone, which needs no event."""
    _one_use = True


def clip_grad_norm(grads, max_norm, *, out=None, stream=None):
    """GradClip for one use: clips grads (or into out) and returns their norm. The table is made anew
    in every call, about 1.4 us of host time a tensor: where the tensors stay, keep a GradClip."""
    clip = _OneUse(grads, out=out, stream=stream)
    norm = clip(max_norm, stream)
    if stream is not None:
        _used_on(stream, *clip._keep[0], *clip._keep[1])
    return norm


# -------------------------------------------------------------------------------------- the block

class Block:
    """A layer in its residual block, prepared once as Layer is:
        h = norm(x) * w_in;  f = layer(h);  y = x + scale * a * norm(f) * w_out
    with the gate a as in block_residual (norm_out=False: f * w_out alone). ``__call__`` returns y;
    with next_norm (or w_next) ``h_next`` holds the next block's norm of y. h: the rows as a block
    before left them (its h_next), instead of norm(x) * w_in. Other keywords go to Layer."""

    def __init__(self, x, W_r, b, W_up, W_down, k, *, w_in=None, w_out=None, norm_out=True,
                 gate=None, gate_act="sigmoid", scale=1.0, next_norm=False, w_next=None, eps=1e-5,
                 h=None, **layer):
        if h is not None and w_in is not None:
            raise ValueError("w_in and h exclude each other")
        self.x, self.w_in, self.eps, self.own_norm = x, w_in, eps, h is None
        self.h = torch.empty_like(x) if h is None else h
        self.layer = Layer(self.h, W_r, b, W_up, W_down, k, **layer)
        self.y = torch.empty_like(x)
        self.h_next = torch.empty_like(x) if next_norm or w_next is not None else None
        self.after = dict(w=w_out, norm=norm_out, gate=gate, gate_act=gate_act, scale=scale,
                          w_next=w_next, eps=eps, out=self.y, h_out=self.h_next)
        self._own = _Own(x.device, self.h if h is None else None, self.y, self.h_next)

    def __call__(self, stream=None):
        if self.own_norm:
            block_norm(self.x, self.w_in, eps=self.eps, out=self.h, stream=stream)
        f = self.layer(stream)
        block_residual(self.x, f, stream=stream, **self.after)
        self._own.used_on(stream)
        return self.y
