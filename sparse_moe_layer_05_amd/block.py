"""The operators around the layer: token rows into expert order and back, the norms before and
after a block with its gate and residual, and gradient clipping, each with its gradients where it
has any. Argument checks and marshalling only, as in binding.py; see include/moe.h for what each
computes."""
from __future__ import annotations

import ctypes as C
import functools

import torch

from .binding import (MoeClip, MoeClipTensor, _check, _float_code, _launch, _need, _p, _used_on, lib)

BLOCK_NORM, GATE_TOKEN, GATE_ELEMENT, GATE_SIGMOID = 1, 2, 4, 8


def _rows_of(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected two dimensions")
    return t.shape


def _out(given, like, shape, dtype, what, made):
    """The output tensor: the caller's, checked, or a new one, which is noted in `made`."""
    if given is None:
        given = like.new_empty(shape, dtype=dtype)
        made.append(given)
    else:
        _need(given, shape, what, dtype, like.device)
    return given


# ------------------------------------------------------------------------------- token rows

@functools.lru_cache(maxsize=256)
def _sort_workspace(T, E, k):
    n = C.c_size_t(0)
    _check(lib().moe_sort_tokens_workspace_size(T, E, k, C.byref(n)),
           "moe_sort_tokens_workspace_size")
    return n.value


def _check_pairs(pos, weights, T, dev, what="pos"):
    if pos.dim() != 2:
        raise ValueError(f"{what} has shape {tuple(pos.shape)}, expected [tokens, slots]")
    _need(pos, (T, pos.shape[1]), what, torch.int32, dev)
    if weights is not None:
        _need(weights, pos.shape, "weights", torch.float32, dev)
    return pos.shape[1]


def sort_tokens(x, idx, E, *, weights=None, out=None, stream=None):
    """(rows, offsets, pos): the rows of x [T, D] (float32 or bfloat16) in expert order, once per
    kept pair of idx [T, k] (int32), rows[pos[t, j]] = weights[t, j] * x[t] (weights float32 or
    None for 1). Expert e's rows are rows[offsets[e]:offsets[e + 1]], tokens ascending; pos is -1
    where a pair is dropped (expert outside [0, E), or repeated in its token). rows has T * k rows;
    those behind offsets[E] are not written. See moe_sort_tokens in moe.h."""
    T, D = _rows_of(x, "x")
    dev, made = x.device, []
    k = _check_pairs(idx, weights, T, dev, "idx")
    dt = _float_code(x.dtype)
    rows = _out(out, x, (T * k, D), x.dtype, "out", made)
    offsets = idx.new_empty(E + 1)
    pos = idx.new_empty((T, k))
    n = _sort_workspace(T, E, k)
    ws = x.new_empty(n, dtype=torch.uint8) if n else None
    _launch(lib().moe_sort_tokens, "moe_sort_tokens", dev, stream, _p(x), dt, _p(idx), _p(weights),
            T, D, E, k, _p(rows), _p(offsets), _p(pos), _p(ws), n)
    _used_on(stream, offsets, pos, ws, *made)
    return rows, offsets, pos


def sort_tokens_backward(drows, pos, *, x=None, weights=None, out_dtype=None, stream=None):
    """(dx, dweights) of sort_tokens given drows [n, D] and its pos [T, k]: dx [T, D] of out_dtype
    (default: that of drows), dweights [T, k] float32 where x (the sorted rows' source, of drows'
    type) is given, else None. See moe_sort_tokens_backward in moe.h."""
    n, D = _rows_of(drows, "drows")
    dev, T, made = drows.device, pos.shape[0], []
    k = _check_pairs(pos, weights, T, dev)
    dt = _float_code(drows.dtype)
    odt = _float_code(out_dtype or drows.dtype)
    if x is not None:
        _need(x, (T, D), "x", drows.dtype, dev)
    dx = _out(None, drows, (T, D), out_dtype or drows.dtype, "dx", made)
    dw = None if x is None else _out(None, drows, (T, k), torch.float32, "dweights", made)
    _launch(lib().moe_sort_tokens_backward, "moe_sort_tokens_backward", dev, stream, _p(drows),
            _p(x), dt, _p(pos), _p(weights), T, D, k, n, _p(dx), odt, _p(dw))
    _used_on(stream, *made)
    return dx, dw


def unsort_tokens(rows, pos, *, weights=None, add=None, out_dtype=None, out=None, stream=None):
    """y [T, D] of rows [n, D] in expert order: y[t] = add[t] + sum_j weights[t, j] *
    rows[pos[t, j]] (dropped pairs add nothing; weights None: 1). y has out_dtype (default: that
    of out, of add, or of rows), add too; out may be add. See moe_unsort_tokens in moe.h."""
    n, D = _rows_of(rows, "rows")
    dev, T, made = rows.device, pos.shape[0], []
    k = _check_pairs(pos, weights, T, dev)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else add.dtype if add is not None else rows.dtype
    dt, odt = _float_code(rows.dtype), _float_code(out_dtype)
    if add is not None:
        _need(add, (T, D), "add", out_dtype, dev)
    y = _out(out, rows, (T, D), out_dtype, "out", made)
    _launch(lib().moe_unsort_tokens, "moe_unsort_tokens", dev, stream, _p(rows), dt, _p(pos),
            _p(weights), _p(add), T, D, k, n, _p(y), odt)
    _used_on(stream, *made)
    return y


def unsort_tokens_backward(dy, pos, *, rows=None, weights=None, n_rows=None, out=None, stream=None):
    """(drows, dweights) of unsort_tokens given dy [T, D]: drows[pos[t, j]] = weights[t, j] * dy[t],
    and dweights [T, k] float32 where the forward's rows are given, else None. drows is as large and
    of the same type as out or rows (out may be rows), else [n_rows or T * k, D] of dy's type; rows
    that no pair names are not written. See moe_unsort_tokens_backward in moe.h."""
    T, D = _rows_of(dy, "dy")
    dev, made = dy.device, []
    k = _check_pairs(pos, weights, T, dev)
    like = rows if rows is not None else out
    n = n_rows if n_rows is not None else like.shape[0] if like is not None else T * k
    dtype = like.dtype if like is not None else dy.dtype
    if rows is not None:
        _need(rows, (n, D), "rows", dtype, dev)
    elif dtype != dy.dtype:
        raise ValueError(f"out has dtype {dtype}: without rows it is dy's, {dy.dtype}")
    drows = _out(out, dy, (n, D), dtype, "out", made)
    dw = None if rows is None else _out(None, dy, (T, k), torch.float32, "dweights", made)
    _launch(lib().moe_unsort_tokens_backward, "moe_unsort_tokens_backward", dev, stream, _p(dy),
            _float_code(dy.dtype), _p(rows), _float_code(dtype), _p(pos), _p(weights), T, D, k, n,
            _p(drows), _p(dw))
    _used_on(stream, *made)
    return drows, dw


# --------------------------------------------------------------------------- the block's norms

def _weight_code(H, dev, dtype, **ws):
    """moe_dtype_t of the norms' weights: all of one type, float32 or bfloat16."""
    for name, w in ws.items():
        if w is not None:
            _need(w, (H,), name, None, dev)
            dtype = w.dtype
    for name, w in ws.items():
        if w is not None and w.dtype != dtype:
            raise ValueError(f"{name} has dtype {w.dtype}, the other weight {dtype}")
    return _float_code(dtype)


def _gate_flags(gate, gate_act, shape, dtype, dev):
    if gate_act not in ("sigmoid", "none"):
        raise ValueError(f"gate_act {gate_act!r} is neither 'sigmoid' nor 'none'")
    if gate is None:
        return 0
    if gate.shape == shape and gate.dim() == 2 and not (shape[1] == 1):
        _need(gate, shape, "gate", dtype, dev)
        kind = GATE_ELEMENT
    else:
        if gate.shape != shape[:1] and gate.shape != (shape[0], 1):
            raise ValueError(f"gate has shape {tuple(gate.shape)}, expected {tuple(shape)}, "
                             f"({shape[0]}, 1) or ({shape[0]},)")
        _need(gate, gate.shape, "gate", torch.float32, dev)
        kind = GATE_TOKEN
    return kind | (GATE_SIGMOID if gate_act == "sigmoid" else 0)


@functools.lru_cache(maxsize=256)
def _block_workspace(T, H):
    n = C.c_size_t(0)
    _check(lib().moe_block_backward_workspace_size(T, H, C.byref(n)),
           "moe_block_backward_workspace_size")
    return n.value


def block_norm(x, w=None, *, eps=1e-5, out=None, stream=None):
    """h = x / sqrt(mean(x^2) + eps) * w per row of x [T, H] (float32 or bfloat16); w [H] float32
    or bfloat16, None for 1. out may be x. See moe_block_norm in moe.h."""
    T, H = _rows_of(x, "x")
    dev, made = x.device, []
    dt = _float_code(x.dtype)
    wdt = _weight_code(H, dev, x.dtype, w=w)
    h = _out(out, x, (T, H), x.dtype, "out", made)
    _launch(lib().moe_block_norm, "moe_block_norm", dev, stream, _p(x), _p(w), _p(h), T, H, dt, wdt,
            eps)
    _used_on(stream, *made)
    return h


def block_norm_backward(dh, x, w=None, *, dres=None, eps=1e-5, out=None, stream=None):
    """(dx, dw) of block_norm given dh [T, H] (x's type, or float32): dx = dres + the norm's
    gradient, of x's type (out may be dres); dw [H] float32, None without w. See
    moe_block_norm_backward in moe.h."""
    T, H = _rows_of(x, "x")
    dev, made = x.device, []
    dt = _float_code(x.dtype)
    _need(dh, (T, H), "dh", None, dev)
    wdt = _weight_code(H, dev, x.dtype, w=w)
    if dres is not None:
        _need(dres, (T, H), "dres", x.dtype, dev)
    dx = _out(out, x, (T, H), x.dtype, "out", made)
    dw = ws = None
    n = 0
    if w is not None:
        dw = _out(None, x, (H,), torch.float32, "dw", made)
        n = _block_workspace(T, H)
        ws = x.new_empty(n, dtype=torch.uint8)
    _launch(lib().moe_block_norm_backward, "moe_block_norm_backward", dev, stream, _p(dh),
            _float_code(dh.dtype), _p(x), _p(w), _p(dres), _p(dx), _p(dw), T, H, dt, wdt, eps,
            _p(ws), n)
    _used_on(stream, ws, *made)
    return dx, dw


def block_residual(x, f, *, w=None, norm=True, gate=None, gate_act="sigmoid", scale=1.0,
                   next_norm=False, w_next=None, eps=1e-5, out=None, h_out=None, stream=None):
    """(y, h): y = x + scale * a * z for the block's output f (x, f [T, H], float32 or bfloat16),
    z the norm of f times w (norm=False: f * w), a the gate or its sigmoid: per token (float32
    [T] or [T, 1]), per element ([T, H], x's type), or None for 1. With next_norm (or h_out, or
    w_next) h is the next block's norm of y, else None. out may be x or f. See moe_block_residual
    in moe.h."""
    T, H = _rows_of(x, "x")
    dev, made = x.device, []
    dt = _float_code(x.dtype)
    _need(f, (T, H), "f", x.dtype, dev)
    wdt = _weight_code(H, dev, x.dtype, w=w, w_next=w_next)
    flags = _gate_flags(gate, gate_act, x.shape, x.dtype, dev) | (BLOCK_NORM if norm else 0)
    y = _out(out, x, (T, H), x.dtype, "out", made)
    h = None
    if next_norm or w_next is not None or h_out is not None:
        h = _out(h_out, x, (T, H), x.dtype, "h_out", made)
    _launch(lib().moe_block_residual, "moe_block_residual", dev, stream, _p(x), _p(f), _p(w),
            _p(gate), _p(w_next), _p(y), _p(h), T, H, dt, wdt, flags, scale, eps)
    _used_on(stream, *made)
    return y, h


def block_residual_backward(dy, f, *, w=None, norm=True, gate=None, gate_act="sigmoid", scale=1.0,
                            y=None, dh=None, w_next=None, eps=1e-5, stream=None):
    """Gradients of block_residual as a dict: dx, df, and dw, dgate, dw_next where w, gate and
    w_next are given. dy [T, H] (f's type, or None where only h was used) reaches y; dh (f's type or
    float32), with the forward's y, reaches h. dw and dw_next are float32. See
    moe_block_residual_backward in moe.h."""
    T, H = _rows_of(f, "f")
    dev, made, dtype = f.device, [], f.dtype
    dt = _float_code(dtype)
    if dy is None and dh is None:
        raise ValueError("dy or dh is required")
    if dy is not None:
        _need(dy, (T, H), "dy", dtype, dev)
    dh_dt = dt
    if dh is not None:
        _need(dh, (T, H), "dh", None, dev)
        _need(y, (T, H), "y", dtype, dev)
        dh_dt = _float_code(dh.dtype)
    elif w_next is not None:
        raise ValueError("w_next has no gradient without dh")
    wdt = _weight_code(H, dev, dtype, w=w, w_next=w_next)
    flags = _gate_flags(gate, gate_act, f.shape, dtype, dev) | (BLOCK_NORM if norm else 0)
    out = {n: _out(None, f, (T, H), dtype, n, made) for n in ("dx", "df")}
    if gate is not None:
        out["dgate"] = _out(None, f, gate.shape, gate.dtype, "dgate", made)
    ws, n = None, 0
    if w is not None or w_next is not None:
        for name, t in (("dw", w), ("dw_next", w_next)):
            if t is not None:
                out[name] = _out(None, f, (H,), torch.float32, name, made)
        n = _block_workspace(T, H)
        ws = f.new_empty(n, dtype=torch.uint8)
    get = out.get
    _launch(lib().moe_block_residual_backward, "moe_block_residual_backward", dev, stream, _p(dy),
            _p(f), _p(w), _p(gate), _p(y), _p(dh), dh_dt, _p(w_next), _p(out["dx"]), _p(out["df"]),
            _p(get("dw")), _p(get("dgate")), _p(get("dw_next")), T, H, dt, wdt, flags, scale, eps,
            _p(ws), n)
    _used_on(stream, ws, *made)
    return out


# ----------------------------------------------------------------------------- gradient clipping

class GradClip:
    """Clipping of a fixed set of gradients (a list, or a dict's values; float32 and bfloat16,
    contiguous, one GPU) by their global norm, prepared once: ``__call__(max_norm)`` writes
    grad * min(1, max_norm / (norm + 1e-6)) into the gradients, or into ``out`` (as many tensors of
    the same shapes and types), and returns the norm (a float32 tensor that the next call
    overwrites; ``coef`` is beside it). A norm that is not finite leaves the values as they are.
    Calls of one GradClip must not overlap. See moe_clip_plan in moe.h."""

    def __init__(self, grads, *, out=None, stream=None):
        grads = list(grads.values()) if isinstance(grads, dict) else list(grads)
        outs = grads if out is None else list(out.values()) if isinstance(out, dict) else list(out)
        if not grads:
            raise ValueError("grads is empty")
        if len(outs) != len(grads):
            raise ValueError(f"{len(outs)} outputs for {len(grads)} gradients")
        dev = grads[0].device
        table = (MoeClipTensor * len(grads))()
        for i, (g, o) in enumerate(zip(grads, outs)):
            _need(g, g.shape, f"grads[{i}]", None, dev)
            _need(o, g.shape, f"out[{i}]", g.dtype, dev)
            table[i].grad, table[i].out, table[i].n = _p(g), _p(o), g.numel()
            table[i].dt = _float_code(g.dtype)
        self._check_apart(grads, outs)
        n = C.c_size_t(0)
        _check(lib().moe_clip_plan_size(table, len(grads), C.byref(n)), "moe_clip_plan_size")
        self._keep = (grads, outs)
        self.device = dev
        self.plan = grads[0].new_empty(n.value, dtype=torch.uint8)
        self.clip = MoeClip()
        _launch(lib().moe_clip_plan, "moe_clip_plan", dev, stream, table, len(grads), _p(self.plan),
                n.value, C.byref(self.clip))
        both = grads[0].new_empty(2, dtype=torch.float32)
        _used_on(stream, self.plan, both)
        self.norm, self.coef = both[0], both[1]
        self._args = (C.byref(self.clip), both.data_ptr())

    @staticmethod
    def _check_apart(grads, outs):
        """Every output lies apart from the others and from the other tensors' gradients."""
        spans = []
        for i, (g, o) in enumerate(zip(grads, outs)):
            for t, writes in ((o, True),) if o.data_ptr() == g.data_ptr() else ((g, False), (o, True)):
                if t.numel():
                    spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i, writes))
        spans.sort()
        end = written = 0    # ends of what was read or written, and of what was written, so far
        for lo, hi, i, writes in spans:
            if lo < written or (writes and lo < end):
                raise ValueError(f"gradient or output {i} overlaps another one that is written")
            end = max(end, hi)
            if writes:
                written = max(written, hi)

    def __call__(self, max_norm, stream=None):
        clip, norm = self._args
        _launch(lib().moe_clip_grads, "moe_clip_grads", self.device, stream, clip, max_norm, norm)
        return self.norm


def clip_grad_norm(grads, max_norm, *, out=None, stream=None):
    """GradClip for one use: clips grads (or into out) and returns their norm."""
    clip = GradClip(grads, out=out, stream=stream)
    _used_on(stream, *clip._keep[0], *clip._keep[1])
    return clip(max_norm, stream)
