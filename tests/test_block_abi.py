"""CPU checks of the operators around the layer (token rows, block norms, clipping): argument errors
are reported before anything is launched, the binding refuses tensors that do not fit, and the
oracle's gradients are those of its own forward passes."""
import ctypes as C

import pytest
import torch

import block_oracle as O
import sparse_moe_layer_05_amd as moe
from sparse_moe_layer_05_amd import binding as B
from sparse_moe_layer_05_amd import block as K

FAKE = C.c_void_p(0x10000)    # aligned, never dereferenced: validation fails or returns first
ODD = C.c_void_p(0x10004)
BAD, UNS, WS, OK = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE, B.MOE_OK
BIG = 1 << 40

SHAPE = [
    (dict(T=-1), BAD), (dict(D=0), BAD), (dict(D=8), BAD), (dict(D=24), BAD), (dict(D=-16), BAD),
    (dict(D=(1 << 20) + 16), BAD), (dict(k=0), BAD), (dict(k=65), BAD),
    (dict(T=(1 << 25) + 1, k=1), BAD), (dict(T=1 << 25, D=528, k=1), BAD),
    (dict(T=1 << 25, D=16, k=64), BAD),
]


@pytest.mark.parametrize("kw,code", SHAPE + [
    (dict(E=0), BAD), (dict(E=1025), BAD), (dict(dt=B.MOE_FP8_E4M3), UNS), (dict(x=None), BAD),
    (dict(idx=None), BAD), (dict(rows=None), BAD), (dict(offsets=None), BAD), (dict(pos=None), BAD),
    (dict(x=ODD), BAD), (dict(rows=ODD), BAD), (dict(ws=None), WS), (dict(ws=ODD), WS),
    (dict(n=16), WS),
])
def test_sort_argument_errors(kw, code):
    a = dict(x=FAKE, dt=1, idx=ODD, w=None, T=4000, D=64, E=8, k=2, rows=FAKE, offsets=ODD, pos=ODD,
             ws=FAKE, n=BIG)
    a.update(kw)
    assert moe.lib().moe_sort_tokens(*a.values(), None) == code


def test_sort_workspace_size():
    n = C.c_size_t(0)
    L = moe.lib()
    assert L.moe_sort_tokens_workspace_size(4000, 8, 2, C.byref(n)) == OK and n.value >= 8 * 4
    assert L.moe_sort_tokens_workspace_size(1 << 18, 1024, 2, C.byref(n)) == OK and n.value >= 8 << 18
    assert L.moe_sort_tokens_workspace_size(64, 8, 2, C.byref(n)) == OK and n.value == 0
    assert L.moe_sort_tokens_workspace_size(64, 2, 8, C.byref(n)) == OK   # a rank with few experts
    assert L.moe_sort_tokens_workspace_size(0, 8, 2, C.byref(n)) == OK
    for bad in ((-1, 8, 2), (4, 0, 2), (4, 1025, 2), (4, 8, 0), (4, 8, 65), (1 << 30, 8, 64)):
        assert L.moe_sort_tokens_workspace_size(*bad, C.byref(n)) == BAD, bad
    assert L.moe_sort_tokens_workspace_size(64, 8, 2, None) == BAD


@pytest.mark.parametrize("kw,code", SHAPE + [
    (dict(T=0), OK), (dict(n=-1), BAD), (dict(dt=2), UNS), (dict(dx_dt=4), UNS),
    (dict(drows=None), BAD), (dict(pos=None), BAD), (dict(dx=None), BAD), (dict(x=None), BAD),
    (dict(drows=ODD), BAD), (dict(x=ODD), BAD), (dict(dx=ODD), BAD),
])
def test_sort_backward_argument_errors(kw, code):
    a = dict(drows=FAKE, x=FAKE, dt=1, pos=ODD, w=ODD, T=4, D=64, k=2, n=8, dx=FAKE, dx_dt=0,
             dweights=ODD)
    a.update(kw)
    assert moe.lib().moe_sort_tokens_backward(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", SHAPE + [
    (dict(T=0), OK), (dict(n=-1), BAD), (dict(dt=2), UNS), (dict(y_dt=4), UNS),
    (dict(rows=None), BAD), (dict(pos=None), BAD), (dict(y=None), BAD), (dict(rows=ODD), BAD),
    (dict(add=ODD), BAD), (dict(y=ODD), BAD),
])
def test_unsort_argument_errors(kw, code):
    a = dict(rows=FAKE, dt=1, pos=ODD, w=ODD, add=FAKE, T=4, D=64, k=2, n=8, y=FAKE, y_dt=0)
    a.update(kw)
    assert moe.lib().moe_unsort_tokens(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", SHAPE + [
    (dict(T=0), OK), (dict(n=-1), BAD), (dict(dt=2), UNS), (dict(dy_dt=4), UNS), (dict(dy=None), BAD),
    (dict(rows=None), BAD), (dict(pos=None), BAD), (dict(drows=None), BAD), (dict(dy=ODD), BAD),
    (dict(rows=ODD), BAD), (dict(drows=ODD), BAD), (dict(dweights=None, dt=0), UNS),
])
def test_unsort_backward_argument_errors(kw, code):
    a = dict(dy=FAKE, dy_dt=1, rows=FAKE, dt=1, pos=ODD, w=ODD, T=4, D=64, k=2, n=8, drows=FAKE,
             dweights=ODD)
    a.update(kw)
    assert moe.lib().moe_unsort_tokens_backward(*a.values(), None) == code


INF, NAN = float("inf"), float("nan")
BLOCK = [
    (dict(T=0), OK), (dict(T=-1), BAD), (dict(T=1 << 23), BAD), (dict(H=0), BAD),
    (dict(H=24), BAD), (dict(H=16400), BAD), (dict(H=-16), BAD), (dict(eps=0.0), BAD), (dict(eps=1e-31), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD), (dict(dt=2), UNS),
    (dict(w_dt=3), UNS),
]
FLAGS = [(dict(flags=16), BAD), (dict(flags=6), BAD), (dict(scale=INF), BAD), (dict(scale=NAN), BAD)]


@pytest.mark.parametrize("kw,code", BLOCK + [
    (dict(x=None), BAD), (dict(h=None), BAD), (dict(x=ODD), BAD), (dict(w=ODD), BAD),
    (dict(h=ODD), BAD),
])
def test_norm_argument_errors(kw, code):
    a = dict(x=FAKE, w=FAKE, h=FAKE, T=4, H=64, dt=1, w_dt=1, eps=1e-5)
    a.update(kw)
    assert moe.lib().moe_block_norm(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", BLOCK + FLAGS + [
    (dict(x=None), BAD), (dict(f=None), BAD), (dict(y=None), BAD), (dict(gate=None, flags=2), BAD),
    (dict(flags=1), BAD), (dict(x=ODD), BAD), (dict(f=ODD), BAD), (dict(w=ODD), BAD),
    (dict(gate=ODD), BAD), (dict(w_next=ODD), BAD), (dict(y=ODD), BAD), (dict(h=ODD), BAD),
])
def test_residual_argument_errors(kw, code):
    a = dict(x=FAKE, f=FAKE, w=FAKE, gate=FAKE, w_next=FAKE, y=FAKE, h=FAKE, T=4, H=64, dt=1, w_dt=1,
             flags=11, scale=1.0, eps=1e-5)
    a.update(kw)
    assert moe.lib().moe_block_residual(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [b for b in BLOCK if b[0] != dict(T=0)] + [
    (dict(dh=None), BAD), (dict(x=None), BAD), (dict(dx=None), BAD), (dict(dh=ODD), BAD),
    (dict(dres=ODD), BAD), (dict(x=ODD), BAD), (dict(dx=ODD), BAD), (dict(ws=None), WS),
    (dict(n=16), WS), (dict(ws=ODD), WS), (dict(dt=0, dh_dt=1), UNS), (dict(dh_dt=2), UNS),
    (dict(T=0, dw=None), OK),
])
def test_norm_backward_argument_errors(kw, code):
    a = dict(dh=FAKE, dh_dt=0, x=FAKE, w=FAKE, dres=FAKE, dx=FAKE, dw=ODD, T=4, H=64, dt=1, w_dt=1,
             eps=1e-5, ws=FAKE, n=BIG)
    a.update(kw)
    assert moe.lib().moe_block_norm_backward(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [b for b in BLOCK if b[0] != dict(T=0)] + FLAGS + [
    (dict(dy=None, dh=None, dw_next=None), BAD), (dict(f=None), BAD), (dict(y=None), BAD),
    (dict(dx=None), BAD), (dict(df=None), BAD), (dict(dh=None), BAD), (dict(gate=None), BAD),
    (dict(flags=1), BAD), (dict(ws=None), WS), (dict(n=16), WS), (dict(dt=0, dh_dt=1), UNS),
    (dict(dy=ODD), BAD), (dict(f=ODD), BAD), (dict(w=ODD), BAD), (dict(gate=ODD), BAD),
    (dict(y=ODD), BAD), (dict(dh=ODD), BAD), (dict(w_next=ODD), BAD), (dict(dx=ODD), BAD),
    (dict(df=ODD), BAD), (dict(dgate=ODD), BAD), (dict(T=0, dw=None, dw_next=None), OK),
])
def test_residual_backward_argument_errors(kw, code):
    a = dict(dy=FAKE, f=FAKE, w=FAKE, gate=FAKE, y=FAKE, dh=FAKE, dh_dt=1, w_next=FAKE, dx=FAKE,
             df=FAKE, dw=ODD, dgate=FAKE, dw_next=ODD, T=4, H=64, dt=1, w_dt=1, flags=11, scale=1.0,
             eps=1e-5, ws=FAKE, n=BIG)
    a.update(kw)
    assert moe.lib().moe_block_residual_backward(*a.values(), None) == code


def table(*rows):
    t = (B.MoeClipTensor * max(1, len(rows)))()
    for i, (g, o, n, dt) in enumerate(rows):
        t[i].grad, t[i].out, t[i].n, t[i].dt = g, o, n, dt
    return t


@pytest.mark.parametrize("rows,count,code", [
    ([(0x1000, None, 5, 0)], 1, OK), ([(0x1002, 0x2002, 5, 1)], 1, OK), ([], 0, OK),
    ([(None, None, 0, 0)], 1, OK), ([(None, None, 5, 0)], 1, BAD), ([(0x1002, None, 5, 0)], 1, BAD),
    ([(0x1001, None, 5, 1)], 1, BAD), ([(0x1000, 0x2002, 5, 0)], 1, BAD),
    ([(0x1000, None, -1, 0)], 1, BAD), ([(0x1000, None, 1 << 49, 0)], 1, BAD),
    ([(0x1000, None, 1 << 43, 0)], 1, BAD),
    ([(0x1000, None, 5, 2)], 1, UNS), ([(0x1000, None, 5, 0)], -1, BAD),
    ([(0x1000, None, 5, 0)], 65537, BAD),
])
def test_clip_plan_argument_errors(rows, count, code):
    n = C.c_size_t(0)
    L = moe.lib()
    assert L.moe_clip_plan_size(table(*rows), count, C.byref(n)) == code
    clip = B.MoeClip()
    if code != OK:
        assert L.moe_clip_plan(table(*rows), count, FAKE, BIG, C.byref(clip), None) == code
        return
    assert L.moe_clip_plan(table(*rows), count, None, BIG, C.byref(clip), None) == WS
    assert L.moe_clip_plan(table(*rows), count, ODD, BIG, C.byref(clip), None) == WS
    assert L.moe_clip_plan(table(*rows), count, FAKE, n.value - 1, C.byref(clip), None) == WS
    assert L.moe_clip_plan(table(*rows), count, FAKE, BIG, None, None) == BAD
    if not any(r[2] for r in rows):      # nothing to write: no launch
        assert L.moe_clip_plan(table(*rows), count, FAKE, n.value, C.byref(clip), None) == OK
        assert clip.chunks == 0


def test_clip_argument_errors():
    L = moe.lib()
    assert L.moe_clip_plan_size(None, 1, C.byref(C.c_size_t(0))) == BAD
    assert L.moe_clip_plan_size(table((0x1000, None, 5, 0)), 1, None) == BAD
    clip = B.MoeClip()
    assert L.moe_clip_grads(C.byref(clip), 1.0, FAKE, None) == BAD          # never filled
    clip.plan = FAKE.value
    for bad in (-1.0, NAN):
        assert L.moe_clip_grads(C.byref(clip), bad, FAKE, None) == BAD
    assert L.moe_clip_grads(C.byref(clip), 1.0, None, None) == BAD
    assert L.moe_clip_grads(C.byref(clip), 1.0, C.c_void_p(0x10002), None) == BAD
    assert L.moe_clip_grads(None, 1.0, FAKE, None) == BAD
    clip.plan = ODD.value
    assert L.moe_clip_grads(C.byref(clip), 1.0, FAKE, None) == BAD


def test_binding_refuses_what_does_not_fit():
    f32, bf = torch.float32, torch.bfloat16
    z = lambda *s, d=f32: torch.zeros(s, dtype=d)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for n, call in enumerate((
            lambda: moe.sort_tokens(z(4, 32), i(4, 2), 8),                       # not on a GPU
            lambda: moe.sort_tokens(z(4, 32), i(3, 2), 8),
            lambda: moe.sort_tokens(z(4, 32), i(4, 2).long(), 8),
            lambda: moe.sort_tokens(z(4, 32), i(8), 8),
            lambda: moe.sort_tokens(z(4, 2, 16), i(4, 2), 8),
            lambda: moe.sort_tokens(z(4, 32, d=torch.float16), i(4, 2), 8),
            lambda: moe.sort_tokens(z(4, 32), i(4, 2), 8, weights=z(4, 2, d=bf)),
            lambda: moe.sort_tokens(z(4, 32), i(4, 2), 8, weights=z(4, 3)),
            lambda: moe.sort_tokens(z(4, 32), i(4, 2), 8, out=z(7, 32)),
            lambda: moe.sort_tokens(z(4, 64)[:, ::2], i(4, 2), 8),               # strided
            lambda: moe.sort_tokens_backward(z(8, 32), i(4, 2), x=z(4, 16)),
            lambda: moe.sort_tokens_backward(z(8, 32), i(4, 2), x=z(4, 32, d=bf)),
            lambda: moe.sort_tokens_backward(z(8, 32), i(4, 2)),                 # not on a GPU
            lambda: moe.unsort_tokens(z(8, 32), i(4, 2)),
            lambda: moe.unsort_tokens(z(8, 32), i(4, 2), add=z(3, 32)),
            lambda: moe.unsort_tokens(z(8, 32), i(4, 2), add=z(4, 32), out_dtype=bf),
            lambda: moe.unsort_tokens(z(8, 32), i(4, 2), out=z(4, 32), out_dtype=bf),
            lambda: moe.unsort_tokens_backward(z(4, 32), i(4, 2)),
            lambda: moe.unsort_tokens_backward(z(4, 32), i(4, 2), rows=z(8, 16)),
            lambda: moe.unsort_tokens_backward(z(4, 32), i(4, 2), rows=z(8, 32), out=z(9, 32)),
            lambda: moe.unsort_tokens_backward(z(4, 32), i(4, 2), out=z(8, 32, d=bf)),
            lambda: moe.unsort_tokens(torch.empty(1, 16).expand(1 << 32, 16), i(4, 2)),
            lambda: moe.block_norm(z(4, 32)),
            lambda: moe.block_norm(z(32)),
            lambda: moe.block_norm(z(4, 32), z(16)),
            lambda: moe.block_norm(z(4, 32), z(32, d=torch.float16)),
            lambda: moe.block_norm_backward(z(4, 32), z(4, 32), dres=z(4, 32, d=bf)),
            lambda: moe.block_norm_backward(z(4, 16), z(4, 32)),
            lambda: moe.block_residual(z(4, 32), z(4, 32)),
            lambda: moe.block_residual(z(4, 32), z(4, 32, d=bf)),
            lambda: moe.block_residual(z(4, 32), z(4, 32), gate=z(4, 2)),
            lambda: moe.block_residual(z(4, 32), z(4, 32), gate=z(4, d=bf)),
            lambda: moe.block_residual(z(4, 32), z(4, 32), gate=z(4, 32, d=bf)),
            lambda: moe.block_residual(z(4, 32), z(4, 32), gate=z(4), gate_act="silu"),
            lambda: moe.block_residual(z(4, 32), z(4, 32), w=z(32), w_next=z(32, d=bf)),
            lambda: moe.block_residual_backward(None, z(4, 32)),
            lambda: moe.block_residual_backward(None, z(4, 32), dh=z(4, 32)),    # no y
            lambda: moe.block_residual_backward(z(4, 32), z(4, 32), w_next=z(32)),
            lambda: moe.block_residual_backward(z(4, 32), z(4, 32)),
            lambda: moe.GradClip([]),
            lambda: moe.GradClip([z(4), z(4)], out=[z(4)]),
            lambda: moe.GradClip([z(4)], out=[z(5)]),
            lambda: moe.GradClip([z(4, d=torch.float16)]),
            lambda: moe.GradClip([z(8)[::2]]),
            lambda: moe.GradClip([z(4)]))):                                      # not on a GPU
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was taken")


def test_clip_refuses_overlap():
    flat, other = torch.zeros(64), torch.zeros(64)

    def apart(grads, outs):
        spans = []
        for g, o in zip(grads, outs):
            size = 4 * g.numel()
            if o.data_ptr() != g.data_ptr():
                spans.append((g.data_ptr(), g.data_ptr() + size, False))
            spans.append((o.data_ptr(), o.data_ptr() + size, True))
        K._check_apart(spans)

    apart([flat[:8], flat[8:20]], [flat[:8], flat[8:20]])
    apart([flat[:8], flat[4:12]], [other[:8], other[8:16]])       # read twice, written apart
    for grads, outs in (([flat[:8]] * 2, [flat[:8]] * 2),                     # the same one twice
                        ([flat[:8], flat[4:12]], [flat[:8], flat[4:12]]),
                        ([flat[:8]], [flat[4:12]]),                           # over itself, shifted
                        ([flat[:8], flat[8:16]], [flat[8:16], other[:8]]),    # over another's
                        ([flat[:8], flat[8:16]], [other[:8], other[4:12]])):
        with pytest.raises(ValueError):
            apart(grads, outs)


# --------------------------------------------------- the oracle's gradients against differences

def differences(fn, x, h=1e-6):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        p, m = x.clone(), x.clone()
        p.view(-1)[i] += h
        m.view(-1)[i] -= h
        g.view(-1)[i] = (fn(p) - fn(m)) / (2 * h)
    return g


@pytest.mark.parametrize("gate,act", [(None, "none"), ("token", "sigmoid"), ("token", "none"),
                                      ("element", "sigmoid"), ("element", "none")])
@pytest.mark.parametrize("norm", [True, False])
def test_block_gradients_against_differences(gate, act, norm):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, H, eps, scale = 3, 5, 1e-2, 0.7
    v = dict(x=r(T, H), f=r(T, H), w=r(H), w_next=r(H),
             gate=None if gate is None else r(T) if gate == "token" else r(T, H))
    cy, ch = r(T, H), r(T, H)

    def loss(**kw):
        a = dict(v, **kw)
        y, _ = O.residual(a["x"], a["f"], a["w"], norm, a["gate"], act, scale, eps)
        return float((cy * y).sum() + (ch * (y / O.rms(y, eps) * a["w_next"])).sum())

    y, _ = O.residual(v["x"], v["f"], v["w"], norm, v["gate"], act, scale, eps)
    got = O.residual_grad(cy, v["f"], v["w"], norm, v["gate"], act, scale, y, ch, v["w_next"], eps)
    for name in ("x", "f", "w", "w_next", "gate"):
        if v[name] is None:
            continue
        want = differences(lambda t: loss(**{name: t}), v[name])
        # central differences of step 1e-6: rounding 1e-16 / 1e-6 of values up to some tens
        assert torch.allclose(got["d" + name][0], want, rtol=1e-7, atol=1e-7), name


def test_row_gradients_against_differences():
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    idx = torch.tensor([[2, 0, 7], [1, 1, 0], [5, -1, 9]], dtype=torch.int32)
    T, k, D, E = 3, 3, 4, 3
    offsets, pos = O.positions(idx, E)
    assert offsets.tolist() == [0, 2, 3, 4] and pos.tolist() == [[3, 0, -1], [2, -1, 1], [-1, -1, -1]]
    n = T * k
    x, w, rows, c, cy = r(T, D), r(T, k), r(n, D), r(n, D), r(T, D)
    zero = torch.zeros(n, D, dtype=torch.float64)
    kept = torch.zeros(n, 1, dtype=torch.float64)
    kept[:4] = 1
    sort = lambda x, w: float((kept * c * O.spread(x, pos, w, zero)).sum())  # noqa: E731
    assert torch.allclose(differences(lambda t: sort(t, w), x), O.gather(c, pos, w, None, T, D), atol=1e-7)
    assert torch.allclose(differences(lambda t: sort(x, t), w), O.dots(x, c, pos), atol=1e-7)
    back = lambda rows, w: float((cy * O.gather(rows, pos, w, x, T, D)).sum())  # noqa: E731
    assert torch.allclose(differences(lambda t: back(t, w), rows), O.spread(cy, pos, w, zero), atol=1e-7)
    assert torch.allclose(differences(lambda t: back(rows, t), w), O.dots(cy, rows, pos), atol=1e-7)


# ------------------------------------------- sizes that the library's 32-bit arguments do not hold

def test_rows_past_32_bits_are_refused():
    """A size is passed as 32 bits: 2^32 + 8 must not arrive as 8."""
    f32 = torch.float32
    z = lambda *s: torch.zeros(s, dtype=f32)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    long = torch.empty(1, 16).expand((1 << 32) + 8, 16)
    for call, word in (
            (lambda: moe.unsort_tokens_backward(z(4, 16), i(4, 2), rows=long), "2^31"),
            (lambda: moe.unsort_tokens_backward(z(4, 16), i(4, 2), out=long), "2^31"),
            (lambda: moe.unsort_tokens_backward(z(4, 16), i(4, 2), n_rows=(1 << 32) + 8), "n_rows"),
            (lambda: moe.unsort_tokens_backward(z(4, 16), i(4, 2), n_rows=-1), "n_rows"),
            (lambda: moe.unsort_tokens_backward(z(4, 16), i(4, 2), rows=z(8, 16), n_rows=9), "expected"),
            (lambda: moe.unsort_tokens_backward(z(4, 16), i(4, 2), rows=z(8)), "two dimensions")):
        with pytest.raises(ValueError, match=word.replace("^", r"\^")):
            call()


def test_numbers_of_experts_that_there_cannot_be_are_refused_first():
    """Before anything of that size is allocated, and none arrives as another one."""
    x, idx = torch.zeros(4, 32), torch.zeros(4, 2, dtype=torch.int32)
    for E in ((1 << 32) + 8, (1 << 31) + 1, -5):
        with pytest.raises(ValueError, match="E is"):
            moe.sort_tokens(x, idx, E)
    for E in (0, 1025, (1 << 31) - 1):
        with pytest.raises(moe.MoeError):
            moe.sort_tokens(x, idx, E)


# ------------------------------------------------- arrays of 32-bit values: aligned to 4 bytes

HALF = C.c_void_p(0x10002)


@pytest.mark.parametrize("fn,args,names", [
    ("moe_sort_tokens", dict(x=FAKE, dt=1, idx=ODD, w=ODD, T=4000, D=64, E=8, k=2, rows=FAKE, offsets=ODD,
                             pos=ODD, ws=FAKE, n=BIG), ("idx", "w", "offsets", "pos")),
    ("moe_sort_tokens_backward", dict(drows=FAKE, x=FAKE, dt=1, pos=ODD, w=ODD, T=4, D=64, k=2, n=8, dx=FAKE,
                                      dx_dt=0, dweights=ODD), ("pos", "w", "dweights")),
    ("moe_unsort_tokens", dict(rows=FAKE, dt=1, pos=ODD, w=ODD, add=FAKE, T=4, D=64, k=2, n=8, y=FAKE,
                               y_dt=0), ("pos", "w")),
    ("moe_unsort_tokens_backward", dict(dy=FAKE, dy_dt=1, rows=FAKE, dt=1, pos=ODD, w=ODD, T=4, D=64, k=2,
                                        n=8, drows=FAKE, dweights=ODD), ("pos", "w", "dweights")),
    ("moe_block_norm_backward", dict(dh=FAKE, dh_dt=0, x=FAKE, w=FAKE, dres=FAKE, dx=FAKE, dw=ODD, T=4, H=64,
                                     dt=1, w_dt=1, eps=1e-5, ws=FAKE, n=BIG), ("dw",)),
    ("moe_block_residual_backward", dict(dy=FAKE, f=FAKE, w=FAKE, gate=FAKE, y=FAKE, dh=FAKE, dh_dt=1,
                                         w_next=FAKE, dx=FAKE, df=FAKE, dw=ODD, dgate=FAKE, dw_next=ODD,
                                         T=4, H=64, dt=1, w_dt=1, flags=11, scale=1.0, eps=1e-5, ws=FAKE,
                                         n=BIG), ("dw", "dw_next")),
])
def test_misaligned_arrays_of_words(fn, args, names):
    for name in names:
        assert getattr(moe.lib(), fn)(*dict(args, **{name: HALF}).values(), None) == BAD, name
