"""Block gradients whose workgroups walk over several rows each, against the formulas in float64 (on the
GPU, in elementary operations), with bounds that a single lost row exceeds."""
import pytest
import torch

import block_oracle as O
import sparse_moe_layer_05_amd as moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
SUM = 32 + 6 + 8
GRAD = 2 * (2 * SUM + 12)
# A weight's gradient: at most 4 rows one after another in a lane, the rows of a wave (3) and its
# workgroup (4), then at most 8 workgroups a lane, 3 steps of the wave and 16 waves. One row in T is
# 1 / T of the sum: 1.4e-5 for the most rows here, where the bound is 2^-24 (GRAD + 38) = 1.5e-5, and 1e-4
# and more elsewhere.
DEPTH = 4 + 3 + 4 + 8 + 3 + 16
SHAPES = [(70000, 16), (70000, 64), (33000, 128), (20000, 144), (9000, 288), (9000, 512), (9000, 1024),
          (4000, 1040), (2400, 2704), (2400, 4096), (700, 6160), (700, 8192), (600, 8208), (600, 16384)]
TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def make(g, *s, dtype=F32, scale=1.0, at=0.0):
    return (torch.randn(*s, generator=g, device="cuda") * scale + at).to(dtype)


def check(got, want, dtype, mag, steps, what):
    """Within one rounding to `dtype`, after `steps` fp32 roundings of terms that add up to mag."""
    slack = steps * O.U32 * mag
    off = (got.double() - want).abs()
    ok = off <= O.unit(dtype) * (want.abs() + slack) + slack + 2.0 ** -133
    assert got.dtype is dtype and got.shape == want.shape and bool(ok.all()), (what, int((~ok).sum()))


@pytest.mark.parametrize("kind", ["token", "element"])
@pytest.mark.parametrize("n,T,H", [(n, *s) for n, s in enumerate(SHAPES)])
def test_every_gradient_over_several_rows_a_workgroup(n, T, H, kind):
    for dtype, dh_dtype in TYPES if H in (16, 288, 2704, 4096) else TYPES[n % 3:n % 3 + 1]:
        g = torch.Generator("cuda").manual_seed(T + H)
        y, f = make(g, T, H, dtype=dtype, scale=2.0), make(g, T, H, dtype=dtype, scale=0.5)
        dy, dh = make(g, T, H, dtype=dtype, scale=0.1), make(g, T, H, dtype=dh_dtype, scale=0.1)
        w, wn = make(g, H, dtype=dtype, scale=0.2, at=1.0), make(g, H, dtype=dtype, scale=0.2, at=1.0)
        gate = make(g, T) if kind == "token" else make(g, T, H, dtype=dtype)
        got = moe.block_residual_backward(dy, f, w=w, gate=gate, scale=0.7, y=y, dh=dh, w_next=wn, eps=EPS)
        d = lambda t: t.double()  # noqa: E731
        ref = O.residual_grad(d(dy), d(f), d(w), True, d(gate), "sigmoid", 0.7, d(y), d(dh), d(wn), EPS)
        assert sorted(got) == sorted(ref)
        for name, (want, mag) in ref.items():
            sums = name in ("dw", "dw_next")
            dt = F32 if sums else gate.dtype if name == "dgate" else dtype
            check(got[name], want, dt, mag, GRAD + (DEPTH if sums else SUM), (name, dtype, dh_dtype))


@pytest.mark.parametrize("dtype,dh_dtype", TYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_the_norm_alone_over_several_rows_a_workgroup(T, H, dtype, dh_dtype):
    g = torch.Generator("cuda").manual_seed(T * 3 + H)
    x, dres = make(g, T, H, dtype=dtype, scale=2.0), make(g, T, H, dtype=dtype, scale=0.1)
    dh, w = make(g, T, H, dtype=dh_dtype, scale=0.1), make(g, H, dtype=dtype, scale=0.2, at=1.0)
    dx, dw = moe.block_norm_backward(dh, x, w, dres=dres, eps=EPS)
    v, gr, res = x.double(), dh.double() * w.double(), dres.double()
    check(dx, O.norm_grad(gr, v, EPS) + res, dtype, O.norm_grad(gr, v, EPS, mag=True) + res.abs(), GRAD, "dx")
    t = dh.double() * v / O.rms(v, EPS)
    check(dw, t.sum(0), F32, t.abs().sum(0), GRAD + DEPTH, "dw")
