"""Block gradients of rows and gradients far from 1, against the formulas in float64: what the row's sums
meet on the way may leave fp32 where the gradient does not."""
import pytest
import torch

import block_oracle as O
import sparse_moe_layer_05_amd as moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# fp32 roundings on the longest path: a sum over a row is 32 columns a lane, the wave and its waves; a
# gradient joins two sums and about ten operations, twice where the second norm's meets the first's
SUM = 32 + 6 + 8
GRAD = 2 * (2 * SUM + 12)
WIDTHS = [16, 64, 304, 1040, 2704, 4112, 16384]


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def near(g, T, H, size, dtype):
    return ((torch.randn(T, H, generator=g) * 0.1 + 1) * size).to(dtype).cuda()


# rows of size y, gradients of size dh, eps: products of the two above fp32 and, in a row of its own,
# subnormal; their sum times 1 / rms above fp32; rows whose squares leave fp32 under small and large
# gradients
SIZES = [(1e15, 1e23, 1e-5), (1e-14, 1e-28, 1e-30), (1e-8, 1e-33, 1e-30), (1e-14, 1e-36, 1e-30),
         (1e25, 1e-20, 1e-5), (1e30, 1e30, 1e-5), (1e37, 1.0, 1e-5), (1.0, 1e-30, 1e-5)]


@pytest.mark.parametrize("dtype,dh_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm_gradients_of_far_rows(H, dtype, dh_dtype):
    g = torch.Generator().manual_seed(H)
    for size, grad, eps in SIZES:
        x = (torch.randn(5, H, generator=g) * size).to(dtype).cuda()
        dh = (torch.randn(5, H, generator=g) * grad).to(dh_dtype).cuda()
        w = (torch.randn(H, generator=g) * 0.2 + 1).cuda()
        x[3], dh[4] = 0, 0
        dx, dw = moe.block_norm_backward(dh, x, w, eps=eps)
        v, gr = O.f64(x), O.f64(dh) * O.f64(w)
        O.check(dx, O.norm_grad(gr, v, eps), dtype, O.norm_grad(gr, v, eps, mag=True), GRAD, (size, grad))
        t = O.f64(dh) * v / O.rms(v, eps)
        O.check(dw, t.sum(0), F32, t.abs().sum(0), GRAD + 5, ("dw", size, grad))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_gradients_along_their_row(H, dtype):
    """Rows and gradients of one sign: the sums of their products are H times one of them."""
    g = torch.Generator().manual_seed(H + 1)
    for size in (1.0, 1e10) if H < 300 else (0.01, 1.0, 1e10):
        x, dh = near(g, 4, H, size, dtype), near(g, 4, H, 1e39 / H, dtype)
        dx, _ = moe.block_norm_backward(dh, x, eps=1e-12)
        O.check(dx, O.norm_grad(O.f64(dh), O.f64(x), 1e-12), dtype,
                O.norm_grad(O.f64(dh), O.f64(x), 1e-12, mag=True), GRAD, size)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_residual_gradients_along_their_row(H, dtype):
    """The same of the output's norm: dy along f. A gate per token scales the sum after it is taken."""
    g = torch.Generator().manual_seed(H + 3)
    f, dy = near(g, 4, H, 1.0, dtype), near(g, 4, H, 1e39 / H, dtype)
    tiny = torch.tensor([0.0, 1e-30, 1e-3, 0.5]).cuda()
    for gate in (None, near(g, 4, H, 1.0, dtype), tiny):
        got = moe.block_residual_backward(dy, f, gate=gate, gate_act="none")
        ref = O.residual_grad(O.f64(dy), O.f64(f), None, True, O.f64(gate), "none", 1.0, None, None, None, 1e-5)
        for n in got:
            if n == "dgate" and gate is tiny:       # H times dy: past fp32 by itself
                assert bool(torch.isinf(got[n]).all())
                continue
            O.check(got[n], ref[n][0], dtype, ref[n][1], GRAD + SUM, n)


@pytest.mark.parametrize("dtype,dh_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("H", [64, 304, 2704])
def test_residual_gradients_of_far_rows(H, dtype, dh_dtype):
    g = torch.Generator().manual_seed(H + 2)
    for size, grad, eps in SIZES:
        y = (torch.randn(5, H, generator=g) * size).to(dtype).cuda()
        f = (torch.randn(5, H, generator=g) * size).to(dtype).cuda()
        dh = (torch.randn(5, H, generator=g) * grad).to(dh_dtype).cuda()
        dy = torch.zeros(5, H, dtype=dtype, device="cuda")
        got = moe.block_residual_backward(dy, f, y=y, dh=dh, eps=eps)
        ref = O.residual_grad(O.f64(dy), O.f64(f), None, True, None, "none", 1.0, O.f64(y), O.f64(dh), None, eps)
        if float(ref["df"][1].max()) > 1e38:      # past fp32 by itself
            continue
        for n in got:
            O.check(got[n], ref[n][0], dtype, ref[n][1], GRAD + SUM, (n, size, grad))


@pytest.mark.parametrize("H", [16, 64, 128, 208, 256, 304, 1040, 2704])
def test_far_rows_leave_the_others_alone(H):
    """Rows that are summed again, next to rows that are not, in one wave where they are short: those come
    out bit for bit as without them, and all as they should."""
    g = torch.Generator().manual_seed(H + 4)
    T = 70
    f, y = torch.randn(T, H, generator=g).cuda(), torch.randn(T, H, generator=g).cuda()
    dy, dh = torch.randn(T, H, generator=g).cuda(), torch.randn(T, H, generator=g).cuda()
    gate = torch.randn(T, generator=g).cuda()
    clean = moe.block_residual_backward(dy, f, gate=gate, y=y, dh=dh)
    far = torch.rand(T, generator=g) < 0.4
    kind = torch.randint(0, 4, (T,), generator=g)
    for t in torch.nonzero(far).flatten().tolist():
        if kind[t] == 0:
            y[t] *= 1e30
        elif kind[t] == 1:
            y[t] *= 1e15
            dh[t] *= 1e23
        elif kind[t] == 2:
            dh[t] = 0
        else:
            f[t] *= 1e25
    got = moe.block_residual_backward(dy, f, gate=gate, y=y, dh=dh)
    ref = O.residual_grad(O.f64(dy), O.f64(f), None, True, O.f64(gate), "sigmoid", 1.0, O.f64(y), O.f64(dh), None,
                          1e-5)
    near_rows = ~far
    for n in got:
        assert torch.equal(got[n].cpu()[near_rows], clean[n].cpu()[near_rows]), n
        O.check(got[n], ref[n][0], F32, ref[n][1], GRAD + SUM, n)


def test_rows_without_a_gradient_pass_what_reaches_them():
    """dh of zeros, as a masked token leaves it: dx is dres bit for bit, whatever the row."""
    g = torch.Generator().manual_seed(3)
    for H in WIDTHS:
        x, dres = torch.randn(6, H, generator=g).cuda(), torch.randn(6, H, generator=g).cuda()
        x[1] *= 1e30
        x[2] = 0
        dx, _ = moe.block_norm_backward(torch.zeros_like(x), x, dres=dres)
        assert torch.equal(dx, dres), H
