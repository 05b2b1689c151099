"""Gates whose sigmoid is below the smallest normal fp32 value, where what they gate is as large."""
import pytest
import torch

import sparse_moe_layer_05_amd as moe

pytestmark = pytest.mark.gpu
Q = [87.0, 87.4, 88.0, 90.5, 95.0, 100.0, 103.0, 103.9, 105.0, 200.0]


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["token", "element"])
def test_sigmoids_below_the_smallest_normal(kind):
    """Bounds: a sigmoid or its complement is off by 8 roundings and, below 2^-126, by half of 2^-149
    twice (the exponential, its product with 1 / (1 + e)); what is multiplied by it afterwards rounds on
    the same grid once more and is then met by |f|."""
    q = torch.tensor([-v for v in Q] + Q)
    T, H = len(q), 48
    g = torch.Generator().manual_seed(1)
    f = (torch.randn(T, H, generator=g) * 1e30).cuda()
    dy = torch.randn(T, H, generator=g).cuda()
    gate = (q if kind == "token" else q[:, None].expand(T, H).contiguous()).cuda()
    zero = torch.zeros_like(f)
    q64, f64, d64 = q.double()[:, None], f.double().cpu(), dy.double().cpu()
    a, rest = torch.sigmoid(q64), torch.sigmoid(-q64)
    step = 2.0 ** -149

    y, _ = moe.block_residual(zero, f, norm=False, gate=gate)
    want = a * f64
    off = (y.double().cpu() - want).abs()
    assert bool((off <= 12 * 2.0 ** -24 * want.abs() + f64.abs() * step + step).all())

    got = moe.block_residual_backward(dy, f, norm=False, gate=gate)
    want = a * d64
    off = (got["df"].double().cpu() - want).abs()
    assert bool((off <= 12 * 2.0 ** -24 * want.abs() + (d64.abs() + 1) * step).all())
    want, mag = d64 * f64, (d64 * f64).abs()
    if kind == "token":
        want, mag = want.sum(1, keepdim=True), mag.sum(1, keepdim=True)
    want, mag = want * a * rest, mag
    off = (got["dgate"].double().cpu().reshape(want.shape) - want).abs()
    grid = mag * step + (f64.abs() * 2 * step if kind == "element" else 0) + step
    assert bool((off <= 64 * 2.0 ** -24 * mag * a * rest + 2 * grid).all())
