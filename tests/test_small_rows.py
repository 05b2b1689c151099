"""Expert rows whose largest magnitude is so small that 448 / amax is past fp32 (amax < 1.3e-36):
the oracle on the CPU, and every path with 8- and 4-bit experts on the GPU against it.

Small x: rows of about 1e-37 and expert weights scaled up by 2^100, so that u, h and y are ordinary
numbers. Small h: rows of about 2^-62, whose squares lie near 5e-37 and below, and W_down scaled up
by 2^100. Half of h is zero, which an overflowed factor turned into NaN. Bar of the GPU paths
against the oracle that rounds the rows alike: 5e-3 relative Frobenius as for ordinary rows, one
bf16 rounding of y (2^-8 of the value at most, 2.3e-3 in the mean square) and, on the tiles, one of
the experts' rows.
"""
import numpy as np
import pytest

import moe_inputs as mi
from oracle import oracle as O

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

PATHS = [("e4m3", "grouped"), ("e4m3", "stream"), ("e4m3", "few"),
         ("mxfp4", "stream"), ("mxfp4", "grouped_mx"), ("mxfp4", "few"),
         ("mxfp8", "stream"), ("mxfp8", "grouped_mx"), ("mxfp8", "few")]


def scaled(s, n):
    """Per-channel fp32 scales or E8M0 codes, times 2^n."""
    return (s * np.float32(2.0 ** n)).astype(np.float32) if s.dtype == np.float32 \
        else (s.astype(np.int32) + n).astype(np.uint8)


def case(w, small, **kw):
    cfg = mi.LayerConfig("small", T=9, H=288, E=8, k=2, I=160, expert_dtype=w, **kw)
    inp = mi.make_layer(cfg, seed=3)
    x = mi.bf16_bits_to_f32(inp["x"])
    down, which = (-122, "s_up") if small == "x" else (-62, "s_down")
    x = x * np.float32(2.0 ** down)
    x[:, ::5] = 0.0
    x[1] = 0.0                       # a row of zeros beside them
    if small == "x":
        x[2] = 0.0
        x[2, 7] = 2.0 ** -133        # the smallest bf16 value
    inp["x"] = mi.f32_to_bf16_bits(x)
    inp[which] = scaled(inp[which], 100)
    t = np.arange(cfg.T)
    idx = np.stack((t % 8, (t + 3) % 8), 1).astype(np.int32)
    gates = np.full((cfg.T, 2), 0.5, np.float32)
    with np.errstate(all="ignore"):
        ref = O.forward_tokens(inp, idx, gates.astype(np.float64), t, True)
    return cfg, inp, idx, gates, ref


@pytest.mark.parametrize("w", ["e4m3", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("small", ["x", "h"])
def test_oracle_keeps_small_rows(w, small):
    """Against the same sums without the e4m3 rounding of the rows: at most 2^-4 of every element
    in two roundings, the first one squared (3 * 2^-4 in all), far less in the norm."""
    cfg, inp, idx, gates, ref = case(w, small)
    with np.errstate(all="ignore"):
        exact = O.forward_tokens(inp, idx, gates.astype(np.float64), np.arange(cfg.T), False)
    # x of 2^-122 and weights of 2^100 give u of 2^-22, y of 2^-44 = 6e-14; h of 2^-124, y of 2^-24
    assert np.isfinite(ref).all() and np.abs(exact).max() > 1e-15
    assert np.all(ref[1] == 0.0)
    assert np.linalg.norm(ref - exact) <= 3 / 16 * np.linalg.norm(exact)


@pytest.mark.gpu
@pytest.mark.parametrize("w,path", PATHS)
@pytest.mark.parametrize("small", ["x", "h"])
def test_layer_keeps_small_rows(w, path, small):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"[gpu] small {small} {w} {path}", flush=True)
    cfg, inp, idx, gates, ref = case(w, small)
    dev = moe.to_device(inp)
    rt = dict(idx=torch.from_numpy(idx).cuda(), gates=torch.from_numpy(gates).cuda())
    y = moe.layer_from(dev, cfg.k, path=path, routing=rt, routing_given=True, expert_dtype=w)()
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all()
    assert np.linalg.norm(y - ref) <= 5e-3 * np.linalg.norm(ref)
