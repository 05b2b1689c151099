"""GPU tests of the few-token layer's sums that end in a rounding to bf16 which decides more than one
bit: the rows of h of 8- and 4-bit experts, whose largest element sets the row's e4m3 scale, and
LatentMoE's u.

Each sum lies on a border of bf16 but for many terms that a sum rounded to fp32 as it grows loses
one by one. u of h's case: 17 (or 17 * 2^12) + 2656 terms t; 17^2 = 289 is the middle of the bf16
numbers 288 and 290 and goes to the even 288 without the terms. 32 of them, what one matrix-core
instruction adds, are 32 t = 2^-21, under half a step 2^-20 of 17 in fp32 (2^-13 under 2^-8 for
17 * 2^12); all of them move h by 34 * 2656 t = 1.3e-3, or 44 steps of fp32 (1.4e3 by 2.7), so h
is 290 in the definition's arithmetic. A kernel that sums up to 256 products in fp32 before it
widens loses at most the first 254 terms, and the rest still move h by 40 (2.5) steps. LatentMoE's
u: 257, the middle of 256 and 258, + 2656 terms 2^-26, 672 of which (a quarter of K) are under half
a step 2^-16 and all of which are 1.3 steps; without the first 254 terms they are 1.17, still
rounded to one. What follows is exact: the row's other codes are zero, weights and gates are 1.
"""
import numpy as np
import pytest

import moe_inputs as mi

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

pytestmark = pytest.mark.gpu
H, I = 2688, 32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield


def stack(v, w, scales=None):
    """One expert's weights v [1, rows, cols] in format w, exactly, with unit scales or those given."""
    if w == "bf16":
        return mi.f32_to_bf16_bits(v), None
    if w == "e4m3":
        return mi.encode_e4m3(v), np.ones(v.shape[:2], np.float32)
    s = np.full(v.shape[:2] + (v.shape[2] // 32,), 127, np.uint8)
    if scales is not None:
        s[:] = scales
    if w == "mxfp8":
        return mi.encode_e4m3(v), s
    c = mi.encode_e2m1(v)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8), s


def run(inp, w, T):
    inp = {n: v for n, v in inp.items() if v is not None}
    dev = moe.to_device(inp)
    rt = dict(idx=torch.zeros((T, 1), dtype=torch.int32, device="cuda"),
              gates=torch.ones((T, 1), device="cuda"))
    print(f"[gpu] few sums {w} T={T}", flush=True)
    y = moe.layer_from(dev, 1, path="few", routing=rt, routing_given=True, expert_dtype=w)()
    return y.double().cpu().numpy()


def layer(x, w, up, down, **kw):
    inp = dict(x=mi.f32_to_bf16_bits(x), W_r=mi.f32_to_bf16_bits(np.zeros((1, H), np.float32)),
               b=np.zeros(1, np.float32), **kw)
    (inp["W_up"], inp["s_up"]), (inp["W_down"], inp["s_down"]) = up, down
    return inp


@pytest.mark.parametrize("w", ["e4m3", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("T", [1, 3, 16])
def test_h_next_to_a_border(w, T):
    x = np.ones((T, H), np.float32)
    up = np.zeros((1, I, H), np.float32)
    scales, unit = None, 1.0
    x[:, 31] = 448.0                      # the row's scale is 1; its weight is zero
    if w == "e4m3":
        x[:, 0], x[:, 1], x[:, 32:] = 256.0, 16.0, 2.0 ** -9
        up[0, 5, :2], up[0, 5, 32:] = 256.0, 2.0 ** -9
        unit = 2.0 ** 24
    else:
        x[:, 0] = 16.0
        up[0, 5, :2] = up[0, 5, 32:] = 1.0
        scales = np.full(H // 32, 127 - 26, np.uint8)
        scales[0] = 127
    x[:, 2:31] = 0.0
    down = np.zeros((1, H, I), np.float32)
    down[0, :, 5] = 1.0
    y = run(layer(x, w, stack(up, w, scales), stack(down, w)), w, T)
    assert np.all(y == 290.0 * unit), y[0, 0] / unit


@pytest.mark.parametrize("w", ["bf16", "e4m3", "mxfp4", "mxfp8"])
def test_latent_u_next_to_a_border(w):
    L, T = 32, 3
    x = np.ones((T, H), np.float32)
    W_in = np.zeros((L, H), np.float32)
    W_in[3, 0], W_in[3, 1], W_in[3, 32:] = 256.0, 1.0, 2.0 ** -26
    W_out = np.zeros((H, L), np.float32)
    W_out[:, 7] = 1.0
    up = np.zeros((1, I, L), np.float32)
    up[0, 5, 3] = 1.0
    down = np.zeros((1, L, I), np.float32)
    down[0, 7, 5] = 1.0
    y = run(layer(x, w, stack(up, w), stack(down, w), W_in=mi.f32_to_bf16_bits(W_in),
                  W_out=mi.f32_to_bf16_bits(W_out)), w, T)
    # 258^2 = 66564, 66560 in bf16 (h of 8- and 4-bit experts, y); 256^2 = 65536
    assert np.all(y == 66560.0), y[0, 0]
