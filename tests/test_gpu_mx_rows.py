"""GPU test of the block-scaled experts on tiles: the experts' rows stay in fp32 until the gated sum,
so that y is rounded to bf16 once.

Inputs for which everything before the sum is exact but for fp32 roundings. x holds integers up to
7 and one 14, so the row scale 14 / 448 is a power of two and the codes are exact; every row of
W_up[e] is plus or minus one pattern of -1, 0 and 1, so that u is plus or minus one integer c, the
nonzero h are all bf16(c^2), their codes 448, and an expert's output is 448 (sum of some of W_down's
elements, a multiple of 1/2 below 2^11: exact) times fp32(bf16(c^2) / 448). The matrix core cuts
nothing: each group of eight products spans less than 13 bits (448 times 1/2 to 6; x's codes times 1).
fp32 roundings: the scale (2^-24), its product (2^-24), each of k products and k sums of the gated
sum (2^-24 of at most sum_j g_j |Y_j|): (2 k + 2) 2^-24 of that sum. Then y's own rounding, half a
step of bf16, at most 2^-8 of the value. Rows rounded to bf16 beforehand are off by up to 2^-8 of
each g_j |Y_j|, which the sum's cancellation leaves standing.
"""
import numpy as np
import pytest

import moe_inputs as mi

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("H,I", [(288, 160), (1056, 1056)])     # a tile per workgroup, walked tiles
@pytest.mark.parametrize("latent", [False, True])
def test_experts_rows_are_rounded_once(fmt, H, I, latent):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    T, E, k = 70, 8, 4
    rng = np.random.default_rng(H + I)
    x = rng.integers(-7, 8, (T, H)).astype(np.float32)
    x[:, 0] = 14.0
    pattern = rng.integers(-1, 2, (E, 1, H)).astype(np.float32)
    pattern[:, :, 0] = 0.0
    sign = rng.choice([-1.0, 1.0], (E, I, 1)).astype(np.float32)
    down = rng.choice([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6], (E, H, I)).astype(np.float32)

    def store(v):      # elements as they are, block scales of one
        if fmt == "mxfp8":
            codes = mi.encode_e4m3(v)
        else:
            c = mi.encode_e2m1(v)
            codes = (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)
        return codes, np.full(v.shape[:-1] + (v.shape[-1] // 32,), 127, np.uint8)

    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    gates = rng.uniform(0.2, 1.0, (T, k)).astype(np.float32)
    inp = dict(x=mi.f32_to_bf16_bits(x), W_r=mi.f32_to_bf16_bits(np.zeros((E, H), np.float32)),
               b=np.zeros(E, np.float32))
    inp["W_up"], inp["s_up"] = store(pattern * sign)
    inp["W_down"], inp["s_down"] = store(down)
    if latent:      # u = x and y = z, through identity projections
        inp["W_in"] = inp["W_out"] = mi.f32_to_bf16_bits(np.eye(H, dtype=np.float32))
    dev = moe.to_device(inp)
    rt = dict(idx=torch.from_numpy(idx).cuda(), gates=torch.from_numpy(gates).cuda())
    print(f"[gpu] rows {fmt} {H} {I} latent={latent}", flush=True)
    y = moe.layer_from(dev, k, path="grouped_mx", routing=rt, routing_given=True, expert_dtype=fmt)()
    y = y.double().cpu().numpy()

    c = x.astype(np.float64) @ (pattern[:, 0].T).astype(np.float64)            # [T, E]
    top = mi.bf16_bits_to_f32(mi.f32_to_bf16_bits((c ** 2).astype(np.float32))).astype(np.float64)
    ref = np.zeros((T, H))
    mass = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            on = (sign[e, :, 0] * c[t, e] > 0).astype(np.float64)
            out = top[t, e] * (down[e].astype(np.float64) @ on)
            ref[t] += float(gates[t, j]) * out
            mass[t] += float(gates[t, j]) * np.abs(out)
    # LatentMoE: z is rounded to a pair of bf16 (2^-17 of z) on its way to W_out
    slack = (2 * k + 2) * 2.0 ** -24 * mass + (2.0 ** -16 * np.abs(ref) if latent else 0.0)
    assert np.abs(ref).max() > 0
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + slack)
