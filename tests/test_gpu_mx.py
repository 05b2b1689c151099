"""GPU tests of the block-scaled (OCP microscaling) operators.

Conversion: codes, scales and decoded values bit for bit against the encoder of ``moe_inputs``.
Product: against numpy in 64 bits on the decoded operands. The products of two elements and two
powers of two are exact in fp32 (at most 8 significant bits), so only the K additions round: a
sum of K terms is off by at most K * u * sum |a w| with u the unit of one addition. u = 2^-23
covers an accumulator that truncates (2^-24 is half a step of one that rounds); a bf16 result is
off by another 2^-8 of its value. With an E4M3 operand the matrix core first cuts the products of
each eight consecutive k to multiples of 2^(e - 13), e the exponent of the group's largest product
(two nonzero products show it: 2^12 + 1.5 * 2^(12 - r) keeps the small one whole up to r = 12, as
0.5 of 0.75 at r = 13, not at all from r = 14; nine apart both stay up to r = 22). The largest
itself has 8 significant bits and is kept, so a group of eight loses less than
7 * 2^-13 * (its largest product), each group's share being at most that.
Layer with block-scaled experts on matrix-core tiles: against the double-precision oracle that
rounds the expert rows as the layer does, 5e-3 relative Frobenius, the bar of the layer's other
paths: one bf16 rounding of h, of the experts' rows and of y, each at most 2^-8 of the value and
2^-8 / sqrt(3) = 2.3e-3 in the mean square, the first two shared by the gated sum and the shared
expert.
"""
import dataclasses

import numpy as np
import pytest

import moe_inputs as mi
from oracle import oracle as O

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

pytestmark = pytest.mark.gpu
FMTS = ("mxfp4", "mxfp8")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    moe.lib()
    yield


def hard_values(rows, cols, seed):
    """Rows over many binades with zeros of both signs, ties of both element grids, subnormals, a
    zero block and values at the saturation edge."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    x = x.astype(np.float32)
    blk = x.reshape(-1, 32)
    for b in range(blk.shape[0]):
        kind = rng.integers(0, 10)
        if kind == 0:
            blk[b] = 0.0
            blk[b, ::3] = -0.0
        elif kind == 1:    # E2M1 grid ties and its edge, at some binade
            blk[b] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -7.5, -0.25], 32)
            blk[b] *= np.float32(2.0 ** int(rng.integers(-100, 100)))
        elif kind == 2:    # E4M3 ties: odd multiples of half a step
            blk[b] = (rng.integers(16, 32, 32) + 0.5) * rng.choice([-1, 1], 32)
            blk[b, 0] = 511.0
        elif kind == 3:    # subnormal and nearly subnormal fp32
            blk[b] = rng.standard_normal(32) * 2.0 ** -130
        elif kind == 4:
            blk[b] = rng.standard_normal(32) * 2.0 ** 125
    return x


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (37, 160), (5, 2688), (300, 288),
                                       (1021, 1856)])
def test_conversion_matches_the_encoder_bit_for_bit(fmt, dt, rows, cols):
    print(f"[gpu] quantise {fmt} {dt} {rows}x{cols}", flush=True)
    x = hard_values(rows, cols, rows * 7 + cols)
    if dt == "bf16":
        bits = mi.f32_to_bf16_bits(x)
        x = mi.bf16_bits_to_f32(bits)
        t = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    else:
        t = torch.from_numpy(x).cuda()
    codes, scales = moe.mx_quantize(t, fmt)
    ref_c, ref_s = mi.quantize_blocks_mx(x, fmt)
    assert np.array_equal(scales.cpu().numpy(), ref_s)
    assert np.array_equal(codes.cpu().numpy(), ref_c)
    want = mi.decode_blocks_mx(ref_c, ref_s, fmt).astype(np.float32)
    assert np.array_equal(moe.mx_dequantize(codes, scales).cpu().numpy(), want)
    got = moe.mx_dequantize(codes, scales, dtype=torch.bfloat16)
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))


@pytest.mark.parametrize("fmt", FMTS)
def test_blocks_that_are_not_finite_become_nan(fmt):
    x = np.ones((4, 96), dtype=np.float32)
    x[0, 5] = np.nan
    x[1, 40] = np.inf
    x[2, 95] = -np.inf
    codes, scales = moe.mx_quantize(torch.from_numpy(x).cuda(), fmt)
    bad = np.zeros((4, 3), dtype=bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert np.array_equal(scales.cpu().numpy() == 255, bad)
    for dtype in (torch.float32, torch.bfloat16):
        v = moe.mx_dequantize(codes, scales, dtype=dtype).float().cpu().numpy()
        assert np.array_equal(np.isnan(v), np.repeat(bad, 32, 1))
        assert np.all(v[~np.repeat(bad, 32, 1)] == 1.0)
    # and every output of a product that such a block enters
    w, ws = moe.mx_quantize(torch.ones(16, 96, device="cuda"), fmt)
    for m in (4, 200):
        a = codes.repeat(m // 4, 1)
        y = moe.mx_gemm(a, scales.repeat(m // 4, 1), w, ws).float().cpu().numpy()
        assert np.array_equal(np.isnan(y), np.repeat(np.tile(bad.any(1), m // 4)[:, None], 16, 1))


def test_conversion_writes_nothing_past_its_outputs():
    for fmt in FMTS:
        x = torch.randn(77, 160, device="cuda")
        n = 77 * 160 // (2 if fmt == "mxfp4" else 1)
        c, s = (torch.full((m + 64,), 171, dtype=torch.uint8, device="cuda") for m in (n, 77 * 5))
        v = torch.full((77 * 160 + 64,), 3.5, device="cuda")
        moe.mx_quantize(x, fmt, codes=c[:n].view(77, -1), scales=s[:77 * 5].view(77, 5))
        moe.mx_dequantize(c[:n].view(77, -1), s[:77 * 5].view(77, 5), out=v[:77 * 160].view(77, 160))
        assert bool((c[n:] == 171).all()) and bool((s[77 * 5:] == 171).all())
        assert bool((v[77 * 160:] == 3.5).all())
    empty = moe.mx_quantize(torch.empty(0, 64, device="cuda"))
    assert empty[0].shape == (0, 32) and moe.mx_dequantize(*empty).shape == (0, 64)


def operand(rows, cols, fmt, seed):
    """(codes, scales, values in 64 bits): random codes whose scales span 13 binades."""
    rng = np.random.default_rng(seed)
    c, s = mi.quantize_blocks_mx(rng.standard_normal((rows, cols)), fmt)
    s = (s.astype(np.int32) + rng.integers(-6, 7, s.shape)).astype(np.uint8)
    return c, s, mi.decode_blocks_mx(c, s, fmt)


def check_product(M, N, K, fa, fw, out):
    print(f"[gpu] product M={M} N={N} K={K} {fa} x {fw} -> {out}", flush=True)
    a, sa, av = operand(M, K, fa, M + K)
    w, sw, wv = operand(N, K, fw, N + K + 1)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    buf = torch.full((M * N + 256,), 7.0, dtype=dt, device="cuda")
    d = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    y = moe.mx_gemm(d(a), d(sa), d(w), d(sw), out_dtype=dt, out=buf[:M * N].view(M, N))
    got = y.double().cpu().numpy()
    assert bool((buf[M * N:] == 7.0).all())
    ref = av @ wv.T
    bound = K * 2.0 ** -23 * (np.abs(av) @ np.abs(wv).T)
    if "mxfp8" in (fa, fw):
        aa, ww = d(np.abs(av)), d(np.abs(wv))
        top = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for k in range(0, K, 8):
            top += (aa[:, None, k:k + 8] * ww[None, :, k:k + 8]).amax(-1)
        bound = bound + 7 * 2.0 ** -13 * top.cpu().numpy()
    if out == "bf16":
        bound = bound + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= bound), float((np.abs(got - ref) / bound).max())


@pytest.mark.parametrize("fa", FMTS)
@pytest.mark.parametrize("fw", FMTS)
@pytest.mark.parametrize("M,N,K", [
    (1, 16, 32), (1, 32, 64), (1, 208, 96), (2, 48, 1856), (16, 16, 2080), (17, 64, 544),
    (31, 80, 160), (33, 48, 128), (64, 208, 512), (65, 16, 4096), (128, 48, 288),
    (129, 16, 32), (130, 208, 64), (200, 400, 96), (257, 192, 544), (300, 1040, 1856),
    (513, 176, 2688)])
def test_product_against_64_bits(fa, fw, M, N, K):
    if fa == fw == "mxfp4":
        check_product(M, N, K, fa, fw, "f32")
    check_product(M, N, K, fa, fw, "bf16")


def test_empty_product():
    w, ws = moe.mx_quantize(torch.ones(16, 64, device="cuda"))
    a, sa = moe.mx_quantize(torch.ones(0, 64, device="cuda"))
    assert moe.mx_gemm(a, sa, w, ws).shape == (0, 16)


def test_quantise_and_multiply_captured_and_replayed():
    """Quantised activations through a product, eagerly on a side stream and as a graph whose
    inputs change between replays."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(48, 288, generator=g, device="cuda").bfloat16()
    w, ws = moe.mx_quantize(torch.randn(160, 288, generator=g, device="cuda"))
    c, s = moe.mx_quantize(x, "mxfp8")
    y = moe.mx_gemm(c, s, w, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cs = moe.mx_quantize(x, "mxfp8", stream=side)
    ys = moe.mx_gemm(*cs, w, ws, stream=side)
    side.synchronize()
    assert torch.equal(y, ys)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.mx_quantize(x, "mxfp8", codes=c, scales=s)
        moe.mx_gemm(c, s, w, ws, out=y)
    for i in range(4):
        x.copy_(torch.randn(48, 288, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = moe.mx_gemm(*moe.mx_quantize(x, "mxfp8"), w, ws)
        assert torch.equal(y, want), i


# ------------------------------------------------- the layer with block-scaled experts, many tokens

LAYERS = {
    "mxfp4_small": mi.LayerConfig("mxfp4_small", T=300, H=288, E=16, k=4, I=160, I_shared=128,
                                  expert_dtype="mxfp4"),
    "mxfp8_small": mi.LayerConfig("mxfp8_small", T=301, H=288, E=16, k=4, I=160,
                                  expert_dtype="mxfp8"),
    "mxfp4_one": mi.LayerConfig("mxfp4_one", T=1, H=2080, E=8, k=3, I=1184, I_shared=96,
                                expert_dtype="mxfp4"),
    "mxfp8_long": mi.LayerConfig("mxfp8_long", T=700, H=2080, E=8, k=3, I=1184, I_shared=96,
                                 expert_dtype="mxfp8"),
    # K of 9 steps, the last a quarter: workgroups that walk several tiles, of 64 and of 128 rows
    "mxfp4_walk64": mi.LayerConfig("mxfp4_walk64", T=1500, H=1056, E=64, k=3, I=1056,
                                   expert_dtype="mxfp4"),
    "mxfp8_walk64": mi.LayerConfig("mxfp8_walk64", T=1500, H=1056, E=64, k=3, I=1056,
                                   expert_dtype="mxfp8"),
    "mxfp4_walk128": mi.LayerConfig("mxfp4_walk128", T=4500, H=1056, E=8, k=3, I=1056,
                                    expert_dtype="mxfp4"),
    "mxfp8_walk128": mi.LayerConfig("mxfp8_walk128", T=4500, H=1056, E=8, k=3, I=1056,
                                    expert_dtype="mxfp8"),
    # the fewest steps of such a K and more experts than two waves' lanes
    "mxfp4_walk_wide": mi.LayerConfig("mxfp4_walk_wide", T=800, H=1024, E=200, k=8, I=1024,
                                      expert_dtype="mxfp4"),
    "latent_mxfp4": mi.LayerConfig("latent_mxfp4", T=90, H=256, E=64, k=8, I=64, latent=96,
                                   I_shared=80, expert_dtype="mxfp4"),
}


def layer_out(inp, path, given=None):
    cfg = inp["config"]
    dev = moe.to_device(inp)
    rt = moe.alloc_routing(cfg.T, cfg.E, cfg.k, "cuda")
    if given is not None:
        rt["idx"].copy_(torch.from_numpy(given[0].astype(np.int32)))
        rt["gates"].copy_(torch.from_numpy(given[1].astype(np.float32)))
    y = moe.layer_from(dev, cfg.k, path=path, routing=rt, routing_given=given is not None,
                       expert_dtype=cfg.expert_dtype)()
    torch.cuda.synchronize()
    return y.double().cpu().numpy(), {n: v.cpu().numpy() for n, v in rt.items()}


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("name", list(LAYERS))
def test_layer_with_block_scaled_experts_on_tiles(name):
    cfg = LAYERS[name]
    inp = mi.make_layer(cfg, seed=2)
    y, rt = layer_out(inp, "grouped_mx")
    t = np.arange(0, cfg.T, 1 + cfg.T // 100)
    t = np.union1d(t, np.arange(cfg.T - 3, cfg.T).clip(0))      # the oracle is one thread
    g = O.gates_for(O.logits(inp, t), rt["idx"][t])
    ref = O.forward_tokens(inp, rt["idx"][t], g, t, True)
    print(f"[gpu] grouped_mx {name}: {rel(y[t], ref):.2e}", flush=True)
    assert rel(y[t], ref) <= 5e-3
    # the decode path on the same selection: the same quantised rows, other summation orders and
    # one more rounding of the experts' rows here
    z, _ = layer_out(inp, "stream", given=(rt["idx"], rt["gates"]))
    assert rel(y, z) <= 5e-3


def test_experts_without_rows_and_with_all_rows():
    """Given routing: one expert takes every token, most take none."""
    cfg = dataclasses.replace(LAYERS["mxfp4_small"], T=261, k=2)
    inp = mi.make_layer(cfg, seed=4)
    idx = np.empty((cfg.T, 2), dtype=np.int32)
    idx[:, 0] = 5
    idx[:, 1] = np.where(np.arange(cfg.T) % 130 == 0, 15, 9)
    gates = np.full((cfg.T, 2), 0.5, dtype=np.float32)
    y, rt = layer_out(inp, "grouped_mx", given=(idx, gates))
    assert sorted(set(np.nonzero(rt["counts"])[0])) == [5, 9, 15]
    ref = O.forward_tokens(inp, idx, gates.astype(np.float64), np.arange(cfg.T), True)
    assert rel(y, ref) <= 5e-3


def test_weights_quantised_on_the_gpu_through_the_layer_and_the_product():
    """The operators together: fp32 expert weights converted on the GPU, one layer call on each
    path over them, and an expert's up projection as a plain product of quantised rows."""
    cfg = mi.LayerConfig("pipe", T=160, H=288, E=8, k=2, I=160, I_shared=0, expert_dtype="mxfp4")
    inp = mi.make_layer(cfg, seed=6)
    rng = np.random.default_rng(6)
    up = rng.standard_normal((8, 160, 288)).astype(np.float32) / np.float32(17.0)
    down = rng.standard_normal((8, 288, 160)).astype(np.float32) / np.float32(12.6)
    dev = moe.to_device(inp)
    for n, v in (("up", up), ("down", down)):
        dev["W_" + n], dev["s_" + n] = moe.mx_quantize(torch.from_numpy(v).cuda(), "mxfp4")
        inp["W_" + n], inp["s_" + n] = mi.quantize_blocks_mx(v, "mxfp4")
    rt = moe.alloc_routing(cfg.T, cfg.E, cfg.k, "cuda")
    y = moe.layer_from(dev, cfg.k, path="grouped_mx", routing=rt)().double().cpu().numpy()
    idx = rt["idx"].cpu().numpy()
    ref = O.forward_tokens(inp, idx, O.gates_for(O.logits(inp), idx), np.arange(cfg.T), True)
    assert rel(y, ref) <= 5e-3
    xq = moe.mx_quantize(dev["x"], "mxfp8")
    a = moe.mx_gemm(*xq, dev["W_up"][3], dev["s_up"][3])
    xv = moe.mx_dequantize(*xq).double()
    wv = moe.mx_dequantize(dev["W_up"][3], dev["s_up"][3]).double()
    # a group of eight's largest product is at most the sum of its products
    bound = (288 * 2.0 ** -23 + 7 * 2.0 ** -13) * (xv.abs() @ wv.abs().t()) \
        + 2.0 ** -8 * (xv @ wv.t()).abs()
    assert bool(((a.double() - xv @ wv.t()).abs() <= bound).all())


# ------------------------------------------------------------------- other ways and sizes to call

def test_layer_on_tiles_captured_on_another_stream_and_without_a_workspace():
    cfg = mi.LayerConfig("cap", T=600, H=1056, E=8, k=3, I=1056, I_shared=96, expert_dtype="mxfp4")
    dev = moe.to_device(mi.make_layer(cfg, seed=9))
    layer, eager = (moe.layer_from(dev, 3, path="grouped_mx", expert_dtype="mxfp4") for _ in range(2))
    want = eager().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer(s)
    s.synchronize()
    assert torch.equal(layer.y, want)
    static = moe.layer_from(dev, 3, path="grouped_mx", expert_dtype="mxfp4", no_alloc=True)
    assert torch.equal(static(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    g = torch.Generator(device="cuda").manual_seed(9)
    for i in range(4):
        dev["x"].copy_(torch.randn(600, 1056, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        eager()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, eager.y), i


@pytest.mark.parametrize("fmt", FMTS)
def test_conversion_past_32_bit_offsets(fmt):
    """More than 2^31 elements: the last rows as when they are converted alone."""
    rows, cols = (1 << 31) // 2048 + 3, 2048
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-5:] = torch.randn(5, cols, generator=g, device="cuda")
    codes, scales = moe.mx_quantize(x, fmt)
    c, s = moe.mx_quantize(x[-5:], fmt)
    assert torch.equal(codes[-5:], c) and torch.equal(scales[-5:], s)
    assert not bool(scales[:-5].any()) and not bool(codes[:5].any())
    x.fill_(1.0)
    moe.mx_dequantize(codes, scales, dtype=torch.bfloat16, out=x)
    assert torch.equal(x[-5:], moe.mx_dequantize(c, s, dtype=torch.bfloat16))
    assert not bool(x[:-5].any())


@pytest.mark.parametrize("M,N", [(65535, 16), (1, 65520), (100, 65520)])
def test_product_of_operands_near_2_gib(M, N):
    """The bound of the accumulation as at the head of the file, on the last rows and columns."""
    K = 32768
    g = torch.Generator(device="cuda").manual_seed(2)

    def operand(rows):
        c, s = moe.mx_quantize(torch.randn(min(rows, 64), K, generator=g, device="cuda"), "mxfp8")
        n = -(-rows // c.shape[0])
        c, s = c.repeat(n, 1)[:rows], s.repeat(n, 1)[:rows]
        tail = moe.mx_quantize(torch.randn(min(rows, 48), K, generator=g, device="cuda"), "mxfp8")
        c[-tail[0].shape[0]:], s[-tail[0].shape[0]:] = tail
        return c, s

    a, w = operand(M), operand(N)
    out = moe.mx_gemm(*a, *w)[-48:, -48:].double()
    x, v = (moe.mx_dequantize(c[-48:], s[-48:]).double() for c, s in (a, w))
    exact = x @ v.t()
    bound = (K * 2.0 ** -23 + 7 * 2.0 ** -13) * (x.abs() @ v.abs().t()) + 2.0 ** -8 * exact.abs()
    assert bool(((out - exact).abs() <= bound).all())
    assert float((out - exact).norm() / exact.norm()) <= 5e-3


def test_experts_rows_near_2_gib():
    """h of 2.1 GB in e4m3: the last tokens as in a call of their own with the same selection."""
    cfg = mi.LayerConfig("long", T=131072, H=32, E=8, k=8, I=2016, expert_dtype="mxfp4")
    dev = moe.to_device(mi.make_layer(cfg, seed=3))
    rt = moe.alloc_routing(cfg.T, cfg.E, cfg.k, "cuda")
    y = moe.layer_from(dev, 8, path="grouped_mx", routing=rt, expert_dtype="mxfp4")()[-70:]
    given = {n: rt[n][-70:].contiguous() for n in ("idx", "gates")}
    z = moe.layer_from(dict(dev, x=dev["x"][-70:].contiguous()), 8, path="grouped_mx",
                       routing=given, routing_given=True, expert_dtype="mxfp4")()
    y, z = y.double().cpu().numpy(), z.double().cpu().numpy()
    assert np.abs(z).max() > 0 and rel(y, z) <= 5e-3
