"""GPU tests of NaN through the layer: a NaN in a token's row, or in a block of an expert's weights
(E8M0 scale code 255, which the conversion gives a block that holds a NaN or an infinity), makes
NaN of exactly the outputs that it enters, on every path. Routing is given, so that the NaN
reaches y through the experts and not through the gates; outputs that it does not enter are those
of the clean call bit for bit (rows do not meet each other in any sum)."""
import numpy as np
import pytest

import moe_inputs as mi

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

pytestmark = pytest.mark.gpu

PATHS = [("f32", "grouped"), ("bf16", "grouped"), ("bf16", "stream"), ("bf16", "few"),
         ("e4m3", "grouped"), ("e4m3", "stream"), ("e4m3", "few"),
         ("mxfp4", "stream"), ("mxfp4", "grouped_mx"), ("mxfp4", "few"),
         ("mxfp8", "stream"), ("mxfp8", "grouped_mx"), ("mxfp8", "few")]
MX = [p for p in PATHS if p[0] in ("mxfp4", "mxfp8")]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    moe.lib()
    yield


def setup(w, T=11, H=1056, I=1056, **kw):
    """A layer whose K spans nine steps of the block-scaled tiles, and a selection in which token
    t takes experts t % E and (t + 3) % E."""
    cfg = mi.LayerConfig("nan", T=T, H=H, E=8, k=2, I=I, act_dtype="f32" if w == "f32" else "bf16",
                         expert_dtype=w, **kw)
    dev = moe.to_device(mi.make_layer(cfg, seed=5))
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    rt = dict(idx=torch.stack((t % 8, (t + 3) % 8), 1).contiguous(),
              gates=torch.full((T, 2), 0.5, device="cuda"))
    return cfg, dev, rt


def out(cfg, dev, rt, path):
    print(f"[gpu] {cfg.expert_dtype} {path} H={cfg.H} latent={cfg.latent} shared={cfg.I_shared}",
          flush=True)
    y = moe.layer_from(dev, cfg.k, path=path, routing=rt, routing_given=True,
                       expert_dtype=cfg.expert_dtype)()
    torch.cuda.synchronize()
    return y


def only(bad, clean, where):
    """`bad` is NaN where `where` says so and `clean` everywhere else."""
    assert bool(torch.isfinite(clean).all())
    assert torch.equal(torch.isnan(bad), where)
    assert torch.equal(bad[~where], clean[~where])


@pytest.mark.parametrize("w,path", PATHS)
@pytest.mark.parametrize("kw", [dict(), dict(H=288, I=160, I_shared=128), dict(H=288, I=96, latent=160),
                                dict(H=288, I=96, latent=160, I_shared=64)])
def test_a_nan_token_with_given_routing_stays_in_its_row(w, path, kw):
    cfg, dev, rt = setup(w, **kw)
    clean = out(cfg, dev, rt, path).clone()
    dev["x"][4, 17] = float("nan")
    bad = out(cfg, dev, rt, path)
    where = torch.zeros_like(bad, dtype=torch.bool)
    where[4] = True
    only(bad, clean, where)


@pytest.mark.parametrize("w,path", MX)
@pytest.mark.parametrize("kw", [dict(), dict(H=288, I=160, I_shared=128),
                                dict(H=288, I=96, latent=160)])
def test_a_nan_block_of_an_experts_weights(w, path, kw):
    cfg, dev, rt = setup(w, **kw)
    clean = out(cfg, dev, rt, path).clone()
    meets = (rt["idx"] == 6).any(1)
    nb = dev["s_up"].shape[-1]
    for blk in (0, nb - 1):               # W_up: every product with the expert's h
        keep = dev["s_up"][6, 37, blk].clone()
        dev["s_up"][6, 37, blk] = 255
        only(out(cfg, dev, rt, path), clean, meets[:, None].expand_as(clean))
        dev["s_up"][6, 37, blk] = keep
    for blk in (0, dev["s_down"].shape[-1] - 1):    # W_down: one column of the expert's output
        keep = dev["s_down"][6, 37, blk].clone()
        dev["s_down"][6, 37, blk] = 255
        where = meets[:, None].expand_as(clean).clone()
        if not cfg.latent:
            where[:] = False
            where[meets, 37] = True
        only(out(cfg, dev, rt, path), clean, where)
        dev["s_down"][6, 37, blk] = keep
    assert torch.equal(out(cfg, dev, rt, path), clean)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_an_infinite_master_weight_through_conversion_and_layer(fmt):
    """The operators together: fp32 masters with one infinity, converted and used by both paths."""
    cfg, dev, rt = setup(fmt, H=288, I=160)
    up = torch.randn(8, 160, 288, generator=torch.Generator("cuda").manual_seed(1), device="cuda") / 17
    up[2, 5, 100] = float("inf")
    dev["W_up"], dev["s_up"] = moe.mx_quantize(up, fmt)
    assert int((dev["s_up"] == 255).sum()) == 1
    meets = (rt["idx"] == 2).any(1)
    for path in ("few", "grouped_mx"):
        y = out(cfg, dev, rt, path)
        assert torch.equal(torch.isnan(y), meets[:, None].expand_as(y))


@pytest.mark.parametrize("w,path", MX)
def test_the_smallest_block_scales(w, path):
    """Scale code 0 (2^-127) throughout W_up, met by tokens large enough that h is of order one: the
    same values as with codes and tokens moved by a power of two, up to the elements that bf16
    subnormals (2^-133 and coarser) cannot hold beside a block's largest: E2M1 none, E4M3 those below
    2^-134 / 2^-127 / 448 = 2^-15.8 of it, far inside a bf16 step of u, which 5e-3 covers."""
    cfg, dev, rt = setup(w, H=288, I=160)
    dev["x"] = dev["x"].sign()
    dev["s_up"] = torch.full_like(dev["s_up"], 127 - 10)
    want = out(cfg, dev, rt, path).double()
    dev["s_up"] = torch.zeros_like(dev["s_up"])
    dev["x"] = dev["x"] * 2.0 ** 117
    got = out(cfg, dev, rt, path).double()
    assert float(want.abs().max()) > 0
    assert float((got - want).norm() / want.norm()) <= 5e-3


@pytest.mark.parametrize("w,path", PATHS)
@pytest.mark.parametrize("kw", [dict(H=288, I=160, I_shared=128), dict(H=288, I=96, latent=160)])
@pytest.mark.parametrize("bits", [0x7FFFFFFF, -1, 0x7F800001])
def test_a_nan_gate_of_any_payload_reaches_its_token(w, path, kw, bits):
    """Memory of all ones is a NaN whose rounding to bf16 must not carry into the sign."""
    cfg, dev, rt = setup(w, **kw)
    clean = out(cfg, dev, rt, path).clone()
    rt["gates"].view(torch.int32)[7, 1] = bits
    bad = out(cfg, dev, rt, path)
    where = torch.zeros_like(bad, dtype=torch.bool)
    where[7] = True
    only(bad, clean, where)


@pytest.mark.parametrize("path", ["few", "stream", "grouped"])
@pytest.mark.parametrize("kw", [dict(), dict(I_shared=128), dict(H=8192, T=16, I=48),
                                dict(H=272, I=144), dict(H=2080, I=160, I_shared=16)])
@pytest.mark.parametrize("at", [0, 9, -1])
def test_an_infinity_that_relu_takes(path, kw, at):
    """x holds one infinity and every weight that meets it is negative: u is -infinity, h and y are 0.
    Nothing else may meet the infinity, as the padding of a row whose width ends inside a step."""
    cfg, dev, rt = setup("bf16", **{**dict(T=3, H=288, I=160), **kw})
    dev["x"][1] = 0.0
    dev["x"][1, at] = float("inf")
    dev["W_up"][:, :, at] = -1.0
    if cfg.I_shared:
        dev["Ws_up"][:, at] = -1.0
    y = out(cfg, dev, rt, path)
    assert bool((y[1] == 0).all())
    assert bool(torch.isfinite(y).all())


@pytest.mark.parametrize("path", ["few", "stream", "grouped"])
@pytest.mark.parametrize("kw,value", [
    (dict(), float("inf")), (dict(), 1e25), (dict(), 2.0 ** 65),
    (dict(latent=160), 1e25), (dict(latent=160), 2.0 ** 65),
    (dict(I_shared=128), float("inf")), (dict(I_shared=128), 1e25)])
def test_an_infinite_h_stays_infinite(path, kw, value):
    """One element of h is infinite (2^65 squared is past fp32), the others are zero: every output is
    infinite with the sign of its weight, not NaN, also where h or z is kept as a pair of bf16. bf16
    weights, whose rows are not rescaled."""
    cfg, dev, rt = setup("bf16", T=3, H=288, I=160, **kw)
    g = torch.Generator(device="cuda").manual_seed(3)

    def up(rows, cols):      # row 7 alone is positive where x is not zero
        w = torch.zeros(rows, cols, device="cuda")
        w[:, 9] = -1.0
        w[7, 9] = 1.0
        return w.bfloat16()

    def signed(*shape):      # no zeros: zero times infinity is NaN
        w = torch.rand(shape, generator=g, device="cuda") + 0.1
        return (w * (torch.rand(shape, generator=g, device="cuda") - 0.5).sign()).bfloat16()

    dev["x"].zero_()
    dev["x"][1, 9] = value
    if cfg.I_shared:         # through the shared expert; the routed ones give zero
        dev["W_up"].fill_(-1.0)
        dev["Ws_up"] = up(128, 288)
        dev["Ws_down"] = signed(288, 128)
        sign = dev["Ws_down"][:, 7].sign()
    elif cfg.latent:         # u = x's first columns, z of one sign, W_out of one sign a row
        dev["W_in"] = torch.eye(160, 288, device="cuda").bfloat16()
        dev["W_up"][:] = up(160, 160)
        dev["W_down"][:] = signed(1, 160, 160).abs()
        dev["W_out"] = signed(288, 1).expand(288, 160).contiguous()
        sign = dev["W_out"][:, 0].sign()
    else:
        dev["W_up"][:] = up(160, 288)
        dev["W_down"][:] = signed(1, 288, 160)
        sign = dev["W_down"][0, :, 7].sign()
    y = out(cfg, dev, rt, path)
    assert bool((y[1].float() == sign.float() * float("inf")).all())
    assert bool(torch.isfinite(y[[0, 2]]).all())
