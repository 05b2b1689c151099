"""GPU test of the few-token layer's column blocks that are cut into parts: calls that follow each
other in one workspace without a wait, each with other tokens, give what the same tokens give in a
workspace of their own, bit for bit (the part that ends last adds the parts in a fixed order)."""
import pytest

import moe_inputs as mi

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("w", ["bf16", "e4m3", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("kw", [dict(H=288, I=160, I_shared=128),          # 18 blocks in 8 parts
                                dict(H=2080, I=1184),                      # 130 in 3
                                dict(H=288, I=96, latent=160, I_shared=64)])
def test_calls_in_one_workspace_join_their_own_parts(w, kw):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    print(f"[gpu] join {w} {kw}", flush=True)
    cfg = mi.LayerConfig("join", T=5, E=8, k=3, expert_dtype=w, **kw)
    dev = moe.to_device(mi.make_layer(cfg, seed=2))
    layer = moe.layer_from(dev, 3, path="few", expert_dtype=w)
    g = torch.Generator(device="cuda").manual_seed(7)
    xs = torch.randn(40, 5, cfg.H, generator=g, device="cuda").bfloat16()
    got = []
    for x in xs:
        dev["x"].copy_(x)
        got.append(layer().clone())
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        alone = moe.layer_from(dict(dev, x=x.contiguous()), 3, path="few", expert_dtype=w)
        want = alone()
        torch.cuda.synchronize()
        assert torch.equal(got[i], want), i
