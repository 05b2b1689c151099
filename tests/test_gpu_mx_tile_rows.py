"""GPU tests of block-scaled experts on every tile: 64 and 128 rows, a workgroup per tile (K under
eight steps of 128) and workgroups that walk several, for both formats, at sizes on each side of the
rule that chooses. Bars as for the other sizes: 5e-3 relative Frobenius against the double-precision
oracle on sampled tokens and against the decode path on all (the roundings are the same; one row of h
in some hundred may take another e4m3 scale, 4% of it)."""
import numpy as np
import pytest

import moe_inputs as mi
from oracle import oracle as O

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("kw", [
    dict(T=1000, H=1056, E=64, k=3, I=1056),       # 47 rows an expert, walked, K of 9 steps
    dict(T=1800, H=1056, E=64, k=3, I=1056),       # 84
    dict(T=3000, H=1056, E=64, k=3, I=1056),       # 141
    dict(T=700, H=1056, E=8, k=3, I=1056),         # 263, fewer tiles than CUs
    dict(T=1100, H=288, E=64, k=3, I=160),         # a tile per workgroup: 52
    dict(T=13000, H=288, E=8, k=3, I=160),         # and 4875
    dict(T=2500, H=288, E=24, k=4, I=544, latent=416)])
def test_tiles_of_both_heights(fmt, kw):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    cfg = mi.LayerConfig("tiles", expert_dtype=fmt, **kw)
    print(f"[gpu] tiles {cfg}", flush=True)
    inp = mi.make_layer(cfg, seed=6)
    dev = moe.to_device(inp)
    rt = moe.alloc_routing(cfg.T, cfg.E, cfg.k, "cuda")
    y = moe.layer_from(dev, cfg.k, path="grouped_mx", routing=rt, expert_dtype=fmt)()
    z = moe.layer_from(dev, cfg.k, path="stream", routing=rt, routing_given=True, expert_dtype=fmt)()
    y, z = y.double().cpu().numpy(), z.double().cpu().numpy()
    assert np.linalg.norm(y - z) <= 5e-3 * np.linalg.norm(z)
    t = np.arange(0, cfg.T, 1 + cfg.T // 40)
    idx = rt["idx"].cpu().numpy()
    ref = O.forward_tokens(inp, idx[t], O.gates_for(O.logits(inp, t), idx[t]), t, True)
    assert np.linalg.norm(y[t] - ref) <= 5e-3 * np.linalg.norm(ref)
