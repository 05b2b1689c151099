"""GPU tests of block-scaled experts on tiles with given routing that drops pairs: experts out of
range, an expert named twice by a token (its first pair counts), tokens with nothing left, and calls
in which every pair is dropped; dropped pairs carry NaN gates. Bar: 5e-3 relative Frobenius against the oracle over the pairs that
are kept, as for whole routing; tokens without any pair have the shared expert alone, or zeros."""
import numpy as np
import pytest

import moe_inputs as mi
from oracle import oracle as O

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("kw", [dict(H=288, I=160), dict(H=1056, I=288, I_shared=96),
                                dict(H=288, I=96, latent=160), dict(H=288, I=96, latent=160, I_shared=64)])
@pytest.mark.parametrize("every", [False, True])
def test_dropped_pairs(fmt, kw, every):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    cfg = mi.LayerConfig("drop", T=100, E=8, k=3, expert_dtype=fmt, **kw)
    print(f"[gpu] dropped {cfg} {every}", flush=True)
    inp = mi.make_layer(cfg, seed=8)
    rng = np.random.default_rng(8)
    idx = np.stack([rng.permutation(8)[:3] for _ in range(cfg.T)]).astype(np.int32)
    idx[::7, 1] = -1
    idx[1::7, 2] = 1 << 30
    idx[2::7, 2] = idx[2::7, 0]
    idx[3::7] = 8
    if every:
        idx[:] = np.array([-1, 8, 2000], np.int32)
    gates = rng.uniform(0.1, 0.9, idx.shape).astype(np.float32)
    keep = (idx >= 0) & (idx < 8)
    for j in range(1, 3):
        keep[:, j] &= ~(idx[:, :j] == idx[:, j:j + 1]).any(1)
    gates[~keep] = np.nan       # a dropped pair's gate is not looked at
    dev = moe.to_device(inp)
    rt = dict(idx=torch.from_numpy(idx).cuda(), gates=torch.from_numpy(gates).cuda(),
              counts=torch.empty(8, dtype=torch.int32, device="cuda"))
    y = moe.layer_from(dev, 3, path="grouped_mx", routing=rt, routing_given=True, expert_dtype=fmt)()
    y = y.double().cpu().numpy()
    assert int(rt["counts"].sum()) == keep.sum()
    ref = O.forward_tokens(inp, np.where(keep, idx, 0), np.where(keep, gates, 0).astype(np.float64),
                           np.arange(cfg.T), True)
    assert np.isfinite(y).all()
    assert np.linalg.norm(y - ref) <= 5e-3 * np.linalg.norm(ref)
    if not cfg.I_shared:
        assert np.all(y[~keep.any(1)] == 0.0)
