"""GPU tests of the few-token layer against the double-precision oracle.

Bars: logits within one rounding to fp32 (2^-24) of the oracle's; the selection that the oracle
makes from those logits, exactly; y within 5e-3 relative Frobenius, the bar of the layer's other
paths (h is rounded to bf16, 2^-8 of the value at most and 2^-8 / sqrt(3) = 2.3e-3 in the mean
square, before it is summed over, y once more), for 8- and 4-bit experts against the oracle that
rounds the expert rows to e4m3 as the layer does.
"""
import dataclasses

import numpy as np
import pytest

import moe_inputs as mi
from oracle import oracle as O

torch = pytest.importorskip("torch")
import sparse_moe_layer_05_amd as moe  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    moe.lib()
    yield


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def run(inp, path="few", given=None, dev=None):
    cfg = inp["config"]
    dev = dev if dev is not None else moe.to_device(inp)
    rt = moe.alloc_routing(cfg.T, cfg.E, cfg.k, "cuda")
    if given is not None:
        rt["idx"].copy_(torch.from_numpy(given[0].astype(np.int32)))
        rt["gates"].copy_(torch.from_numpy(given[1].astype(np.float32)))
    buf = torch.full((cfg.T + 3, cfg.H), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.layer_from(dev, cfg.k, path=path, routing=rt, routing_given=given is not None,
                   out=buf[:cfg.T], expert_dtype=cfg.expert_dtype)()
    torch.cuda.synchronize()
    assert bool((buf[cfg.T:] == 9.0).all())
    return buf[:cfg.T].double().cpu().numpy(), {n: v.cpu().numpy() for n, v in rt.items()}


def check(cfg, seed=1):
    print(f"[gpu] few {cfg.name} T={cfg.T} {cfg.expert_dtype}", flush=True)
    inp = mi.make_layer(cfg, seed=seed)
    y, rt = run(inp)
    z = O.logits(inp)
    x64 = O.bf16_to_f64(inp["x"])
    slack = 2.0 ** -24 * np.abs(z) + cfg.H * 2.0 ** -52 * (np.abs(x64) @ np.abs(O.bf16_to_f64(inp["W_r"])).T)
    assert np.all(np.abs(rt["logits"] - z) <= slack)
    idx, _, _ = O.route_f32(rt["logits"], inp["b"], cfg.k)
    assert np.array_equal(idx, rt["idx"])
    g = O.gates_for(z, idx)
    # a score is off by half a step of fp32 and what the logit's rounding moves it by; so is their
    # sum (k terms, k additions) and the quotient
    assert np.all(np.abs(rt["gates"] - g) <= (cfg.k + 8) * 2.0 ** -23 * g)
    for a, b in zip(O.dispatch(idx, cfg.E), ("counts", "offsets", "perm", "pos")):
        assert np.array_equal(a, rt[b]), b
    ref = O.forward_tokens(inp, idx, g, np.arange(cfg.T), cfg.expert_dtype != "bf16")
    err = rel(y, ref)
    print(f"[gpu]   {err:.2e}", flush=True)
    assert err <= 5e-3
    return inp, y, rt


def L(**kw):
    base = dict(name="few", T=3, H=288, E=16, k=4, I=160, I_shared=128)
    base.update(kw)
    return mi.LayerConfig(**base)


@pytest.mark.parametrize("w", ["bf16", "e4m3", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("kw", [
    dict(T=1), dict(T=2, I_shared=0), dict(T=5), dict(T=16), dict(T=15, E=24, k=5),
    dict(T=4, E=8, k=8),                                  # every expert for every token
    dict(T=3, E=1, k=1), dict(T=7, E=200, k=3), dict(T=9, E=1024, k=64, I=32, H=64),
    dict(T=6, H=2080, I=1184, E=8, k=3), dict(T=16, H=4096, I=64, E=4, k=2, I_shared=0),
    dict(T=1, H=32, I=32, E=3, k=2, I_shared=16), dict(T=2, I_shared=2064),
    dict(T=3, latent=96, I_shared=0), dict(T=16, latent=64, H=256, E=64, k=8),
    dict(T=1, latent=1024, H=512, E=40, k=12, I=512)])
def test_few_tokens_against_the_oracle(w, kw):
    check(L(expert_dtype=w, **kw))


@pytest.mark.parametrize("w,kw", [("bf16", dict(H=272, I=144, I_shared=208)),
                                  ("bf16", dict(H=16, I=16, I_shared=16)),
                                  ("e4m3", dict(H=272, I=144)), ("e4m3", dict(H=16, I=16, E=4)),
                                  ("bf16", dict(H=128, latent=48, I=80))])
def test_widths_that_end_inside_a_step(w, kw):
    for T in (1, 16):
        check(L(expert_dtype=w, T=T, **kw))


@pytest.mark.parametrize("name", ["nano_decode_bf16", "nano_fp8_decode", "nano_mxfp4_decode",
                                  "latent_decode_k22_bf16"])
def test_layer_widths_against_the_decode_path(name):
    """The benchmark's widths with 1 and 16 tokens: the same selection through the decode path,
    whose sums run in another order."""
    for T in (1, 16):
        cfg = mi.CONFIGS[name].with_T(T)
        inp = mi.make_layer(cfg, seed=3)
        dev = moe.to_device(inp)
        y, rt = run(inp, dev=dev)
        ys, _ = run(inp, "stream", given=(rt["idx"], rt["gates"]), dev=dev)
        print(f"[gpu] {name} T={T}: few against stream {rel(y, ys):.2e}", flush=True)
        assert rel(y, ys) <= 5e-3


def test_given_routing_with_dropped_pairs():
    """Experts out of range, repeated experts, a token with nothing left."""
    for w in ("bf16", "mxfp4"):
        cfg = L(T=5, k=3, expert_dtype=w)
        inp = mi.make_layer(cfg, seed=8)
        idx = np.array([[3, 3, 7], [-1, 16, 1 << 30], [0, 15, 0], [2, 1, 0], [9, 9, 9]], np.int32)
        gates = np.linspace(0.1, 0.9, 15).reshape(5, 3).astype(np.float32)
        y, rt = run(inp, given=(idx, gates))
        keep = np.array([[1, 0, 1], [0, 0, 0], [1, 1, 0], [1, 1, 1], [1, 0, 0]], bool)
        ref = O.forward_tokens(inp, np.where(keep, idx, 0), np.where(keep, gates, 0.0).astype(np.float64),
                               np.arange(5), w != "bf16")
        assert rel(y, ref) <= 5e-3
        assert np.array_equal(rt["idx"], idx)           # given: read, not written
        assert rt["counts"].sum() == keep.sum()
        # token 1 has the shared expert alone; without one it gets zeros
        bare = dataclasses.replace(cfg, I_shared=0)
        y, _ = run(mi.make_layer(bare, seed=8), given=(idx, gates))
        assert np.all(y[1] == 0.0) and np.all(np.abs(y[[0, 2, 3, 4]]).max(1) > 0)


@pytest.mark.parametrize("w", ["bf16", "e4m3", "mxfp4"])
def test_a_nan_token_stays_in_its_row(w):
    cfg = L(T=6, expert_dtype=w)
    inp = mi.make_layer(cfg, seed=5)
    y, _ = run(inp)
    bad = dict(inp, x=inp["x"].copy())
    bad["x"][2, 17] = 0x7FC0
    z, rt = run(bad)
    others = [0, 1, 3, 4, 5]
    assert np.array_equal(z[others], y[others])
    assert np.isnan(z[2]).all()
    assert np.all((rt["idx"] >= 0) & (rt["idx"] < cfg.E))


def test_no_tokens():
    dev = moe.to_device(mi.make_layer(L(T=1), seed=0))
    dev["x"] = dev["x"][:0]
    assert moe.layer_from(dev, 4, path="few")().shape == (0, 288)


def test_two_streams_and_a_replayed_graph():
    """Calls of two layers at once on two streams, and a captured decode step of both (the second
    reads the first's output) replayed with new tokens between eager calls."""
    a, b = (moe.to_device(mi.make_layer(L(T=4, expert_dtype=w), seed=i))
            for i, w in ((1, "mxfp4"), (2, "bf16")))
    la = moe.layer_from(a, 4, path="few", expert_dtype="mxfp4")
    b["x"] = la.y
    lb = moe.layer_from(b, 4, path="few")
    ea = moe.layer_from(a, 4, path="few", expert_dtype="mxfp4")
    eb = moe.layer_from(dict(b, x=ea.y), 4, path="few")
    other = moe.layer_from(moe.to_device(mi.make_layer(L(T=16), seed=3)), 4, path="few")
    want_other = other().clone()
    la(), lb()
    torch.cuda.synchronize()
    want = lb.y.clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        la(s1), lb(s1), other(s2)
    torch.cuda.synchronize()
    assert torch.equal(lb.y, want) and torch.equal(other.y, want_other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la(), lb()
    g = torch.Generator(device="cuda").manual_seed(4)
    for i in range(5):
        a["x"].copy_(torch.randn(4, 288, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ea(), eb()
        torch.cuda.synchronize()
        assert torch.equal(la.y, ea.y) and torch.equal(lb.y, eb.y), i
        other()


def test_weights_quantised_on_the_gpu_serve_prefill_and_decode():
    """The operators as they are used together: experts' weights converted once on the GPU, a
    prompt through the tiles, its last tokens again through the few-token layer."""
    cfg = L(T=200, I_shared=128, expert_dtype="mxfp8")
    inp = mi.make_layer(cfg, seed=11)
    rng = np.random.default_rng(12)
    dev = moe.to_device(inp)
    for n, shape in (("up", (16, 160, 288)), ("down", (16, 288, 160))):
        v = (rng.standard_normal(shape) / np.sqrt(shape[2])).astype(np.float32)
        dev["W_" + n], dev["s_" + n] = moe.mx_quantize(torch.from_numpy(v).cuda(), "mxfp8")
        inp["W_" + n], inp["s_" + n] = mi.quantize_blocks_mx(v, "mxfp8")
    rt = moe.alloc_routing(cfg.T, cfg.E, cfg.k, "cuda")
    y = moe.layer_from(dev, cfg.k, path="grouped_mx", routing=rt)()[-9:].double().cpu().numpy()
    tail = dict(dev, x=dev["x"][-9:].contiguous())
    given = {n: rt[n][-9:].contiguous() for n in ("idx", "gates")}
    z = moe.layer_from(tail, cfg.k, path="few", routing=given, routing_given=True)()
    z = z.double().cpu().numpy()
    idx = rt["idx"].cpu().numpy()
    ref = O.forward_tokens(inp, idx, O.gates_for(O.logits(inp), idx), np.arange(cfg.T), True)[-9:]
    assert rel(y, ref) <= 5e-3 and rel(z, ref) <= 5e-3
