"""The operators around the layer as they are used together: a block around the layer, a training
step of it, and a block whose experts run outside the layer."""
import numpy as np
import pytest
import torch

import block_oracle as O
import moe_inputs as mi
import sparse_moe_layer_05_amd as moe
from oracle import oracle

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def weights(dev):
    return dict(W_r=dev["W_r"], b=dev["b"], W_up=dev["W_up"], W_down=dev["W_down"],
                Ws_up=dev.get("Ws_up"), Ws_down=dev.get("Ws_down"), s_up=dev.get("s_up"),
                s_down=dev.get("s_down"), W_in=dev.get("W_in"), W_out=dev.get("W_out"))


CONFIGS = [
    (mi.LayerConfig("bf16", T=33, H=272, E=16, k=4, I=144, I_shared=208), "auto"),
    (mi.LayerConfig("bf16", T=300, H=272, E=16, k=4, I=144, I_shared=208), "grouped"),
    (mi.LayerConfig("few", T=1, H=272, E=16, k=4, I=144, I_shared=208), "few"),
    (mi.LayerConfig("mx", T=7, H=288, E=8, k=2, I=160, expert_dtype="mxfp4"), "stream"),
    (mi.LayerConfig("latent", T=40, H=256, E=32, k=6, I=64, latent=64), "auto"),
    (mi.LayerConfig("f32", T=20, H=256, E=16, k=2, I=128, act_dtype="f32", expert_dtype="f32"), "auto"),
]


@pytest.mark.parametrize("cfg,path", CONFIGS, ids=lambda v: getattr(v, "name", v))
def test_block_is_its_parts(cfg, path):
    dev = moe.to_device(mi.make_layer(cfg, seed=3))
    x, k, wts = dev["x"], cfg.k, weights(dev)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = [(torch.randn(cfg.H, generator=g, device="cuda") * 0.1 + 1).to(x.dtype) for _ in range(3)]
    gate = torch.randn(cfg.T, generator=g, device="cuda")
    block = moe.Block(x, k=k, path=path, w_in=w[0], w_out=w[1], gate=gate, scale=0.5, w_next=w[2],
                      expert_dtype=cfg.expert_dtype, **wts)
    y = block().clone()
    h = moe.block_norm(x, w[0])
    f = moe.Layer(h, k=k, path=path, expert_dtype=cfg.expert_dtype, **wts)()
    want, want_h = moe.block_residual(x, f, w=w[1], gate=gate, scale=0.5, w_next=w[2])
    assert torch.equal(y, want) and torch.equal(block.h_next, want_h)
    ref, mag = O.residual(O.f64(x), O.f64(f), O.f64(w[1]), True, O.f64(gate), "sigmoid", 0.5, EPS)
    O.check(y, ref, x.dtype, mag, 64, "y")
    # the next block takes y and its norm as they are; the block alone on another stream; captured
    after = moe.Block(block.y, k=k, path=path, h=block.h_next, expert_dtype=cfg.expert_dtype, **wts)
    y2 = after().clone()
    f2 = moe.Layer(want_h, k=k, path=path, expert_dtype=cfg.expert_dtype, **wts)()
    assert torch.equal(y2, moe.block_residual(want, f2)[0])
    side = torch.cuda.Stream()
    block.y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    block(side)
    side.synchronize()
    assert torch.equal(block.y, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
        after()
    for turn in range(3):
        block.y.zero_()
        after.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(block.y, y) and torch.equal(after.y, y2), turn


def test_training_step_of_a_block():
    """norm -> layer (training forward) -> residual, its gradients through moe's own backward pass,
    clipping and the bias step; each part against its own oracle on what reached it."""
    cfg = mi.LayerConfig("step", T=200, H=272, E=12, k=3, I=144, I_shared=96)
    inp = mi.make_layer(cfg, seed=5)
    dev = moe.to_device(inp)
    g = torch.Generator(device="cuda").manual_seed(2)
    w1, w2 = [(torch.randn(cfg.H, generator=g, device="cuda") * 0.1 + 1) for _ in range(2)]
    gate = torch.randn(cfg.T, generator=g, device="cuda")
    x = dev["x"]
    h = torch.empty_like(x)
    back = moe.Backward(h, dev["W_r"], dev["b"], dev["W_up"], dev["W_down"], cfg.k,
                        Ws_up=dev["Ws_up"], Ws_down=dev["Ws_down"])
    moe.block_norm(x, w1, out=h)
    f = back.forward_train()
    y, _ = moe.block_residual(x, f, w=w2, gate=gate)
    dy = torch.randn(cfg.T, cfg.H, generator=g, device="cuda").to(BF)
    d = moe.block_residual_backward(dy, f, w=w2, gate=gate)
    grads = back(d["df"], saved=True)
    dx, dw1 = moe.block_norm_backward(grads["dx"], x, w1, dres=d["dx"])
    # the layer's part: the oracle on the rows that reached it, with the GPU's selection
    given = dict(inp, x=h.view(torch.int16).cpu().numpy().view(np.uint16))
    idx, _, _ = moe.route(dev["b"], cfg.k, x=h, W_r=dev["W_r"])
    ref = oracle.backward(given, idx.cpu().numpy(), d["df"].double().cpu().numpy())
    for name in ("dx", "dW_up", "dW_down", "dW_r", "dWs_up", "dWs_down"):
        got = grads[name].double().cpu().numpy()
        err = np.linalg.norm(got - ref[name]) / np.linalg.norm(ref[name])
        # the bounds of the layer's own backward tests
        assert err <= (2e-2 if name == "dW_r" else 1e-2), (name, err)
    # the norms' parts
    want = O.residual_grad(O.f64(dy), O.f64(f), O.f64(w2), True, O.f64(gate), "sigmoid", 1.0, None,
                           None, None, EPS)
    for name in d:
        O.check(d[name], want[name][0], d[name].dtype, want[name][1], 512 + cfg.T, name)
    gr = O.f64(grads["dx"]) * O.f64(w1)
    O.check(dx, O.norm_grad(gr, O.f64(x), EPS) + O.f64(d["dx"]), BF,
            O.norm_grad(gr, O.f64(x), EPS, mag=True) + O.f64(d["dx"]).abs(), 256, "dx")
    # clipping of the layer's weight gradients, in place, and of all of them with the norms'
    before = {n: t.double().clone() for n, t in grads.items()}
    true = float(sum(t.square().sum() for n, t in before.items() if n != "dx")) ** 0.5
    norm = back.clip(true / 3)
    assert abs(float(norm) - true) <= 1e-6 * true
    for n, t in grads.items():
        scale = 1.0 if n == "dx" else (true / 3) / (true + 1e-6)
        assert torch.allclose(t.double(), before[n] * scale, rtol=4 * 2.0 ** -24, atol=0), n
    again = back.clip(1e30)
    assert abs(float(again) - true / 3) <= 1e-5 * true
    every = [*grads.values(), d["dw"], dw1]
    total = float(sum(t.double().square().sum() for t in every)) ** 0.5
    assert abs(float(moe.clip_grad_norm(every, total * 2)) - total) <= 1e-6 * total
    counts = moe.dispatch(idx, cfg.E)[0]
    moe.bias_update(counts, dev["b"], 1e-3)


@pytest.mark.parametrize("T,E,k,stray", [(37, 6, 3, 0.0), (300, 8, 2, 0.3), (1, 5, 5, 0.0)])
def test_experts_outside_the_layer(T, E, k, stray):
    """A whole block in fp32 whose experts are the caller's: norm, route, sort, experts, gated
    return, residual and the next norm; every gradient against autograd in float64."""
    H, I = 96, 48
    g = torch.Generator().manual_seed(T)
    r = lambda *s, scale=1.0: torch.randn(*s, generator=g) * scale  # noqa: E731
    p = dict(x=r(T, H), w1=r(H, scale=0.1) + 1, w2=r(H, scale=0.1) + 1, w3=r(H, scale=0.1) + 1,
             A=r(E, I, H, scale=H ** -0.5), B=r(E, H, I, scale=I ** -0.5), gate=r(T))
    W_r, b = r(E, H, scale=H ** -0.5), torch.zeros(E)
    cy, ch = r(T, H), r(T, H)
    c = {n: t.cuda().contiguous() for n, t in p.items()}
    h = moe.block_norm(c["x"], c["w1"])
    idx, gates, _ = moe.route(b.cuda(), k, x=h, W_r=W_r.cuda())
    if stray:
        idx = torch.where(torch.rand(T, k, generator=g).cuda() < stray, -1, idx).int()
    rows, offsets, pos = moe.sort_tokens(h, idx, E)
    ends = offsets.tolist()
    out, act = torch.zeros_like(rows), torch.zeros(T * k, I, device="cuda")
    for e in range(E):
        s = slice(ends[e], ends[e + 1])
        act[s] = torch.tanh(rows[s] @ c["A"][e].t())
        out[s] = act[s] @ c["B"][e].t()
    f = moe.unsort_tokens(out, pos, weights=gates)
    y, h2 = moe.block_residual(c["x"], f, w=c["w2"], gate=c["gate"], w_next=c["w3"])
    # backward
    d = moe.block_residual_backward(cy.cuda(), f, w=c["w2"], gate=c["gate"], y=y, dh=ch.cuda(),
                                    w_next=c["w3"])
    dout, dgates = moe.unsort_tokens_backward(d["df"], pos, rows=out, weights=gates)
    drows = torch.zeros_like(rows)
    dA, dB = torch.zeros_like(c["A"]), torch.zeros_like(c["B"])
    for e in range(E):
        s = slice(ends[e], ends[e + 1])
        da = (dout[s] @ c["B"][e]) * (1 - act[s] ** 2)
        dB[e], dA[e], drows[s] = dout[s].t() @ act[s], da.t() @ rows[s], da @ c["A"][e]
    dh, _ = moe.sort_tokens_backward(drows, pos)
    dx, dw1 = moe.block_norm_backward(dh, c["x"], c["w1"], dres=d["dx"])
    # the same in float64 by autograd, the selection and the gates given
    q = {n: t.double().requires_grad_() for n, t in p.items()}
    wts = gates.double().cpu().requires_grad_()
    ii = idx.cpu()
    h64 = q["x"] / O.rms(q["x"], EPS) * q["w1"]
    f64 = torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        for e in range(E):
            t = torch.nonzero(ii[:, j] == e).flatten()
            v = torch.tanh(h64[t] @ q["A"][e].t()) @ q["B"][e].t()
            f64 = f64.index_add(0, t, v * wts[t, j].unsqueeze(1))
    y64 = q["x"] + torch.sigmoid(q["gate"]).unsqueeze(1) * (f64 / O.rms(f64, EPS) * q["w2"])
    h264 = y64 / O.rms(y64, EPS) * q["w3"]
    ((cy.double() * y64).sum() + (ch.double() * h264).sum()).backward()
    # a path of some 600 fp32 roundings (four norms, two products, the sums), each relative to terms
    # at most ten times the result: 600 * 10 * 2^-24 in norm
    tol = 600 * 10 * 2.0 ** -24
    got = dict(x=dx, w1=dw1, w2=d["dw"], w3=d["dw_next"], A=dA, B=dB, gate=d["dgate"])
    for name, t in got.items():
        want = q[name].grad
        assert float((t.double().cpu() - want).norm()) <= tol * float(want.norm()), name
    assert float((dgates.double().cpu() - wts.grad).norm()) <= tol * float(wts.grad.norm())
    for t, want in ((y, y64), (h2, h264)):
        assert float((t.double().cpu() - want.detach()).norm()) <= tol * float(want.detach().norm())


def test_a_plan_made_in_a_capture_serves_it_alone():
    grads = [torch.randn(100, device="cuda")]
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
        clip = moe.GradClip(grads)
        clip(1.0)
    with pytest.raises(ValueError):
        clip(1.0)
    before = grads[0].clone()
    for turn in range(2):
        grads[0].copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        assert float(grads[0].double().norm()) == pytest.approx(1.0, abs=1e-5)
    dev = moe.to_device(mi.make_layer(mi.LayerConfig("c", T=8, H=32, E=4, k=2, I=16), seed=0))
    back = moe.backward_from(dev, 2)
    with pytest.raises(ValueError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            back.clip(1.0)
