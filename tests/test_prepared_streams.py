"""Prepared calls (Layer, Backward, Block) on other streams than their constructor's: what they have
allocated stays theirs until that stream's work ends. The first tests replace the GPU by a record."""
import pytest
import torch

import moe_inputs as mi
import sparse_moe_layer_05_amd as moe
from sparse_moe_layer_05_amd import binding as B
from sparse_moe_layer_05_amd import block as K

CFG = mi.LayerConfig("s", T=8, H=32, E=4, k=2, I=16)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def marked(monkeypatch):
    """({stream handle: addresses marked as in use on it}, a list whose entry is the current stream)."""
    out, now = {}, [Stream(0)]
    monkeypatch.setattr(B, "_raw", lambda s, d: (now[0] if s is None else s).cuda_stream, raising=False)
    monkeypatch.setattr(B, "_torch_stream", lambda s, d: now[0] if s is None else s, raising=False)
    monkeypatch.setattr(B, "_stream", lambda s: None)

    def used_on(s, *tensors):
        if s is not None:
            out.setdefault(s.cuda_stream, set()).update(t.data_ptr() for t in tensors if t is not None)

    for m in (B, K):
        monkeypatch.setattr(m, "_launch", lambda *a: None)
        monkeypatch.setattr(m, "_used_on", used_on)
    return out, now


def cpu_layer():
    return {n: (torch.from_numpy(v.copy()) if v is not None else None)
            for n, v in mi.make_layer(mi.LayerConfig("s", T=8, H=32, E=4, k=2, I=16, act_dtype="f32",
                                                     expert_dtype="f32"), seed=0).items()
            if n in ("x", "W_r", "b", "W_up", "W_down")}


def test_a_layer_on_another_stream(marked):
    out, now = marked
    layer = moe.Layer(**cpu_layer(), k=2)
    layer()
    assert not out
    layer(Stream(7))
    assert out[7] >= {layer.ws.data_ptr(), layer.y.data_ptr()}
    now[0] = Stream(9)
    layer()
    assert out[9] >= {layer.ws.data_ptr(), layer.y.data_ptr()}


def test_a_block_on_another_stream(marked):
    out, now = marked
    block = moe.Block(**cpu_layer(), k=2, next_norm=True)
    block()
    assert not out
    block(Stream(7))
    own = {t.data_ptr() for t in (block.h, block.y, block.h_next, block.layer.ws, block.layer.y)}
    assert out[7] >= own
    now[0] = Stream(9)
    block()
    assert out[9] >= own


# -------------------------------------------------------------------------------- on the GPU

@pytest.fixture
def side():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    return torch.cuda.Stream()


LONG = 20_000_000      # clock ticks of a stream that is busy for some milliseconds


def busy(stream):
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(LONG)


def others(tensors):
    """New tensors of the same sizes, written at once; none may lie where the given ones did."""
    return [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in tensors.values()
            for _ in range(4)]


def sizes(*tensors):
    return {t.data_ptr(): t.numel() * t.element_size() for t in tensors if t is not None}


@pytest.mark.gpu
@pytest.mark.parametrize("given", [True, False])
def test_dropped_while_its_stream_is_busy(side, given):
    dev = moe.to_device(mi.make_layer(CFG, seed=1))
    w = {n: dev[n] for n in ("W_r", "b", "W_up", "W_down")}

    def call(fn):
        if given:
            return fn(side)
        with torch.cuda.stream(side):
            return fn()

    for make in (lambda: moe.Layer(dev["x"], k=2, **w), lambda: moe.Block(dev["x"], k=2, **w)):
        p = make()
        want = p().clone()
        p = make()
        own = sizes(*([p.ws] if isinstance(p, moe.Layer) else [p.h, p.layer.ws, p.layer.y]))
        busy(side)
        y = call(p)
        del p
        new = others(own)
        assert all(t.data_ptr() not in own for t in new)
        side.synchronize()
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_a_backward_dropped_while_its_stream_is_busy(side):
    dev = moe.to_device(mi.make_layer(CFG, seed=2))
    dy = torch.randn(CFG.T, CFG.H, device="cuda").to(torch.bfloat16)
    first = moe.backward_from(dev, 2)
    first.forward_train()
    want = first(dy, saved=True)
    back = moe.backward_from(dev, 2)
    own = sizes(back.ws)
    busy(side)
    y = back.forward_train(stream=side)
    got = dict(back(dy, stream=side, saved=True))
    del back
    new = others(own)
    assert all(t.data_ptr() not in own for t in new)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want) and y.shape == dy.shape
