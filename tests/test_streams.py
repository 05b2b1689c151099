"""Streams that calls take: torch streams and objects that only carry a raw handle."""
import pytest
import torch

import moe_inputs as mi
import sparse_moe_layer_05_amd as moe
from sparse_moe_layer_05_amd import binding as B


class Raw:
    """Another library's stream: nothing but the handle."""

    def __init__(self, handle):
        self.cuda_stream = handle


def test_a_stream_object_needs_only_its_handle(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    seen = []
    B._launch(lambda *a: seen.append(a) or B.MOE_OK, "call", torch.device("cuda", 0), Raw(7), 1, 2)
    assert seen == [(1, 2, 7)]


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    other = Raw(7)
    other.device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        B._launch(lambda *a: B.MOE_OK, "call", torch.device("cuda", 0), other)


@pytest.mark.gpu
def test_every_call_on_a_raw_stream():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    s = torch.cuda.Stream()
    raw = Raw(s.cuda_stream)
    cfg = mi.LayerConfig("s", T=4, H=288, E=8, k=2, I=160, expert_dtype="mxfp4")
    dev = moe.to_device(mi.make_layer(cfg, seed=1))
    for path in ("auto", "few", "grouped_mx"):
        layer = moe.layer_from(dev, 2, path=path, expert_dtype="mxfp4")
        want = layer().clone()
        layer.y.zero_()
        s.wait_stream(torch.cuda.current_stream())
        layer(raw)
        s.synchronize()
        assert torch.equal(layer.y, want), path
    x = torch.randn(40, 288, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    q = moe.mx_quantize(x, "mxfp8", stream=raw)
    y = moe.mx_gemm(*q, dev["W_up"][0], dev["s_up"][0], stream=raw)
    v = moe.mx_dequantize(*q, stream=raw)
    idx, gates, _ = moe.route(dev["b"], 2, x=dev["x"], W_r=dev["W_r"], stream=raw)
    moe.dispatch(idx, 8, stream=raw)
    s.synchronize()
    p = moe.mx_quantize(x, "mxfp8")
    assert torch.equal(p[0], q[0]) and torch.equal(v, moe.mx_dequantize(*p))
    assert torch.equal(y, moe.mx_gemm(*p, dev["W_up"][0], dev["s_up"][0]))
