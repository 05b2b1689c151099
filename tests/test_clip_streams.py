"""What a GradClip does for the stream of a call: it waits for the table, and the memory that the
kernels follow addresses in stays theirs. The first tests replace the GPU by a record of the calls."""
import pytest
import torch

import moe_inputs as mi
import sparse_moe_layer_05_amd as moe
from sparse_moe_layer_05_amd import block as K


class Stream:
    def __init__(self, name, log):
        self.name, self.log, self.cuda_stream = name, log, hash(name)

    def wait_event(self, event):
        self.log.append((self.name, "waits for", event.where))

    def __repr__(self):
        return self.name


class Event:
    def record(self, stream):
        self.where = stream.name


@pytest.fixture
def calls(monkeypatch):
    """The log, the streams a and b, and a list whose entry is the current one."""
    log = []
    a, b, now = Stream("a", log), Stream("b", log), []
    now.append(a)
    monkeypatch.setattr(K, "_raw", lambda s, d: (now[0] if s is None else s).cuda_stream, raising=False)
    monkeypatch.setattr(K, "_torch_stream", lambda s, d: now[0] if s is None else s, raising=False)
    monkeypatch.setattr(K, "_is_capturing", lambda s: False, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(K, "_launch", lambda fn, name, dev, s, *args: log.append(
        ((now[0] if s is None else s).name, name)))
    monkeypatch.setattr(K, "_used_on", lambda s, *t: log.append(
        (s.name, "keeps", sorted(x.numel() * x.element_size() for x in t))))
    return log, a, b, now


def kept(clip):
    return sorted((clip.plan.numel(), 8))


def test_a_call_on_another_stream_waits_and_keeps_the_table(calls):
    log, a, b, _ = calls
    clip = moe.GradClip([torch.zeros(5)])
    log.clear()
    clip(1.0, stream=b)
    assert log == [("b", "waits for", "a"), ("b", "moe_clip_grads"), ("b", "keeps", kept(clip))]
    log.clear()
    clip(1.0)
    assert log == [("a", "moe_clip_grads")]


def test_another_current_stream_is_another_stream(calls):
    log, a, b, now = calls
    clip = moe.GradClip([torch.zeros(5)])
    log.clear()
    now[0] = b
    clip(1.0)
    assert log == [("b", "waits for", "a"), ("b", "moe_clip_grads"), ("b", "keeps", kept(clip))]


def test_the_stream_of_the_constructor_is_what_counts(calls):
    log, a, b, _ = calls
    clip = moe.GradClip([torch.zeros(5)], stream=b)
    assert log == [("b", "moe_clip_plan"), ("b", "keeps", kept(clip))]
    log.clear()
    clip(1.0, stream=b)
    clip(1.0)
    assert log == [("b", "moe_clip_grads"), ("a", "waits for", "b"), ("a", "moe_clip_grads"),
                   ("a", "keeps", kept(clip))]


def test_one_use(calls):
    log, a, b, _ = calls
    moe.clip_grad_norm([torch.zeros(5)], 1.0, stream=b)
    assert [e for e in log if "waits" in e[1]] == [] and all(e[0] == "b" for e in log)


# -------------------------------------------------------------------------------- on the GPU

@pytest.fixture
def side():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    return torch.cuda.Stream()


LONG = 20_000_000      # clock ticks of a stream that is busy for some milliseconds


@pytest.mark.gpu
def test_the_table_outlives_its_object(side):
    grads = [torch.full((1000,), 2.0, device="cuda"), torch.ones(3, 5, device="cuda")]
    true = float(sum(t.double().square().sum() for t in grads)) ** 0.5
    clip = moe.GradClip(grads)
    clip(1e9)                                  # (the library is loaded, the streams are at rest)
    clip = moe.GradClip(grads)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    norm = clip(true / 2, stream=side)
    at, size = clip.plan.data_ptr(), clip.plan.numel()
    del clip
    taken = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert all(t.data_ptr() != at for t in taken)
    side.synchronize()
    assert abs(float(norm) - true) <= 1e-6 * true
    assert torch.allclose(grads[0], torch.full_like(grads[0], 1.0), rtol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["stream", "current"])
def test_a_call_waits_for_a_table_made_on_another_stream(side, how):
    """Nothing but the call itself orders the two streams."""
    grads = [torch.full((70000,), 0.5, device="cuda")]
    true = float(grads[0].double().norm())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    clip = moe.GradClip(grads, stream=side)
    other = torch.cuda.Stream()
    if how == "stream":
        norm = clip(true / 4, stream=other)
    else:
        with torch.cuda.stream(other):
            norm = clip(true / 4)
    other.synchronize()
    assert abs(float(norm) - true) <= 1e-6 * true
    assert torch.allclose(grads[0], torch.full_like(grads[0], 0.125), rtol=1e-5)


@pytest.mark.gpu
def test_clip_of_a_backward_on_other_streams(side):
    dev = moe.to_device(mi.make_layer(mi.LayerConfig("c", T=8, H=32, E=4, k=2, I=16), seed=0))
    back = moe.backward_from(dev, 2)
    dy = torch.randn(8, 32, device="cuda").to(torch.bfloat16)
    back(dy)
    want = float(sum(g.double().square().sum() for n, g in back.grads.items() if n != "dx")) ** 0.5
    torch.cuda.synchronize()
    norm = back.clip(1e9, stream=side)
    side.synchronize()
    assert abs(float(norm) - want) <= 1e-6 * want
    assert abs(float(back.clip(1e9)) - want) <= 1e-6 * want


@pytest.mark.gpu
def test_a_captured_call_of_a_table_made_before(side):
    grads = [torch.full((300,), 3.0, device="cuda")]
    clip = moe.GradClip(grads, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip(1.0)
    for turn in range(3):
        grads[0].fill_(3.0 + turn)
        graph.replay()
        torch.cuda.synchronize()
        true = (3.0 + turn) * 300 ** 0.5
        assert abs(float(norm) - true) <= 1e-6 * true
        assert abs(float(grads[0].double().norm()) - 1.0) <= 1e-5


@pytest.mark.gpu
def test_a_table_made_in_a_capture_is_refused_in_another(side):
    """Only replays of the first graph write the table: in the second one it may be anything."""
    grads = [torch.randn(200, device="cuda")]
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        clip = moe.GradClip(grads)
        clip(1.0)
    with torch.cuda.graph(second):
        grads[0].mul_(2.0)
        with pytest.raises(ValueError, match="capture"):
            clip(1.0)
    with pytest.raises(ValueError, match="capture"):
        clip(1.0)
    with pytest.raises(moe.MoeError):
        clip(-1.0)
    for g in (first, second, first):
        g.replay()
    torch.cuda.synchronize()
    assert abs(float(grads[0].double().norm()) - 1.0) <= 1e-5


@pytest.mark.gpu
def test_a_captured_stream_that_is_not_the_current_one(side):
    """The stream that is given decides, not the current one."""
    grads = [torch.randn(200, device="cuda")]
    dev = moe.to_device(mi.make_layer(mi.LayerConfig("c", T=8, H=32, E=4, k=2, I=16), seed=0))
    back = moe.backward_from(dev, 2)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(other):                   # memory of that stream, which a capture cannot get
        held = torch.zeros(1000, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        grads[0].mul_(1.0)
        with torch.cuda.stream(other):
            with pytest.raises(ValueError, match="capture"):
                back.clip(1.0, stream=side)
            clip = moe.GradClip(grads, stream=side)
            clip(1.0, stream=side)
    with pytest.raises(ValueError, match="capture"):
        clip(1.0)
    grads[0].fill_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(grads[0].double().norm()) - 1.0) <= 1e-5 and held.numel() == 1000
