"""The norms before and after a block, with gate, residual and next norm, and their gradients,
against the formulas in float64."""
import pytest
import torch

import block_oracle as O
import sparse_moe_layer_05_amd as moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
# fp32 roundings on the longest path. A sum over a row: 32 columns a lane, the wave, eight waves; the
# root halves its error. A norm's value: half of that and six operations. A gradient joins two sums
# and about ten operations, the second norm's the first's error too.
SUM = 32 + 6 + 8
VALUE = SUM // 2 + 8
GRAD = 2 * (2 * SUM + 12)


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def rand(g, *s, dtype=F32, scale=1.0):
    return (torch.randn(*s, generator=g) * scale).to(dtype).cuda()


def gate_input(g, kind, T, H, dtype):
    if kind is None:
        return None
    return rand(g, T, scale=2.0) if kind == "token" else rand(g, T, H, dtype=dtype, scale=2.0)


SHAPES = [(1, 2688), (3, 16), (65, 48), (7, 512), (5, 520 + 8), (4, 1040), (3, 1552), (2, 2048),
          (3, 2064), (2, 3088), (5, 4096), (2, 4112), (3, 6160), (2, 8192), (1, 8208), (2, 12304),
          (3, 16384), (1100, 288), (37, 64), (19, 80), (9, 128), (21, 144), (70, 256), (5, 272),
          (40000, 16)]
KINDS = [(None, "none"), ("token", "sigmoid"), ("token", "none"), ("element", "sigmoid"),
         ("element", "none")]


def run(T, H, dtype, wdt, gate_kind, act, norm, weights, nxt, dh_dtype, seed=0, scale=0.7):
    g = torch.Generator().manual_seed(seed * 100003 + T * 17 + H)
    size = torch.exp2(torch.randint(-3, 4, (T, 1), generator=g).float())
    x = (torch.randn(T, H, generator=g) * size).to(dtype).cuda()
    f = rand(g, T, H, dtype=dtype, scale=0.5)
    w = (torch.randn(H, generator=g) * 0.2 + 1).to(wdt).cuda() if weights else None
    wn = (torch.randn(H, generator=g) * 0.2 + 1).to(wdt).cuda() if weights and nxt else None
    gate = gate_input(g, gate_kind, T, H, dtype)
    a = (O.f64(x), O.f64(f), O.f64(w), norm, O.f64(gate), act, scale, EPS)
    y, h = moe.block_residual(x, f, w=w, norm=norm, gate=gate, gate_act=act, scale=scale,
                              next_norm=nxt, w_next=wn, eps=EPS)
    want, mag = O.residual(*a)
    O.check(y, want, dtype, mag, VALUE + 4, "y")
    stored = O.f64(y)
    if nxt:
        wh = stored / O.rms(stored, EPS) * (1.0 if wn is None else O.f64(wn))
        O.check(h, wh, dtype, wh.abs(), VALUE, "h")
    else:
        assert h is None
    dy = rand(g, T, H, dtype=dtype, scale=0.1)
    dh = rand(g, T, H, dtype=dh_dtype, scale=0.1) if nxt else None
    got = moe.block_residual_backward(dy, f, w=w, norm=norm, gate=gate, gate_act=act, scale=scale,
                                      y=y if nxt else None, dh=dh, w_next=wn, eps=EPS)
    ref = O.residual_grad(O.f64(dy), O.f64(f), O.f64(w), norm, O.f64(gate), act, scale,
                          stored if nxt else None, O.f64(dh), O.f64(wn), EPS)
    assert sorted(got) == sorted(ref)
    for name, (value, m) in ref.items():
        dt = F32 if name in ("dw", "dw_next") else gate.dtype if name == "dgate" else dtype
        steps = GRAD + (T if name in ("dw", "dw_next") else SUM)
        O.check(got[name], value, dt, m, steps, name)
    return y, got


@pytest.mark.parametrize("dtype,dh_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_shapes(T, H, dtype, dh_dtype):
    run(T, H, dtype, dtype, "token", "sigmoid", True, True, True, dh_dtype)


@pytest.mark.parametrize("dtype,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("norm,weights,nxt", [(True, True, True), (True, False, True),
                                              (False, True, True), (False, False, True),
                                              (True, True, False), (False, True, False),
                                              (False, False, False)])
@pytest.mark.parametrize("kind,act", KINDS)
def test_forms(kind, act, norm, weights, nxt, dtype, wdt):
    run(13, 304, dtype, wdt, kind, act, norm, weights, nxt, dtype)
    run(3, 2704, dtype, wdt, kind, act, norm, weights, nxt, dtype, seed=1, scale=-1.5)


@pytest.mark.parametrize("dtype,dh_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_before(T, H, dtype, dh_dtype):
    g = torch.Generator().manual_seed(T + H)
    x, dres = rand(g, T, H, dtype=dtype, scale=3.0), rand(g, T, H, dtype=dtype, scale=0.1)
    dh = rand(g, T, H, dtype=dh_dtype, scale=0.1)
    for w in (None, (torch.randn(H, generator=g) * 0.2 + 1).to(dtype).cuda()):
        h = moe.block_norm(x, w, eps=EPS)
        n = O.f64(x) / O.rms(O.f64(x), EPS)
        want = n if w is None else n * O.f64(w)
        O.check(h, want, dtype, want.abs(), VALUE, "h")
        over = x.clone()
        assert moe.block_norm(over, w, eps=EPS, out=over) is over and torch.equal(over, h)
        gr = O.f64(dh) if w is None else O.f64(dh) * O.f64(w)
        for res in (None, dres):
            dx, dw = moe.block_norm_backward(dh, x, w, dres=res, eps=EPS)
            want, mag = O.norm_grad(gr, O.f64(x), EPS), O.norm_grad(gr, O.f64(x), EPS, mag=True)
            if res is not None:
                want, mag = want + O.f64(res), mag + O.f64(res).abs()
            O.check(dx, want, dtype, mag, GRAD, "dx")
            if w is None:
                assert dw is None
            else:
                t = O.f64(dh) * n
                O.check(dw, t.sum(0), F32, t.abs().sum(0), GRAD + T, "dw")
        over = dres.clone()
        dx2, _ = moe.block_norm_backward(dh, x, w, dres=over, eps=EPS, out=over)
        assert dx2 is over and torch.equal(over, dx)


@pytest.mark.parametrize("H", [304, 2704])
def test_residual_over_its_inputs(H):
    g = torch.Generator().manual_seed(8)
    x, f = rand(g, 9, H, dtype=BF), rand(g, 9, H, dtype=BF)
    y, h = moe.block_residual(x, f, next_norm=True)
    for i in (0, 1):
        t = [x.clone(), f.clone()]
        y2, h2 = moe.block_residual(*t, next_norm=True, out=t[i])
        assert y2 is t[i] and torch.equal(y2, y) and torch.equal(h2, h)
    # h over f as well: the same lane has read it
    t = [x.clone(), f.clone()]
    y2, h2 = moe.block_residual(*t, out=t[0], h_out=t[1])
    assert torch.equal(y2, y) and torch.equal(h2, h)


def test_only_the_next_norm_has_a_gradient():
    g = torch.Generator().manual_seed(9)
    T, H = 11, 320
    x, f, dh = rand(g, T, H), rand(g, T, H), rand(g, T, H)
    y, _ = moe.block_residual(x, f, next_norm=True)
    got = moe.block_residual_backward(None, f, y=y, dh=dh)
    zero = moe.block_residual_backward(torch.zeros_like(f), f, y=y, dh=dh)
    assert sorted(got) == ["df", "dx"] and all(torch.equal(got[n], zero[n]) for n in got)
    ref = O.residual_grad(None, O.f64(f), None, True, None, "none", 1.0, O.f64(y), O.f64(dh), None, EPS)
    for n in got:
        O.check(got[n], *ref[n][:1], F32, ref[n][1], GRAD + SUM, n)


def test_next_weights_without_their_gradient_are_not_met():
    """The C call takes w_next where dh is absent: nothing of it may reach dx or df."""
    T, H = 5, 48
    g = torch.Generator().manual_seed(15)
    f, dy = rand(g, T, H), rand(g, T, H)
    wn = torch.full((H,), float("inf"), device="cuda")
    dx, df = torch.empty_like(f), torch.empty_like(f)
    rc = moe.lib().moe_block_residual_backward(
        dy.data_ptr(), f.data_ptr(), None, None, None, None, 0, wn.data_ptr(), dx.data_ptr(),
        df.data_ptr(), None, None, None, T, H, 0, 0, 1, 1.0, EPS, None, 0, None)
    torch.cuda.synchronize()
    want = moe.block_residual_backward(dy, f)
    assert rc == 0 and torch.equal(dx, want["dx"]) and torch.equal(df, want["df"])


def test_no_tokens():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    assert moe.block_norm(x, w).shape == (0, 64)
    y, h = moe.block_residual(x, x, w=w, w_next=w, gate=torch.empty(0, device="cuda"))
    assert y.shape == h.shape == (0, 64)
    dx, dw = moe.block_norm_backward(x, x, w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    got = moe.block_residual_backward(x, x, w=w, y=x, dh=x, w_next=w)
    assert bool((got["dw"] == 0).all()) and bool((got["dw_next"] == 0).all())


@pytest.mark.parametrize("H", [304, 2704])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_zeros_and_far_values(H, dtype):
    """Zero rows stay zero; squares past fp32 do not lose the row; small rows meet eps."""
    g = torch.Generator().manual_seed(10)
    T = 6
    x = torch.randn(T, H, generator=g)
    x[0] = 0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3, 5] = 3e38
    x[4] *= 1e19
    x = x.to(dtype).cuda()
    h = moe.block_norm(x, eps=EPS)
    want = O.f64(x) / O.rms(O.f64(x), EPS)
    O.check(h, want, dtype, want.abs(), VALUE, "h")
    assert bool((h[0] == 0).all())
    dh = rand(g, T, H, dtype=dtype)
    dx, _ = moe.block_norm_backward(dh, x, eps=EPS)
    O.check(dx, O.norm_grad(O.f64(dh), O.f64(x), EPS), dtype,
            O.norm_grad(O.f64(dh), O.f64(x), EPS, mag=True), GRAD, "dx")
    small = rand(g, T, H, dtype=dtype)
    y, hn = moe.block_residual(small, x, next_norm=True, eps=EPS)
    want, mag = O.residual(O.f64(small), O.f64(x), None, True, None, "none", 1.0, EPS)
    O.check(y, want, dtype, mag, VALUE + 4, "y")
    dy = rand(g, T, H, dtype=dtype)
    got = moe.block_residual_backward(dy, x, y=y, dh=dh, eps=EPS)
    ref = O.residual_grad(O.f64(dy), O.f64(x), None, True, None, "none", 1.0, O.f64(y), O.f64(dh), None, EPS)
    for n in got:
        O.check(got[n], ref[n][0], dtype, ref[n][1], GRAD + SUM, n)


def test_rows_past_32_bits():
    """More than 2^31 elements: the last rows are those of a call on them alone."""
    T, H = (1 << 31) // 16384 + 9, 16384
    x = torch.randn(64, H, device="cuda").to(BF).repeat(T // 64 + 1, 1)[:T].contiguous()
    f = x.flip(0).contiguous()
    y, h = moe.block_residual(x, f, next_norm=True)
    y1, h1 = moe.block_residual(x[-20:].contiguous(), f[-20:].contiguous(), next_norm=True)
    assert torch.equal(y[-20:], y1) and torch.equal(h[-20:], h1)
    got = moe.block_residual_backward(x, f, y=y, dh=h)
    part = moe.block_residual_backward(x[-20:].contiguous(), f[-20:].contiguous(), y=y1, dh=h1)
    assert all(torch.equal(got[n][-20:], part[n]) for n in part)


def test_gates_at_their_ends():
    """Sigmoids of far and infinite gates, and their slopes, which are small on both sides."""
    T, H = 8, 128
    g = torch.Generator().manual_seed(11)
    x, f, dy = rand(g, T, H), rand(g, T, H), rand(g, T, H)
    q = torch.tensor([0.0, 20.0, -20.0, 80.0, -80.0, float("inf"), -float("inf"), 3.0])
    for gate in (q.cuda(), q[:, None].expand(T, H).contiguous().cuda(), q[:, None].cuda()):
        y, _ = moe.block_residual(x, f, gate=gate)
        want, mag = O.residual(O.f64(x), O.f64(f), None, True, O.f64(gate), "sigmoid", 1.0, EPS)
        O.check(y, want, F32, mag, VALUE + 6, "y")
        got = moe.block_residual_backward(dy, f, gate=gate)
        a = torch.sigmoid(O.f64(gate).reshape(T, -1))
        da = O.f64(dy) * (O.f64(f) / O.rms(O.f64(f), EPS))
        m = da.abs()
        if a.shape[1] == 1:
            da, m = da.sum(1, keepdim=True), m.sum(1, keepdim=True)
        slope = a * torch.sigmoid(-O.f64(gate).reshape(T, -1))   # 1 - a without its cancellation
        O.check(got["dgate"], (da * slope).reshape(gate.shape), F32, (m * slope).reshape(gate.shape),
                GRAD + SUM, "dgate")


@pytest.mark.parametrize("H", [304, 2704])
def test_values_that_are_not_finite_stay_in_their_row(H):
    g = torch.Generator().manual_seed(12)
    T = 9
    x, f = rand(g, T, H, dtype=BF), rand(g, T, H, dtype=BF)
    clean = moe.block_residual(x, f, next_norm=True)
    x[2, 3], f[4, 5], f[6, 7] = float("nan"), float("nan"), float("inf")
    y, h = moe.block_residual(x, f, next_norm=True)
    rows = [t for t in range(T) if t not in (2, 4, 6)]
    assert torch.equal(y[rows], clean[0][rows]) and torch.equal(h[rows], clean[1][rows])
    assert bool(torch.isnan(h[[2, 4, 6]]).any(1).all())
    dy = rand(g, T, H, dtype=BF)
    got = moe.block_residual_backward(dy, f, y=y, dh=dy)
    assert all(bool(torch.isfinite(got[n][rows]).all()) for n in ("dx", "df"))


def test_gradients_against_differences_on_the_gpu():
    """The loss along random directions, by the fp32 kernels' own forward pass."""
    g = torch.Generator().manual_seed(13)
    T, H = 7, 1024
    v = dict(x=rand(g, T, H), f=rand(g, T, H), w=rand(g, H, scale=0.2) + 1,
             w_next=rand(g, H, scale=0.2) + 1, gate=rand(g, T))
    cy, ch = rand(g, T, H), rand(g, T, H)

    def loss(a):
        y, h = moe.block_residual(a["x"], a["f"], w=a["w"], gate=a["gate"], w_next=a["w_next"], eps=1e-2)
        return float((cy.double() * y.double()).sum() + (ch.double() * h.double()).sum()), y

    _, y = loss(v)
    got = moe.block_residual_backward(cy, v["f"], w=v["w"], gate=v["gate"], y=y, dh=ch,
                                      w_next=v["w_next"], eps=1e-2)
    for name in v:
        u = torch.randn(v[name].shape, generator=g).cuda()
        step = 2.0 ** -7
        up, _ = loss(dict(v, **{name: v[name] + step * u}))
        down, _ = loss(dict(v, **{name: v[name] - step * u}))
        want = float((got["d" + name].double() * u.double()).sum())
        # 2 T H results, each rounded to 2^-24 of about 4 and met by a unit weight: their sum is off
        # by 4 * 2^-24 * sqrt(2 T H), over two steps; the third derivative adds step^2 of the scale
        scale = float((got["d" + name].double().square().sum() * u.double().square().mean()).sqrt())
        noise = 4 * 2.0 ** -24 * (2 * T * H) ** 0.5 / step
        assert abs((up - down) / (2 * step) - want) <= 4 * noise + 16 * step ** 2 * max(scale, 1.0), name


@pytest.mark.parametrize("backward", [False, True])
def test_captured_and_on_another_stream(backward):
    g = torch.Generator().manual_seed(14)
    T, H = 130, 1056
    w = rand(g, H)
    first = [rand(g, T, H, dtype=BF) for _ in range(4)]
    other = [rand(g, T, H, dtype=BF) for _ in range(4)]
    now = [t.clone() for t in first]
    gate = rand(g, T)

    def call(s=None):
        a, b, c, d = now
        if not backward:
            return [*moe.block_residual(a, b, w=w, gate=gate, w_next=w, stream=s),
                    moe.block_norm(c, w, stream=s)]
        out = moe.block_residual_backward(a, b, w=w, gate=gate, y=c, dh=d, w_next=w, stream=s)
        return [out[n] for n in sorted(out)] + list(moe.block_norm_backward(a, b, w, dres=c, stream=s))

    want = [[t.clone() for t in call()]]
    for t, o in zip(now, other):
        t.copy_(o)
    want.append([t.clone() for t in call()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for turn in range(4):
        for t, a, b in zip(now, first, other):
            t.copy_(b if turn % 2 else a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[turn % 2])), turn
