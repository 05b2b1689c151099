"""Token rows into expert order and back, and their gradients, against the formulas in float64."""
import pytest
import torch

import block_oracle as O
import sparse_moe_layer_05_amd as moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def rand(g, *s, dtype=F32, scale=1.0):
    return (torch.randn(*s, generator=g) * scale).to(dtype).cuda()


def experts(g, T, k, E, stray=0.0):
    """Distinct experts a token where E allows it, some of them outside [0, E) or repeated."""
    of = max(E, k)
    idx = torch.rand(T, of, generator=g).argsort(1)[:, :k].int()
    if stray:
        out = torch.rand(T, k, generator=g) < stray
        idx = torch.where(out, torch.randint(-3, 2 * E + 3, (T, k), generator=g).int(), idx)
    return idx


# additions on the longest path of a dot product: eight columns a lane, the wave, the passes over the
# row (4096 columns each), the waves
def dot_steps(D):
    return 8 * -(-D // 4096) + 6 + 8 + 2


CASES = [   # T, k, E, D, stray
    (1, 6, 128, 2688, 0.0), (1, 1, 1, 16, 0.0), (2, 3, 5, 48, 0.3), (7, 24, 512, 1024, 0.0),
    (3, 64, 64, 32, 0.2), (5, 24, 6, 528, 0.0), (64, 6, 128, 512, 0.0), (256, 2, 16, 64, 0.5),
    (257, 3, 16, 80, 0.2), (300, 5, 24, 288, 0.0), (33, 64, 1024, 144, 0.1), (600, 8, 128, 1040, 0.1),
    (4, 2, 3, 4112, 0.0), (3, 4, 8, 16400, 0.3), (9, 3, 4, 64, 1.0),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,E,D,stray", CASES)
def test_sort_and_back(T, k, E, D, stray, dtype):
    g = torch.Generator().manual_seed(T * 1000 + D)
    idx = experts(g, T, k, E, stray)
    offsets, pos = O.positions(idx, E)
    n = int(offsets[-1])
    x = rand(g, T, D, dtype=dtype)
    w = torch.rand(T, k, generator=g) + 0.1
    w[pos < 0] = NAN                           # weights of dropped pairs are not looked at
    wc = w.cuda()
    mark = rand(g, T * k, D, dtype=dtype)      # rows behind the last stay as they were
    # the sort, without and with weights
    for weights in (None, wc):
        out = mark.clone()
        rows, off, p = moe.sort_tokens(x, idx.cuda(), E, weights=weights, out=out)
        assert rows is out and torch.equal(off.cpu(), offsets) and torch.equal(p.cpu(), pos)
        want = O.spread(O.f64(x), pos, None if weights is None else w.double(), O.f64(mark))
        if weights is None:
            assert torch.equal(O.f64(rows), want)
        else:
            O.check(rows, want, dtype, want.abs(), 1, "rows")
        assert torch.equal(rows[n:], mark[n:])
    fresh, _, _ = moe.sort_tokens(x, idx.cuda(), E)
    assert torch.equal(fresh[:n].double().cpu(), O.spread(O.f64(x), pos, None, O.f64(mark))[:n])
    # its gradients
    pc = pos.cuda()
    drows = rand(g, T * k, D, dtype=dtype)
    drows[n:] = NAN                            # nor are rows behind the last
    d64, x64, w64 = O.f64(drows), O.f64(x), w.double()
    for out_dtype in (BF, F32):
        dx, none = moe.sort_tokens_backward(drows, pc, out_dtype=out_dtype)
        assert none is None and dx.dtype is out_dtype
        O.check(dx, O.gather(d64, pos, None, None, T, D), out_dtype,
                O.gather(d64, pos, None, None, T, D, mag=True), k, "dx")
        dx, dw = moe.sort_tokens_backward(drows, pc, x=x, weights=wc, out_dtype=out_dtype)
        O.check(dx, O.gather(d64, pos, w64, None, T, D), out_dtype,
                O.gather(d64, pos, w64, None, T, D, mag=True), k, "dx weighted")
        O.check(dw, O.dots(x64, d64, pos), F32, O.dots(x64, d64, pos, mag=True), dot_steps(D), "dw")
        assert bool((dw[pc < 0] == 0).all())
    # the way back
    for out_dtype in (BF, F32):
        add = rand(g, T, D, dtype=out_dtype)
        for weights, a in ((None, None), (wc, None), (wc, add)):
            y = moe.unsort_tokens(drows, pc, weights=weights, add=a, out_dtype=out_dtype)
            args = (d64, pos, None if weights is None else w64, O.f64(a), T, D)
            O.check(y, O.gather(*args), out_dtype, O.gather(*args, mag=True), k + 1, "y")
        over = add.clone()
        assert moe.unsort_tokens(drows, pc, weights=wc, add=over, out=over) is over
        assert torch.equal(over, y)
    # its gradients: rows of either type
    rows = drows
    for dy_dtype in (BF, F32):
        dy = rand(g, T, D, dtype=dy_dtype)
        out = mark.clone()
        dr, dw = moe.unsort_tokens_backward(dy, pc, rows=rows, weights=wc, out=out)
        want = O.spread(O.f64(dy), pos, w64, O.f64(mark))
        O.check(dr, want, dtype, want.abs(), 1, "drows")
        O.check(dw, O.dots(O.f64(dy), d64, pos), F32, O.dots(O.f64(dy), d64, pos, mag=True),
                dot_steps(D), "dweights")
        assert torch.equal(dr[n:], mark[n:]) and bool((dw[pc < 0] == 0).all())
        over = rows.clone()
        dr2, dw2 = moe.unsort_tokens_backward(dy, pc, rows=over, weights=wc, out=over)
        assert torch.equal(dr2[:n], dr[:n]) and torch.equal(dw2, dw)
        if dy_dtype is dtype:
            dr3, none = moe.unsort_tokens_backward(dy, pc, out=mark.clone())
            assert none is None and torch.equal(O.f64(dr3), O.spread(O.f64(dy), pos, None, O.f64(mark)))


@pytest.mark.parametrize("T,k,E", [(2000, 2, 1), (70000, 3, 1024), (262144, 2, 1024), (300000, 1, 2)])
def test_many_tokens(T, k, E):
    """Every way the sort finds its positions, against a stable sort; some choices of no expert here
    (the first slot's are distinct from the second's by their parity)."""
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(0, max(1, E // k), (T, k), generator=g) * k + torch.arange(k)
    idx = torch.where(torch.rand(T, k, generator=g) < 0.1, E + 3, idx).int().cuda()
    x = rand(g, T, 16)
    rows, offsets, pos = moe.sort_tokens(x, idx, E)
    key = torch.where(idx < E, idx, E).flatten().long()
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    want = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    want[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(pos.flatten(), want)
    assert torch.equal(offsets[1:].long(), torch.bincount(key, minlength=E + 1)[:E].cumsum(0))
    assert int(offsets[0]) == 0 and torch.equal(rows[:n], x[order[:n] // k])


def test_no_tokens_and_no_rows():
    x = torch.empty(0, 32, device="cuda")
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    rows, off, pos = moe.sort_tokens(x, idx, 5)
    assert rows.shape == (0, 32) and off.tolist() == [0] * 6 and pos.shape == (0, 2)
    assert moe.unsort_tokens(rows, pos).shape == (0, 32)
    dx, dw = moe.sort_tokens_backward(rows, pos, x=x)
    assert dx.shape == (0, 32) and dw.shape == (0, 2)
    dr, dw = moe.unsort_tokens_backward(x, pos, rows=rows)
    assert dr.shape == (0, 32) and dw.shape == (0, 2)
    # tokens, but no row at all
    pos = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    add = torch.randn(3, 32, device="cuda")
    assert torch.equal(moe.unsort_tokens(rows, pos, add=add), add)
    assert bool((moe.unsort_tokens(rows, pos) == 0).all())
    dr, dw = moe.unsort_tokens_backward(add, pos, rows=rows)
    assert dr.shape == (0, 32) and bool((dw == 0).all())


def test_positions_outside_the_rows_are_dropped():
    g = torch.Generator().manual_seed(1)
    rows = rand(g, 6, 48)
    pos = torch.tensor([[0, 6], [-7, 5], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    pc = pos.cuda()
    y = moe.unsort_tokens(rows, pc)
    assert torch.equal(y[0], rows[0]) and torch.equal(y[1], rows[5]) and bool((y[2] == 0).all())
    dy = rand(g, 3, 48)
    out = rows.clone()
    dr, dw = moe.unsort_tokens_backward(dy, pc, rows=rows, out=out)
    assert torch.equal(dr[1:5], rows[1:5]) and torch.equal(dr[0], dy[0]) and torch.equal(dr[5], dy[1])
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and bool((dw[2] == 0).all())


def test_values_that_are_not_finite_stay_in_their_token():
    g = torch.Generator().manual_seed(2)
    T, k, E, D = 20, 3, 6, 544
    idx = experts(g, T, k, E)
    x = rand(g, T, D, dtype=BF)
    x[4, 7], x[5, 8], x[6, 9] = NAN, float("inf"), -float("inf")
    w = torch.rand(T, k, generator=g)
    w[9, 1] = float("inf")
    rows, _, pos = moe.sort_tokens(x, idx.cuda(), E, weights=w.cuda())
    want = O.spread(O.f64(x), pos.cpu(), w.double(), torch.zeros(T * k, D, dtype=torch.float64))
    O.check(rows, want, BF, want.abs().nan_to_num(0, 0, 0), 1)
    y = moe.unsort_tokens(rows, pos)
    bad = ~torch.isfinite(y).all(1)
    assert bad.nonzero().flatten().tolist() == [4, 5, 6, 9]


@pytest.mark.parametrize("op", ["sort", "sort_backward", "unsort", "unsort_backward"])
def test_captured_and_on_another_stream(op):
    g = torch.Generator().manual_seed(5)
    T, k, E, D = 300, 4, 16, 272
    x, x2 = rand(g, T, D, dtype=BF), rand(g, T, D, dtype=BF)
    idx, idx2 = experts(g, T, k, E).cuda(), experts(g, T, k, E).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    rows, rows2 = rand(g, T * k, D, dtype=BF), rand(g, T * k, D, dtype=BF)
    _, _, pos = moe.sort_tokens(x, idx, E)
    _, _, pos2 = moe.sort_tokens(x, idx2, E)
    sx, si, sr, sp = x.clone(), idx.clone(), rows.clone(), pos.clone()
    calls = {
        "sort": lambda s=None: moe.sort_tokens(sx, si, E, weights=w, stream=s),
        "sort_backward": lambda s=None: moe.sort_tokens_backward(sr, sp, x=sx, weights=w, stream=s),
        "unsort": lambda s=None: (moe.unsort_tokens(sr, sp, weights=w, stream=s),),
        "unsort_backward": lambda s=None: moe.unsort_tokens_backward(sx, sp, rows=sr, weights=w,
                                                                     stream=s),
    }
    call = calls[op]
    first = [t.clone() for t in call()]
    sx.copy_(x2); si.copy_(idx2); sr.copy_(rows2); sp.copy_(pos2)
    second = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for turn in range(3):
        for a, b in ((x, x2), (idx, idx2), (rows, rows2), (pos, pos2)):
            {id(x): sx, id(idx): si, id(rows): sr, id(pos): sp}[id(a)].copy_(b if turn % 2 else a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, second if turn % 2 else first)), turn


def test_repeated_calls_agree():
    g = torch.Generator().manual_seed(6)
    x, idx = rand(g, 500, 1040, dtype=BF), experts(g, 500, 6, 128).cuda()
    w = torch.rand(500, 6, generator=g).cuda()
    rows, _, pos = moe.sort_tokens(x, idx, 128, weights=w)
    a = moe.sort_tokens_backward(rows, pos, x=x, weights=w)
    b = moe.unsort_tokens_backward(x, pos, rows=rows, weights=w)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, moe.sort_tokens_backward(rows, pos, x=x, weights=w)))
        assert all(torch.equal(p, q) for p, q in zip(b, moe.unsort_tokens_backward(x, pos, rows=rows, weights=w)))


def test_rows_past_32_bits():
    """Row offsets past 2^31 elements and 2^32 bytes: the last rows of a large buffer."""
    n, D = (1 << 31) // 4096 + 5, 4096
    rows = torch.zeros(n, D, dtype=BF, device="cuda")
    pos = torch.tensor([[0, n - 1], [n - 2, 1]], dtype=torch.int32, device="cuda")
    dy = torch.randn(2, D, device="cuda").to(BF)
    dr, _ = moe.unsort_tokens_backward(dy, pos, out=rows)
    assert torch.equal(dr[n - 1], dy[0]) and torch.equal(dr[n - 2], dy[1])
    assert torch.equal(dr[0], dy[0]) and torch.equal(dr[1], dy[1])
    assert int((dr[2:n - 2] != 0).any()) == 0
    y = moe.unsort_tokens(dr, pos)
    assert torch.equal(y, (2 * dy.float()).to(BF))


def test_short_rows_past_32_bits():
    n, D, T = (1 << 31) // 128 + 5, 128, 5000
    rows = torch.zeros(n, D, dtype=BF, device="cuda")
    pos = torch.arange(n - T, n, dtype=torch.int32, device="cuda")[:, None]
    dy = torch.randn(T, D, device="cuda").to(BF)
    dr, _ = moe.unsort_tokens_backward(dy, pos, out=rows)
    assert torch.equal(dr[n - T:], dy) and int((dr[:n - T] != 0).any()) == 0
    assert torch.equal(moe.unsort_tokens(dr, pos), dy)
