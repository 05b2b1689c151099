"""Token rows of many tokens, against the formulas in float64 (vectorised, on the GPU): short rows side by
side in a wave, more than one batch of pairs, what passes the last-level cache."""
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


def make(g, *s, dtype=F32):
    return torch.randn(*s, generator=g, device="cuda").to(dtype)


def choices(g, T, k, E, stray):
    """Distinct experts a token; some pairs outside [0, E)."""
    idx = torch.rand(T, max(E, k), generator=g, device="cuda").argsort(1)[:, :k].int()
    return torch.where(torch.rand(T, k, generator=g, device="cuda") < stray, -1 - idx, idx)


def positions(idx, E):
    """(offsets, pos) by a stable sort."""
    key = torch.where((idx >= 0) & (idx < E), idx, E).flatten().long()
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    pos = torch.full((key.numel(),), -1, dtype=torch.int32, device="cuda")
    pos[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    return torch.bincount(key, minlength=E + 1)[:E].cumsum(0), pos.view(idx.shape)


def taken(rows, pos, j):
    """float64 rows of slot j's pairs, zeros where there are none."""
    p = pos[:, j].long()
    return torch.where((p >= 0)[:, None], rows[p.clamp(min=0)].double(), 0.0)


def gather(rows, pos, w, add, mag=False):
    T, k = pos.shape
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64, device="cuda")
    if add is not None:
        y += add.double().abs() if mag else add.double()
    for j in range(k):
        v = taken(rows, pos, j)
        if w is not None:
            v = v * torch.where(pos[:, j] >= 0, w[:, j].double(), 0.0)[:, None]
        y += v.abs() if mag else v
    return y


def dots(a, rows, pos, mag=False):
    out = [a.double() * taken(rows, pos, j) for j in range(pos.shape[1])]
    return torch.stack([(v.abs() if mag else v).sum(1) for v in out], 1)


def close(got, want, dtype, mag, steps, what):
    """Within one rounding to `dtype`, after `steps` fp32 roundings of terms that add up to mag."""
    slack = steps * O.U32 * mag
    off = (got.double() - want).abs()
    ok = off <= O.unit(dtype) * (want.abs() + slack) + slack + 2.0 ** -133
    assert got.dtype is dtype and bool(ok.all()), (what, int((~ok).sum()))


def dot_steps(D):
    return 8 * -(-D // 4096) + 6 + 8 + 2


def spread(src, pos, w, into):
    """`into` with w * src at every kept pair's row, rounded once to its type."""
    out = into.clone()
    for j in range(pos.shape[1]):
        keep = pos[:, j] >= 0
        v = src[keep].double()
        if w is not None:
            v = v * w[keep, j].double()[:, None]
        out[pos[keep, j].long()] = v.to(out.dtype) if w is None else v.float().to(out.dtype)
    return out


def run(T, D, k, E, dtype, other, stray, seed=0):
    g = torch.Generator("cuda").manual_seed(T + D * 131 + k + seed)
    idx = choices(g, T, k, E, stray)
    ends, pos = positions(idx, E)
    n = int(ends[-1])
    x, mark = make(g, T, D, dtype=dtype), make(g, T * k, D, dtype=dtype)
    w = torch.rand(T, k, generator=g, device="cuda") + 0.1
    w[pos < 0] = NAN                       # not looked at
    for weights in (None, w):
        out = mark.clone()
        rows, off, p = moe.sort_tokens(x, idx, E, weights=weights, out=out)
        assert torch.equal(p, pos) and torch.equal(off[1:].long(), ends) and int(off[0]) == 0
        # one fp32 product (exact in fp64) and one rounding to the type: exactly that
        assert torch.equal(rows, spread(x, pos, weights, mark)), weights is None
    del rows, out
    drows = make(g, T * k, D, dtype=dtype)
    drows[n:] = NAN
    for odt in (dtype, other):
        dx, _ = moe.sort_tokens_backward(drows, pos, out_dtype=odt)
        close(dx, gather(drows, pos, None, None), odt, gather(drows, pos, None, None, True), k, "dx")
        dx, dw = moe.sort_tokens_backward(drows, pos, x=x, weights=w, out_dtype=odt)
        close(dx, gather(drows, pos, w, None), odt, gather(drows, pos, w, None, True), k, "weighted dx")
        close(dw, dots(x, drows, pos), F32, dots(x, drows, pos, True), dot_steps(D), "dweights")
        assert bool((dw[pos < 0] == 0).all())
        add = make(g, T, D, dtype=odt)
        for weights, a in ((None, None), (w, None), (w, add)):
            y = moe.unsort_tokens(drows, pos, weights=weights, add=a, out_dtype=odt)
            close(y, gather(drows, pos, weights, a), odt, gather(drows, pos, weights, a, True), k + 1, "y")
        over = add.clone()
        assert moe.unsort_tokens(drows, pos, weights=w, add=over, out=over) is over and torch.equal(over, y)
    for dyt in (dtype, other):
        dy = make(g, T, D, dtype=dyt)
        dr, dw = moe.unsort_tokens_backward(dy, pos, rows=drows, weights=w, out=mark.clone())
        assert torch.equal(dr, spread(dy, pos, w, mark)), dyt
        close(dw, dots(dy, drows, pos), F32, dots(dy, drows, pos, True), dot_steps(D), "dweights")
        assert bool((dw[pos < 0] == 0).all())
        over = drows.clone()
        dr2, dw2 = moe.unsort_tokens_backward(dy, pos, rows=over, weights=w, out=over)
        assert torch.equal(dr2[:n], dr[:n]) and torch.equal(dw2, dw)
    dy = make(g, T, D, dtype=dtype)
    dr, none = moe.unsort_tokens_backward(dy, pos, out=mark.clone())
    assert none is None and torch.equal(dr, spread(dy, pos, None, mark))


@pytest.mark.parametrize("dtype,other", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("k", [1, 3, 5, 24])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 144, 256])
def test_short_rows(D, k, dtype, other):
    """Rows of up to 256 columns, several tokens a wave; the last wave is not full."""
    run(4099, D, k, 32, dtype, other, 0.2)


@pytest.mark.parametrize("dtype,other", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,D,k", [(8200, 512, 24), (4100, 1040, 12), (8200, 288, 9), (2000, 2704, 24)])
def test_more_than_one_batch_of_pairs(T, D, k, dtype, other):
    run(T, D, k, 64, dtype, other, 0.1)


@pytest.mark.parametrize("dtype,other", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,D,k", [(17000, 2704, 2), (10400, 2704, 4), (8200, 2704, 6), (5400, 1040, 24)])
def test_past_the_last_level_cache(T, D, k, dtype, other):
    """More than 256 MB of operands and results in each of the passes."""
    assert T * D * (2 + 2 * k) > 256 << 20
    run(T, D, k, 64, dtype, other, 0.0)


@pytest.mark.parametrize("T,k,E", [(5000, 4, 3), (3000, 24, 512), (262144, 2, 1024)])
def test_repeated_experts_of_many_tokens(T, k, E):
    """The first of a token's pairs with an expert is kept, on every way to the positions."""
    g = torch.Generator("cuda").manual_seed(T)
    idx = torch.randint(-2, E + 2, (T, k), generator=g, device="cuda").int()
    first = idx.clone()
    for j in range(1, k):
        first[:, j] = torch.where((idx[:, :j] == idx[:, j:j + 1]).any(1), -1, idx[:, j])
    ends, want = positions(first, E)
    x = make(g, T, 16)
    rows, off, pos = moe.sort_tokens(x, idx, E)
    assert torch.equal(pos, want) and torch.equal(off[1:].long(), ends)
    n = int(ends[-1])
    assert torch.equal(rows[:n], spread(x, want, None, torch.zeros_like(rows))[:n])
