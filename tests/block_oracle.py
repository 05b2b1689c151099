"""The operators around the layer in float64 on the CPU, from their formulas, each with a bound's
ingredient: the same expression with every term's magnitude, which roundings are relative to."""
import torch

U32 = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().double().cpu()


def check(got, want, dtype, mag, steps, what=""):
    """Every element within one rounding to `dtype` of `want`, after `steps` fp32 roundings of terms
    that add up to `mag` at most; NaN and infinities where `want` has them."""
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = torch.isnan(want) == torch.isnan(got)
    assert bool(same.all()), (what, "NaN in other places")
    fin = torch.isfinite(want)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), (what, "infinities")
    slack = steps * U32 * mag.expand_as(want)
    bound = unit(dtype) * (want.abs() + slack) + slack + torch.finfo(dtype).smallest_normal * unit(dtype) * 2
    off = (got - want).abs()
    bad = fin & ~(off <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((off / bound)[fin].max()))


# ---------------------------------------------------------------------------------- token rows

def positions(idx, E):
    """offsets, pos by walking the pairs in token order."""
    T, k = idx.shape
    chosen = [[] for _ in range(E)]
    for t in range(T):
        seen = set()
        for j in range(k):
            e = int(idx[t, j])
            if 0 <= e < E and e not in seen:
                seen.add(e)
                chosen[e].append((t, j))
    pos = torch.full((T, k), -1, dtype=torch.int32)
    offsets, at = [0], 0
    for pairs in chosen:
        for t, j in pairs:
            pos[t, j] = at
            at += 1
        offsets.append(at)
    return torch.tensor(offsets, dtype=torch.int32), pos


def spread(src, pos, weights, rows):
    out = rows.clone()
    T, k = pos.shape
    for t in range(T):
        for j in range(k):
            r = int(pos[t, j])
            if 0 <= r < rows.shape[0]:
                out[r] = src[t] * (1.0 if weights is None else weights[t, j])
    return out


def gather(rows, pos, weights, add, T, D, mag=False):
    y = torch.zeros(T, D, dtype=torch.float64) if add is None else (add.abs() if mag else add).clone()
    for t in range(T):
        for j in range(pos.shape[1]):
            r = int(pos[t, j])
            if 0 <= r < rows.shape[0]:
                v = rows[r] * (1.0 if weights is None else weights[t, j])
                y[t] += v.abs() if mag else v
    return y


def dots(a, rows, pos, mag=False):
    out = torch.zeros(pos.shape, dtype=torch.float64)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            r = int(pos[t, j])
            if 0 <= r < rows.shape[0]:
                v = a[t] * rows[r]
                out[t, j] = (v.abs() if mag else v).sum()
    return out


# --------------------------------------------------------------------------- the block's norms

def rms(v, eps):
    return (v.square().mean(-1, keepdim=True) + eps).sqrt()


def norm_grad(g, v, eps, mag=False):
    """Gradient of v / rms(v) against g; mag: with every term's magnitude."""
    m = rms(v, eps)
    if mag:
        n = v.abs() / m
        return (g.abs() + n * (g.abs() * n).mean(-1, keepdim=True)) / m
    n = v / m
    return (g - n * (g * n).mean(-1, keepdim=True)) / m


def gate_of(gate, act):
    if gate is None:
        return torch.ones(1, 1, dtype=torch.float64)
    a = gate.reshape(gate.shape[0], -1)
    return torch.sigmoid(a) if act == "sigmoid" else a


def residual(x, f, w, norm, gate, act, scale, eps):
    """y and the magnitude of its terms."""
    z = f / rms(f, eps) if norm else f
    if w is not None:
        z = z * w
    z = scale * gate_of(gate, act) * z
    return x + z, x.abs() + z.abs()


def residual_grad(dy, f, w, norm, gate, act, scale, y, dh, w_next, eps):
    """{name: (gradient, magnitude)}; dw and dw_next summed over the rows."""
    one = torch.ones(f.shape[1], dtype=torch.float64)
    wn = one if w_next is None else w_next
    ww = one if w is None else w
    d = torch.zeros_like(f) if dy is None else dy
    dm = d.abs()
    out = {}
    if dh is not None:
        g = dh * wn
        d = d + norm_grad(g, y, eps)
        dm = dm + norm_grad(g, y, eps, mag=True)
        n = y / rms(y, eps)
        if w_next is not None:
            out["dw_next"] = ((dh * n).sum(0), (dh * n).abs().sum(0))
    out["dx"] = (d, dm)
    a = gate_of(gate, act)
    n = f / rms(f, eps) if norm else f
    dz, dzm = scale * a * d, abs(scale) * a.abs() * dm
    if w is not None:
        out["dw"] = ((dz * n).sum(0), (dzm * n.abs()).sum(0))
    g, gm = dz * ww, dzm * ww.abs()
    out["df"] = (norm_grad(g, f, eps), norm_grad(gm, f, eps, mag=True)) if norm else (g, gm)
    if gate is not None:
        da, dam = scale * d * n * ww, abs(scale) * dm * (n * ww).abs()
        slope = a * (1 - a) if act == "sigmoid" else torch.ones_like(a)
        if gate.dim() == 1 or gate.shape[1] == 1:
            da, dam = da.sum(1, keepdim=True), dam.sum(1, keepdim=True)
        out["dgate"] = ((da * slope).reshape(gate.shape), (dam * slope.abs()).reshape(gate.shape))
    return out
