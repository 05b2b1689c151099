"""What the library's operators around the layer are measured on, each beside a plain form in
elementary torch operations.

Three groups of operators:
  sort, sort_grad, unsort, unsort_grad    token rows moved into expert order and back, with a
            weight per (token, slot), and their gradients
  norm, norm_grad, residual, residual_grad    the norms before and after a block, with its gate,
            its residual and the next block's norm, and their gradients
  clip      the global norm of many gradients, and their clipping by it

``own`` chooses the side: False computes the plain form, True calls the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-5
MAX_NORM = 1.0


# ------------------------------------------------------------------------------------- cases

def _rows(name, op, T, D, E, of, k, dt, weighted, add=False, out=None):
    """`of` experts in all, of which this rank holds E (pairs of the others are dropped)."""
    return dict(name=name, op=op, T=T, D=D, E=E, of=of, k=k, dt=dt, weighted=weighted, add=add,
                out=out or dt)


def _block(name, op, T, H, dt, **kw):
    c = dict(name=name, op=op, T=T, H=H, dt=dt, w=True)
    if op == "norm_grad":
        c.update(dh=dt, dres=True)
    elif op.startswith("residual"):
        c.update(norm=True, gate="none", sigmoid=True, scale=1.0, next=True)
    c.update(kw)
    return c


def listed():
    return [
        # one decoded token's row to its six experts (Nano width)
        _rows("sort_one_token", "sort", 1, 2688, 128, 128, 6, "bf16", False),
        # a prefill batch to six of 128 experts
        _rows("sort_prefill", "sort", 8192, 2688, 128, 128, 6, "bf16", False),
        # training in fp32, weights on the experts' inputs, an odd batch: the gradient of the sort
        _rows("sort_train", "sort_grad", 1999, 288, 24, 24, 5, "f32", True),
        # one of four ranks of a LatentMoE layer: the gated sum of the experts it holds, from
        # their fp32 rows, on top of what another path gave
        _rows("unsort_share", "unsort", 1001, 1024, 128, 512, 24, "f32", True, True, "bf16"),
        # LatentMoE training: gradients of the gated sum, of the rows and of the gates
        _rows("unsort_train", "unsort_grad", 4096, 1024, 512, 512, 24, "bf16", True),
        # one decoded token: norm of the layer's output, residual, the next block's norm
        _block("residual_one_token", "residual", 1, 2688, "bf16"),
        # a prefill batch, the layer's output gated per token
        _block("residual_prefill", "residual", 8192, 2688, "bf16", gate="token", scale=0.5),
        # the norm before a small fp32 layer, an odd batch, joined with the residual's gradient
        _block("norm_train", "norm_grad", 1001, 288, "f32"),
        # the largest training batch: gate per element, both norms, every gradient
        _block("residual_train", "residual_grad", 8192, 4096, "bf16", gate="element"),
        # the gradients of the tiny fp32 layer, inside the limit: nothing to clip
        dict(name="clip_tiny", op="clip", of="tiny", n=3, total=0, dt="f32", active=False),
        # 24 small blocks, matrices in bf16, routers and norms in fp32: 192 tensors, clipped
        dict(name="clip_blocks", op="clip", of="blocks", n=192, total=0, dt="mixed", active=True),
        # the LatentMoE layer's fp32 gradients, clipped into other buffers
        dict(name="clip_latent", op="clip", of="latent", n=5, total=0, dt="f32", active=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rows", "rows", "block", "block", "clip"])
    if kind == "rows":
        of, k = rng.choice([(16, 1), (16, 2), (24, 5), (64, 4), (128, 6), (128, 8), (512, 22),
                            (512, 24)])
        D = 16 * _log(rng, 1, 256)
        T = _log(rng, 1, min(16384, 8192 * 6 * 2688 // (k * D)))
        op = rng.choice(["sort", "sort_grad", "unsort", "unsort_grad"])
        dt = rng.choice(["bf16", "f32"])
        out = rng.choice(["bf16", "f32"]) if op == "unsort" else dt
        return dict(op=op, T=T, D=D, E=of // rng.choice([1, 1, 4]), of=of, k=k, dt=dt,
                    weighted=rng.random() < 0.7, add=op == "unsort" and rng.random() < 0.5,
                    out=out)
    if kind == "block":
        H = 16 * _log(rng, 1, 512)
        T = _log(rng, 1, min(16384, 8192 * 4096 // H))
        op = rng.choice(["norm", "norm_grad", "residual", "residual_grad"])
        c = dict(op=op, T=T, H=H, dt=rng.choice(["bf16", "f32"]), w=rng.random() < 0.8)
        if op == "norm_grad":
            c.update(dh=rng.choice([c["dt"], "f32"]), dres=rng.random() < 0.5)
        elif op.startswith("residual"):
            c.update(norm=rng.random() < 0.7, gate=rng.choice(["none", "token", "element"]),
                     sigmoid=rng.random() < 0.7, scale=rng.choice([1.0, 0.5, 0.22]),
                     next=rng.random() < 0.7)
        return c
    n = _log(rng, 1, 400)
    return dict(op="clip", of="ragged", n=n, total=_log(rng, 16 * n, 2 ** 26),
                dt=rng.choice(["bf16", "f32", "mixed"]), active=rng.random() < 0.6)


# ------------------------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(_TYPES[dt])


def _clip_tensors(case):
    """[(elements, type)] of a clip case."""
    if case["of"] == "tiny":
        return [(16 * 256, "f32"), (16 * 128 * 256, "f32"), (16 * 256 * 128, "f32")]
    if case["of"] == "latent":
        return [(512 * 4096, "f32"), (512 * 512 * 1024, "f32"), (512 * 1024 * 512, "f32"),
                (1024 * 4096, "f32"), (4096 * 1024, "f32")]
    if case["of"] == "blocks":
        mat = [24 * 160 * 288, 24 * 288 * 160, 208 * 288, 288 * 208]
        return 24 * ([(n, "bf16") for n in mat] + [(24 * 288, "f32"), (24, "f32"), (288, "f32"),
                                                   (288, "f32")])
    # ragged: sizes spread over their logarithm, odd ones among them, scaled to the total
    r = random.Random(case["n"] * 1000003 + case["total"])
    part = [math.exp(r.uniform(0.0, 9.0)) for _ in range(case["n"])]
    scale = case["total"] / sum(part)
    out = []
    for p in part:
        dt = r.choice(["bf16", "f32"]) if case["dt"] == "mixed" else case["dt"]
        out.append((max(1, int(p * scale)), dt))
    return out


def _experts(case, g):
    """A router's answer: k distinct experts a token of Zipf(1.1) popularity, numbered as this
    rank numbers them (its own 0 .. E - 1, the other ranks' outside)."""
    T, of, k = case["T"], case["of"], case["k"]
    rank = torch.randperm(of, generator=g, device=DEV).float() + 1
    u = torch.rand(T, of, generator=g, device=DEV).clamp(1e-6, 1 - 1e-6)
    idx = torch.topk(-torch.log(-torch.log(u)) - 1.1 * torch.log(rank), k, dim=1).indices
    first = of // 2 if case["E"] < of else 0
    return (idx - first).int()


def _prepare_rows(case, g):
    T, D, k, P = case["T"], case["D"], case["k"], case["T"] * case["k"]
    s = dict(case=case, idx=_experts(case, g))
    if case["weighted"]:
        sc = torch.rand(T, k, generator=g, device=DEV) * 0.5 + 0.5
        s["weights"] = sc / sc.sum(1, keepdim=True)
    else:
        s["weights"] = None
    op = case["op"]
    if op != "sort":     # the sort's answer, in hand since the forward pass
        s["pos"] = _positions(s["idx"], case["E"])[1]
    if op == "sort":
        s["x"] = _normal(g, (T, D), case["dt"])
        s["rows"] = torch.zeros(P, D, dtype=_TYPES[case["dt"]], device=DEV)
    elif op == "sort_grad":
        s["drows"] = _normal(g, (P, D), case["dt"], 1e-2)
        s["x"] = _normal(g, (T, D), case["dt"])
    elif op == "unsort":
        s["rows"] = _normal(g, (P, D), case["dt"])
        s["add"] = _normal(g, (T, D), case["out"]) if case["add"] else None
    else:
        s["rows"] = _normal(g, (P, D), case["dt"])
        s["dy"] = _normal(g, (T, D), case["dt"], 1e-2)
        s["drows"] = torch.zeros(P, D, dtype=_TYPES[case["dt"]], device=DEV)
    return s


def _prepare_block(case, g):
    T, H, dt = case["T"], case["H"], case["dt"]
    s = dict(case=case, w=None)
    if case["w"]:
        s["w"] = (torch.randn(H, generator=g, device=DEV) * 0.1 + 1).to(_TYPES[dt])
    # rows differ in size as tokens do
    size = torch.exp2(torch.randint(-2, 4, (T, 1), generator=g, device=DEV).float())
    s["x"] = (torch.randn(T, H, generator=g, device=DEV) * size).to(_TYPES[dt])
    if case["op"] == "norm_grad":
        s["dh"] = _normal(g, (T, H), case["dh"], 1e-2)
        s["dres"] = _normal(g, (T, H), dt, 1e-2) if case["dres"] else None
    if not case["op"].startswith("residual"):
        return s
    s["f"] = _normal(g, (T, H), dt, 0.5)
    s["gate"] = None
    if case["gate"] == "token":
        s["gate"] = torch.randn(T, generator=g, device=DEV)
    elif case["gate"] == "element":
        s["gate"] = _normal(g, (T, H), dt)
    s["w_next"] = None
    if case["next"] and case["w"]:
        s["w_next"] = (torch.randn(H, generator=g, device=DEV) * 0.1 + 1).to(_TYPES[dt])
    if case["op"] == "residual_grad":
        s["dy"] = _normal(g, (T, H), dt, 1e-2)
        s["y"] = s["dh"] = None
        if case["next"]:
            s["y"] = _plain_residual(s)["y"]
            s["dh"] = _normal(g, (T, H), dt, 1e-2)
    return s


def _prepare_clip(case, g):
    """Gradients as a training loop holds them, views of one bucket per type: where sizes are odd,
    tensors begin anywhere in it."""
    sizes = _clip_tensors(case)
    total = sum(n for n, _ in sizes)
    std = (3.0 if case["active"] else 0.3) * MAX_NORM / math.sqrt(total)
    kinds = sorted({dt for _, dt in sizes})
    bucket = {dt: _normal(g, (sum(n for n, d in sizes if d == dt),), dt, std) for dt in kinds}
    # clipped into other buffers; inside the limit nothing changes, so in place
    target = {dt: torch.zeros_like(b) for dt, b in bucket.items()} if case["active"] else bucket

    def views(buffers):
        at = dict.fromkeys(kinds, 0)
        for n, dt in sizes:
            yield buffers[dt][at[dt]:at[dt] + n]
            at[dt] += n

    s = dict(case=case, grads=list(views(bucket)), out=list(views(target)),
             buckets=[target[dt] for dt in kinds])
    if own:
        import sparse_moe_layer_05_amd as moe
        s["clip"] = moe.GradClip(s["grads"], out=s["out"] if case["active"] else None)
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "clip":
        return _prepare_clip(case, g)
    if "H" in case:
        return _prepare_block(case, g)
    return _prepare_rows(case, g)


# --------------------------------------------------------------------------------- plain forms

def _positions(idx, E):
    """(offsets [E + 1], pos [T, k], order [T k]) of a stable sort of the pairs by expert;
    experts outside [0, E) go last and have no position."""
    e = idx.reshape(-1).long()
    key = torch.where((e >= 0) & (e < E), e, E)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=DEV)
    counts = torch.zeros(E + 1, dtype=torch.long, device=DEV).scatter_add_(
        0, key, torch.ones_like(key))
    offsets = torch.cat((counts.new_zeros(1), counts[:E].cumsum(0))).int()
    return offsets, torch.where(key < E, place, -1).reshape(idx.shape).int(), order


def _taken(rows, pos):
    """fp32 [T, k, D]: the row of every pair, zeros where it has none."""
    got = rows[pos.clamp(min=0).long()].float()
    return torch.where((pos >= 0).unsqueeze(-1), got, 0.0)


def _placed(values, pos, out):
    """values [T, k, D] written to their rows of a copy of `out`."""
    P, D = out.shape
    # pairs without a row go to one more, which is cut off
    full = torch.cat((out, out.new_zeros(1, D)))
    full[torch.where(pos >= 0, pos, P).reshape(-1).long()] = values.reshape(P, D).to(out.dtype)
    return full[:P]


def _weighted(values, s):
    return values if s["weights"] is None else values * s["weights"].unsqueeze(-1)


def _plain_rows(s):
    c, op = s["case"], s["case"]["op"]
    if op == "sort":
        offsets, pos, _ = _positions(s["idx"], c["E"])
        spread = s["x"].float().unsqueeze(1).expand(c["T"], c["k"], c["D"])
        return {"rows": _placed(_weighted(spread, s), pos, s["rows"]), "offsets": offsets,
                "pos": pos}
    pos = s["pos"]
    if op == "sort_grad":
        d = _taken(s["drows"], pos)
        out = {"dx": _weighted(d, s).sum(1).to(s["drows"].dtype)}
        if c["weighted"]:
            out["dweights"] = (d * s["x"].float().unsqueeze(1)).sum(-1)
        return out
    if op == "unsort":
        y = _weighted(_taken(s["rows"], pos), s).sum(1)
        if s["add"] is not None:
            y = y + s["add"].float()
        return {"y": y.to(_TYPES[c["out"]])}
    dy = s["dy"].float().unsqueeze(1).expand(c["T"], c["k"], c["D"])
    out = {"drows": _placed(_weighted(dy, s), pos, s["drows"])}
    if c["weighted"]:
        out["dweights"] = (_taken(s["rows"], pos) * dy).sum(-1)
    return out


def _unit(v):
    """(n(v), 1 / rms) of fp32 rows."""
    r = 1.0 / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * r, r


def _unit_grad(g, n, r):
    return r * (g - n * (g * n).mean(-1, keepdim=True))


def _times(v, w):
    return v if w is None else v * w.float()


def _gate_of(s):
    if s["gate"] is None:
        return 1.0
    a = s["gate"].float()
    a = 1.0 / (1.0 + torch.exp(-a)) if s["case"]["sigmoid"] else a
    return a.unsqueeze(-1) if a.dim() == 1 else a


def _plain_residual(s):
    c, f = s["case"], s["f"].float()
    z = _times(_unit(f)[0] if c["norm"] else f, s["w"])
    y = (s["x"].float() + c["scale"] * _gate_of(s) * z).to(s["x"].dtype)
    out = {"y": y}
    if c["next"]:
        out["h"] = _times(_unit(y.float())[0], s["w_next"]).to(y.dtype)
    return out


def _plain_residual_grad(s):
    c, dt = s["case"], s["f"].dtype
    d, out = s["dy"].float(), {}
    if c["next"]:
        n, r = _unit(s["y"].float())
        dh = s["dh"].float()
        d = d + _unit_grad(_times(dh, s["w_next"]), n, r)
        if s["w_next"] is not None:
            out["dw_next"] = (dh * n).sum(0)
    out["dx"] = d.to(dt)
    f = s["f"].float()
    n, r = _unit(f) if c["norm"] else (f, 1.0)
    a = _gate_of(s)
    dz = c["scale"] * a * d
    if s["w"] is not None:
        out["dw"] = (dz * n).sum(0)
    g = _times(dz, s["w"])
    out["df"] = (_unit_grad(g, n, r) if c["norm"] else g).to(dt)
    if s["gate"] is not None:
        da = c["scale"] * d * _times(n, s["w"])
        if c["gate"] == "token":
            da = da.sum(-1, keepdim=True)
        if c["sigmoid"]:
            da = da * a * (1 - a)
        out["dgate"] = da.reshape(s["gate"].shape).to(s["gate"].dtype)
    return out


def _plain_block(s):
    op = s["case"]["op"]
    if op == "norm":
        return {"h": _times(_unit(s["x"].float())[0], s["w"]).to(s["x"].dtype)}
    if op == "norm_grad":
        n, r = _unit(s["x"].float())
        dh = s["dh"].float()
        dx = _unit_grad(_times(dh, s["w"]), n, r)
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        out = {"dx": dx.to(s["x"].dtype)}
        if s["w"] is not None:
            out["dw"] = (dh * n).sum(0)
        return out
    return _plain_residual(s) if op == "residual" else _plain_residual_grad(s)


def _plain_clip(s):
    # a long sum: in 64 bits
    sq = [t.float().square().sum(dtype=torch.float64) for t in s["grads"]]
    norm = torch.stack(sq).sum().sqrt()
    coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * coef)
    return {"norm": norm.float(), "buckets": s["buckets"]}


# ------------------------------------------------------------------------- the library's calls

def _own_rows(s):
    import sparse_moe_layer_05_amd as moe
    c, op = s["case"], s["case"]["op"]
    if op == "sort":
        rows, offsets, pos = moe.sort_tokens(s["x"], s["idx"], c["E"], weights=s["weights"],
                                             out=s["rows"])
        return {"rows": rows, "offsets": offsets, "pos": pos}
    if op == "sort_grad":
        dx, dweights = moe.sort_tokens_backward(s["drows"], s["pos"], x=s["x"],
                                                weights=s["weights"])
        return {"dx": dx, "dweights": dweights} if c["weighted"] else {"dx": dx}
    if op == "unsort":
        return {"y": moe.unsort_tokens(s["rows"], s["pos"], weights=s["weights"], add=s["add"],
                                       out_dtype=_TYPES[c["out"]])}
    drows, dweights = moe.unsort_tokens_backward(s["dy"], s["pos"], rows=s["rows"],
                                                 weights=s["weights"], out=s["drows"])
    return {"drows": drows, "dweights": dweights} if c["weighted"] else {"drows": drows}


def _own_block(s):
    import sparse_moe_layer_05_amd as moe
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        return {"h": moe.block_norm(s["x"], s["w"], eps=EPS)}
    if op == "norm_grad":
        dx, dw = moe.block_norm_backward(s["dh"], s["x"], s["w"], dres=s["dres"], eps=EPS)
        return {"dx": dx} if dw is None else {"dx": dx, "dw": dw}
    act = "sigmoid" if c["sigmoid"] else "none"
    if op == "residual":
        y, h = moe.block_residual(s["x"], s["f"], w=s["w"], norm=c["norm"], gate=s["gate"],
                                  gate_act=act, scale=c["scale"], next_norm=c["next"],
                                  w_next=s["w_next"], eps=EPS)
        return {"y": y} if h is None else {"y": y, "h": h}
    return moe.block_residual_backward(s["dy"], s["f"], w=s["w"], norm=c["norm"], gate=s["gate"],
                                       gate_act=act, scale=c["scale"], y=s["y"], dh=s["dh"],
                                       w_next=s["w_next"], eps=EPS)


def _own_clip(s):
    norm = s["clip"](MAX_NORM)
    return {"norm": norm, "buckets": s["buckets"]}


def run(state):
    c = state["case"]
    if c["op"] == "clip":
        return _own_clip(state) if own else _plain_clip(state)
    if "H" in c:
        return _own_block(state) if own else _plain_block(state)
    return _own_rows(state) if own else _plain_rows(state)


# ---------------------------------------------------------------------------------------- work

_BYTES = {"bf16": 2, "f32": 4}


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(m for m, _ in _clip_tensors(case))
        b = sum(m * _BYTES[dt] for m, dt in _clip_tensors(case))
        return {"bytes": b * 2 if case["active"] else b, "flops": 3 * n}
    b = _BYTES[case["dt"]]
    if "H" in case:
        n, H = case["T"] * case["H"], case["H"]
        wb = H * b * (1 if case["w"] else 0)
        if op == "norm":
            return {"bytes": 2 * n * b + wb, "flops": 4 * n}
        if op == "norm_grad":
            return {"bytes": n * (2 * b + _BYTES[case["dh"]] + b * case["dres"])
                    + (wb + 4 * H if wb else 0), "flops": 10 * n}
        nxt = 1 if case["next"] else 0
        gate = {"none": 0, "token": 4 * case["T"], "element": n * b}[case["gate"]]
        if op == "residual":
            return {"bytes": n * b * (3 + nxt) + gate + wb * (1 + nxt), "flops": (8 + 4 * nxt) * n}
        return {"bytes": n * b * (4 + 2 * nxt) + 2 * gate + (wb + 4 * H) * (1 + nxt) * case["w"],
                "flops": (14 + 10 * nxt) * n}
    T, D, k = case["T"], case["D"], case["k"]
    kept = T * k * case["E"] // case["of"]       # pairs of this rank's experts, on average
    w = 4 * T * k if case["weighted"] else 0
    if op == "sort":
        return {"bytes": (T + kept) * D * b + 8 * T * k + w, "flops": kept * D}
    if op == "sort_grad":
        return {"bytes": (T * (2 if w else 1) + kept) * D * b + 4 * T * k + 2 * w,
                "flops": (4 if w else 1) * kept * D}
    if op == "unsort":
        return {"bytes": kept * D * b + T * D * _BYTES[case["out"]] * (2 if case["add"] else 1)
                + 4 * T * k + w, "flops": 2 * kept * D}
    return {"bytes": (T + kept * (2 if w else 1)) * D * b + 4 * T * k + 2 * w,
            "flops": (3 if w else 1) * kept * D}


# --------------------------------------------------------------------- the definition in 64 bits

def _count_positions(idx, E):
    """offsets and pos by counting: a pair's place among its expert's is the number of pairs
    before it, token by token, that chose the same expert."""
    chose = idx.reshape(-1, 1) == torch.arange(E, device=DEV, dtype=torch.int32)     # [P, E]
    before = torch.cumsum(chose, 0, dtype=torch.int32)
    ends = torch.cumsum(before[-1], 0)
    start = ends - before[-1]
    at = torch.where(chose, before - 1 + start, 0).sum(1)
    pos = torch.where(chose.any(1), at, -1).reshape(idx.shape)
    return torch.cat((start[:1], ends)).int(), pos.int()


def _f64_rows(s):
    c, op = s["case"], s["case"]["op"]
    T, k, D = c["T"], c["k"], c["D"]
    wt = torch.ones(T, k, device=DEV) if s["weights"] is None else s["weights"]
    wt = wt.double()
    if op == "sort":
        offsets, pos = _count_positions(s["idx"], c["E"])
    else:
        pos = s["pos"]
    t, j = torch.nonzero(pos >= 0, as_tuple=True)
    at = pos[t, j].long()
    if op in ("sort", "unsort_grad"):
        src = (s["x"] if op == "sort" else s["dy"]).double()
        moved = torch.zeros(T * k, D, dtype=torch.float64, device=DEV)
        moved[at] = src[t] * wt[t, j].unsqueeze(1)
        if op == "sort":
            return {"rows": moved, "offsets": offsets, "pos": pos}
        out = {"drows": moved}
        other, own_rows = src, s["rows"]
    else:
        own_rows = s["drows"] if op == "sort_grad" else s["rows"]
        total = torch.zeros(T, D, dtype=torch.float64, device=DEV)
        if op == "unsort" and s["add"] is not None:
            total += s["add"]
        for slot in range(k):      # one slot at a time: no token twice
            m = j == slot
            total[t[m]] += own_rows[at[m]].double() * wt[t[m], slot].unsqueeze(1)
        if op == "unsort":
            return {"y": total}
        out = {"dx": total}
        other = s["x"].double()
    if c["weighted"]:
        dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
        for slot in range(k):
            m = j == slot
            dw[t[m], slot] = torch.linalg.vecdot(other[t[m]], own_rows[at[m]].double())
        out["dweights"] = dw
    return out


def _f64_rms(v):
    return torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)


def _f64_norm_grad(g, v):
    """Gradient of v / rms(v) against g: (g - v <g, v> / (H rms^2)) / rms."""
    m = _f64_rms(v)
    return (g - v * ((g * v).sum(1, keepdim=True) / (v.shape[1] * m * m))) / m


def _f64_block(s):
    c, op = s["case"], s["case"]["op"]
    one = torch.ones(c["H"], dtype=torch.float64, device=DEV)
    w = one if s["w"] is None else s["w"].double()
    x = s["x"].double()
    if op == "norm":
        return {"h": x / _f64_rms(x) * w}
    if op == "norm_grad":
        dh = s["dh"].double()
        dx = _f64_norm_grad(dh * w, x)
        if s["dres"] is not None:
            dx += s["dres"]
        out = {"dx": dx}
        if s["w"] is not None:
            out["dw"] = (dh * (x / _f64_rms(x))).sum(0)
        return out
    f = s["f"].double()
    wn = one if s["w_next"] is None else s["w_next"].double()
    gate = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    if s["gate"] is not None:
        raw = s["gate"].double().reshape(c["T"], -1)
        gate = torch.sigmoid(raw) if c["sigmoid"] else raw
    n = f / _f64_rms(f) if c["norm"] else f
    if op == "residual":
        y = x + n * w * gate * c["scale"]
        out = {"y": y}
        if c["next"]:     # the next norm reads y as it is stored
            stored = y.to(s["x"].dtype).double()
            out["h"] = stored / _f64_rms(stored) * wn
        return out
    d, out = s["dy"].double(), {}
    if c["next"]:
        y, dh = s["y"].double(), s["dh"].double()
        d = d + _f64_norm_grad(dh * wn, y)
        if s["w_next"] is not None:
            out["dw_next"] = (dh * (y / _f64_rms(y))).sum(0)
    out["dx"] = d
    dz = d * gate * c["scale"]
    if s["w"] is not None:
        out["dw"] = (dz * n).sum(0)
    out["df"] = _f64_norm_grad(dz * w, f) if c["norm"] else dz * w
    if s["gate"] is not None:
        da = d * n * w * c["scale"]
        if c["gate"] == "token":
            da = da.sum(1, keepdim=True)
        out["dgate"] = (da * gate * (1 - gate) if c["sigmoid"] else da).reshape(s["gate"].shape)
    return out


def _f64_clip(s):
    square = torch.zeros((), dtype=torch.float64, device=DEV)
    for t in s["grads"]:
        d = t.double()
        square += torch.dot(d, d)
    norm = torch.sqrt(square)
    coef = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + 1e-6))
    kinds = sorted({t.dtype for t in s["grads"]}, key=str)      # bfloat16 before float32
    return {"norm": norm, "buckets": [torch.cat([t for t in s["grads"] if t.dtype == dt]).double()
                                      * coef for dt in kinds]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        return _f64_clip(s)
    return _f64_block(s) if "H" in case else _f64_rows(s)
