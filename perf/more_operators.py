"""Cases of the operators that complete a voxel-transformer layer: the norm of
each query and key head with the rotation by the voxel's position, the router of
rows to experts, the products grouped by expert, and the sum of what a row's
experts returned; forward and backward.

``run`` computes a case either in plain torch operations in fp32 (``own`` is
false) or through the framework's calls (``own`` is true); ``exact`` gives the
same outputs from the definitions in fp64.

Rotation: ``pairs[a]`` channel pairs turn with axis a; with P pairs in all, pair i
is channels (i, i + P), or (2i, 2i + 1) where interleaved, and turns by the angle
coordinate * freqs[i].  Channels from 2 P on stay as they are.

Routing: a row's `top` largest logits, the lowest expert first among equals; gates
are the softmax over those, or (over_all) over all logits.  The chosen (row,
expert) pairs, expert by expert and by row within one, are the grouped rows.

Grouped products: y[p] = x[rows[p]] W[e] for the grouped rows p of expert e; with
glu W has twice the columns and y = silu(first half) * second half.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def _rope(name, train, dtype, n, hq, hk, d, pairs, norm=True, interleaved=False, reach=512):
    return {"name": name, "kind": "rope", "train": train, "dtype": dtype, "n": n, "hq": hq, "hk": hk, "d": d, "px": pairs[0],
            "py": pairs[1], "pz": pairs[2] if len(pairs) > 2 else -1, "norm": norm, "interleaved": interleaved, "reach": reach}


def _route(name, train, dtype, n, experts, top, over_all):
    return {"name": name, "kind": "route", "train": train, "dtype": dtype, "n": n, "experts": experts, "top": top,
            "over_all": over_all}


def _group(name, use, dtype, n, experts, top, cin, cout):
    return {"name": name, "kind": "group", "use": use, "dtype": dtype, "n": n, "experts": experts, "top": top, "cin": cin,
            "cout": cout}


def _combine(name, train, dtype, n, experts, top, c):
    return {"name": name, "kind": "combine", "train": train, "dtype": dtype, "n": n, "experts": experts, "top": top, "c": c}


def listed():
    return [
        # the pixels of one image, 2-D, two heads: the smallest call, where latency counts
        _rope("rope_few", False, "f16", 39, 2, 2, 16, (4, 4)),
        # the training scenes (304,878 voxels): queries and keys of a projected matrix, and the gradients
        _rope("rope_train", True, "bf16", 304878, 4, 4, 32, (6, 6, 4)),
        # a LiDAR scene in fp32 far from the origin, shared key heads, part of the head turned, adjacent pairs
        _rope("rope_far", True, "f32", 102835, 6, 3, 40, (6, 6, 4), interleaved=True, reach=32000),
        # the rows of one image to 8 experts
        _route("route_few", False, "f32", 39, 8, 2, False),
        # the training scenes to 64 experts, with the logits' gradient
        _route("route_train", True, "bf16", 304878, 64, 2, True),
        # one object query through its two experts' first layer: serving a single token
        _group("expert_token", "glu", "f16", 1, 8, 2, 256, 512),
        # 64 queries over 64 experts: every expert's weights are read for a few rows each
        _group("experts_serve", "fwd", "bf16", 64, 64, 4, 1024, 1024),
        # the training scenes: first layer of the experts, and the gradient that the second one sends back through it
        _group("experts_voxels", "glu_train", "bf16", 304878, 8, 2, 128, 256),
        # wide experts over 16,384 rows, all three products: the largest
        _group("experts_wide", "train", "bf16", 16384, 16, 2, 1024, 4096),
        # channel counts that are no multiple of anything
        _group("experts_odd", "train", "f16", 4999, 7, 3, 77, 133),
        # what a few queries' experts returned
        _combine("combine_few", False, "f16", 37, 8, 2, 64),
        # the training scenes, with the gradients of the rows and of the gates
        _combine("combine_train", True, "bf16", 304878, 8, 2, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "route", "group", "group", "group", "group", "combine"])
    dtype = rng.choice(["f16", "bf16"])
    if kind == "rope":
        d = rng.choice([16, 24, 32, 40, 48, 64, 77, 80, 96, 128])
        hk = rng.choice([1, 2, 3, 4, 8])
        ndim = rng.choice([2, 3])
        turned = d // 2 if rng.random() < 0.7 else rng.randint(ndim, d // 2)
        last = turned // ndim
        pairs = [last] * (ndim - 1)
        pairs.insert(0, turned - sum(pairs))
        c = _rope("", rng.random() < 0.6, rng.choice([dtype, dtype, "f32"]), _log(rng, 1, 300000), hk * rng.choice([1, 1, 2, 4]), hk,
                  d, pairs, rng.random() < 0.7, rng.random() < 0.4, rng.choice([100, 2000, 32000]))
        c["n"] = max(1, min(c["n"], 2 ** 26 // ((c["hq"] + hk) * d)))
    elif kind == "route":
        e = _log(rng, 2, 256)
        c = _route("", rng.random() < 0.5, rng.choice([dtype, "f32"]), _log(rng, 1, 300000), e, rng.randint(1, min(8, e)),
                   rng.random() < 0.5)
        c["n"] = max(1, min(c["n"], 2 ** 25 // e))
    elif kind == "group":
        e = _log(rng, 2, 128)
        c = _group("", rng.choice(["fwd", "fwd", "glu", "glu", "glu_train", "train", "train"]), dtype, _log(rng, 1, 100000), e,
                   rng.randint(1, min(4, e)), _log(rng, 32, 2048), _log(rng, 32, 4096))
        if rng.random() < 0.7:
            c["cin"], c["cout"] = max(32, c["cin"] // 32 * 32), max(32, c["cout"] // 32 * 32)
        while e * c["cin"] * c["cout"] > 2 ** 27:
            c["cout"] //= 2
        # no more rows of channels, and no more products, than the largest listed cases have
        while c["n"] * c["top"] * max(c["cin"], c["cout"]) > 2 ** 27 or c["n"] * c["top"] * c["cin"] * c["cout"] > 2 ** 36:
            c["n"] = max(1, c["n"] // 2)
    else:
        e = _log(rng, 2, 64)
        c = _combine("", rng.random() < 0.6, rng.choice([dtype, dtype, "f32"]), _log(rng, 1, 300000), e, rng.randint(1, min(6, e)),
                     _log(rng, 8, 1024))
        if rng.random() < 0.6:
            c["c"] = c["c"] // 8 * 8
        c["n"] = max(1, min(c["n"], 2 ** 26 // (c["c"] * c["top"])))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _pairs(case):
    return [p for p in (case["px"], case["py"], case["pz"]) if p >= 0]


def _lean(experts):
    """What routing leans towards: some experts get several times the rows of others, and of 6 or more one gets none."""
    lean = 1.5 * torch.frac((torch.arange(experts, device="cuda") + 1) * 0.6180339887498949)
    if experts >= 6:
        lean[experts // 2] = -torch.inf
    return lean


def _grouped(g, case):
    """starts, rows and place of a routing, and the rows of each expert on the host."""
    n, e = case["n"], case["experts"]
    top = min(case["top"], e - (e >= 6))
    score = torch.randn(n, e, generator=g, device="cuda") + _lean(e)
    pick = score.topk(top, 1).indices.reshape(-1)
    order = torch.sort(pick, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(n * top, device="cuda")
    counts = torch.bincount(pick, minlength=e)
    starts = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    starts[1:] = counts.cumsum(0)
    return {"starts": starts, "rows": (order // top).int(), "place": place.int().reshape(n, top), "host": starts.tolist()}


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["kind"] == "rope":
        n, hq, hk, d, pairs = case["n"], case["hq"], case["hk"], case["d"], _pairs(case)
        # queries, keys and values are columns of one projected matrix
        s["q"], s["k"], _ = normal(n, hq + 2 * hk, d, scale=2.0).split((hq, hk, hk), 1)
        s["coords"] = torch.randint(-case["reach"], case["reach"], (n, len(pairs) + 1), generator=g, device="cuda", dtype=torch.int32)
        s["coords"][:, 0] = 0
        s["freqs"] = torch.cat([100.0 ** (-torch.arange(p, dtype=torch.float32) / max(p, 1)) for p in pairs]).cuda()
        s["wq"], s["wk"] = (normal(d, scale=0.2, dtype=torch.float32) + 1.0 if case["norm"] else None for _ in range(2))
        if case["train"]:
            s["dq"], s["dk"] = normal(n, hq, d), normal(n, hk, d)
    elif case["kind"] == "route":
        n, e = case["n"], case["experts"]
        s["logits"] = (torch.randn(n, e, generator=g, device="cuda") + _lean(e).clamp(min=-8.0)).to(dt)
        if case["train"]:
            s["dgates"] = normal(n, case["top"], dtype=torch.float32)
    elif case["kind"] == "group":
        s.update(_grouped(g, case))
        e, cin, cout, p = case["experts"], case["cin"], case["cout"], s["rows"].numel()
        s["x"] = normal(case["n"], cin)
        s["w"] = normal(e, cin, cout * (2 if case["use"].startswith("glu") else 1), scale=cin ** -0.5)
        if case["use"] == "train":
            s["dy"] = normal(p, cout)
        if case["use"] == "glu_train":  # the second layer goes back to cin channels; h was kept by the forward pass
            s["w2"] = normal(e, cout, cin, scale=cout ** -0.5)
            s["dy"], s["h"] = normal(p, cin), normal(p, 2 * cout)
        if own:
            from convolution_voxelised_point_amd import ts
            s["groups"] = ts.Groups(s["starts"], s["rows"])
    else:
        s.update(_grouped(g, case))
        n, top, c = case["n"], s["place"].shape[1], case["c"]
        s["y"] = normal(n * top, c)
        s["gates"] = torch.softmax(torch.randn(n, top, generator=g, device="cuda"), 1)
        if case["train"]:
            s["dout"] = normal(n, c)
    return s


def work(case):
    e, n = BYTES[case["dtype"]], case["n"]
    if case["kind"] == "rope":
        full = n * (case["hq"] + case["hk"]) * case["d"]
        b = 2 * full * e + n * 4 * (len(_pairs(case)) + 1)
        return {"bytes": b + 2 * full * e if case["train"] else b, "flops": full * (20 if case["train"] else 8)}
    if case["kind"] == "route":
        b = n * case["experts"] * e + n * case["top"] * 16 + 8 * (case["experts"] + 1)
        return {"bytes": b + n * (case["experts"] * e + case["top"] * 4) if case["train"] else b,
                "flops": n * case["experts"] * (8 if case["train"] else 4)}
    top = min(case["top"], case["experts"] - (case["experts"] >= 6))
    p = n * top
    if case["kind"] == "combine":
        c = case["c"]
        b = (p + n) * c * e + p * 8
        return {"bytes": b + (p + n) * c * e + p * 4 if case["train"] else b, "flops": p * c * (5 if case["train"] else 2)}
    cin, cout, use = case["cin"], case["cout"], case["use"]
    full = min(case["experts"] - (case["experts"] >= 6), p)  # experts that can have rows
    wide = cout * (2 if use.startswith("glu") else 1)
    b = (n * cin + full * cin * wide + p * cout) * e + 4 * p
    flops = 2 * p * cin * wide
    if use == "glu_train":
        b += (2 * p * cout + p * cin + full * cin * cout + 4 * p * cout) * e  # h; dy, w2, h again, dh
        flops += 2 * p * cin * cout
    if use == "train":
        b += (p * cout + p * cin) * e + full * cin * cout * 4  # dy, dx, dw
        flops *= 3
    return {"bytes": b, "flops": flops}


# ---------------------------------------------------------------- plain forms (fp32)
def _angles(s):
    """cos and sin of every row's pairs; the angles in fp64, which far positions need."""
    axis = torch.cat([torch.full((p,), a + 1) for a, p in enumerate(_pairs(s["case"]))]).cuda()
    t = s["coords"][:, axis].double() * s["freqs"].double()
    return torch.cos(t).float()[:, None], torch.sin(t).float()[:, None]


def _turn(x, cos, sin, interleaved):
    p = cos.shape[2]
    a, b = (x[..., 0:2 * p:2], x[..., 1:2 * p:2]) if interleaved else (x[..., :p], x[..., p:2 * p])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], 3).flatten(2) if interleaved else torch.cat([a, b], 2)
    return torch.cat([turned, x[..., 2 * p:]], 2)


def _rope_plain(s):
    c = s["case"]
    cos, sin = _angles(s)
    res = {}
    for name in ("q", "k"):
        x, w, dt = s[name].float(), s["w" + name], DT[c["dtype"]]
        xn = x
        if c["norm"]:
            rstd = torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)
            xn = x * rstd
        res[name] = _turn(xn * w if c["norm"] else x, cos, sin, c["interleaved"]).to(dt)
        if c["train"]:
            g = _turn(s["d" + name].float(), cos, -sin, c["interleaved"])
            if c["norm"]:
                res["dw" + name] = (g * xn).sum((0, 1))
                g = g * w
                g = rstd * (g - xn * (g * xn).mean(2, keepdim=True))
            res["d" + name] = g.to(dt)
    return res


def _route_plain(s):
    c = s["case"]
    z, top, e = s["logits"].float(), c["top"], c["experts"]
    ids = torch.arange(e, device="cuda")
    rest, experts, best = z, [], []
    for _ in range(top):
        m = rest.amax(1, keepdim=True)
        i = torch.where(rest == m, ids, e).amin(1, keepdim=True)
        experts.append(i)
        best.append(m)
        rest = torch.where(ids == i, -torch.inf, rest)
    experts, best = torch.cat(experts, 1), torch.cat(best, 1)
    p = torch.exp(z - best[:, :1])
    gates = torch.exp(best - best[:, :1]) / (p if c["over_all"] else torch.exp(best - best[:, :1])).sum(1, keepdim=True)
    flat = experts.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device="cuda")
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.bincount(flat, minlength=e).cumsum(0)])
    res = {"experts": experts.int(), "gates": gates, "starts": starts, "rows": (order // top).int(), "place": place.int().reshape(-1, top)}
    if c["train"]:
        g = s["dgates"]
        inner = (g * gates).sum(1, keepdim=True)
        if c["over_all"]:
            p = p / p.sum(1, keepdim=True)
            dz = -p * inner
            dz = dz.scatter_add(1, experts, gates * g)
        else:
            dz = torch.zeros_like(z).scatter(1, experts, gates * (g - inner))
        res["dlogits"] = dz.to(DT[c["dtype"]])
    return res


def _each(s):
    """(expert, its grouped rows) of the experts that have any."""
    return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(s["host"][:-1], s["host"][1:])) if b > a]


def _silu_plain(h):
    a, b = h.chunk(2, 1)
    return a / (1.0 + torch.exp(-a)) * b


def _group_plain(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    use, p = c["use"], s["rows"].numel()
    x, w = s["x"].float()[s["rows"]], s["w"].float()
    y = torch.empty(p, w.shape[2], device="cuda")
    for e, r in _each(s):
        y[r] = x[r] @ w[e]
    if use == "fwd":
        return {"y": y.to(dt)}
    if use == "glu":
        return {"y": _silu_plain(y).to(dt)}
    if use == "glu_train":
        w2, dy = s["w2"].float(), s["dy"].float()
        da = torch.empty(p, c["cout"], device="cuda")
        for e, r in _each(s):
            da[r] = dy[r] @ w2[e].t()
        a, b = s["h"].float().chunk(2, 1)
        sig = 1.0 / (1.0 + torch.exp(-a))
        dh = torch.cat([da * b * (sig + a * sig * (1.0 - sig)), da * a * sig], 1)
        return {"y": _silu_plain(y).to(dt), "h": y.to(dt), "dh": dh.to(dt)}
    dy = s["dy"].float()
    dx, dw = torch.empty(p, c["cin"], device="cuda"), torch.zeros_like(w)
    for e, r in _each(s):
        dx[r] = dy[r] @ w[e].t()
        dw[e] = x[r].t() @ dy[r]
    return {"y": y.to(dt), "dx": dx.to(dt), "dw": dw}


def _combine_plain(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    y = s["y"].float()[s["place"]]
    res = {"out": (s["gates"][:, :, None] * y).sum(1).to(dt)}
    if c["train"]:
        d = s["dout"].float()
        res["dgates"] = (y * d[:, None]).sum(2)
        dy = torch.empty(s["y"].shape, dtype=dt, device="cuda")
        dy[s["place"].reshape(-1)] = (s["gates"][:, :, None] * d[:, None]).to(dt).reshape(-1, c["c"])
        res["dy"] = dy
    return res


# ---------------------------------------------------------------- the framework's calls
def _rope_own(s, ts):
    c = s["case"]
    options = dict(wq=s["wq"], wk=s["wk"], eps=EPS, interleaved=c["interleaved"])
    q, k = ts.rope_fwd(s["q"], s["k"], s["coords"], s["freqs"], _pairs(c), **options)
    res = {"q": q, "k": k}
    if c["train"]:
        r = ts.rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["coords"], s["freqs"], _pairs(c), **options)
        if c["norm"]:
            res["dwq"], res["dwk"] = r.dwq, r.dwk
        res["dq"], res["dk"] = r.dq, r.dk
    return res


def _route_own(s, ts):
    c = s["case"]
    r = ts.route_fwd(s["logits"], c["top"], over_all=c["over_all"])
    res = {"experts": r.experts, "gates": r.gates, "starts": r.starts, "rows": r.rows, "place": r.place}
    if c["train"]:
        res["dlogits"] = ts.route_bwd(s["dgates"], s["logits"], r, over_all=c["over_all"])
    return res


def _group_own(s, ts):
    use, groups = s["case"]["use"], s["groups"]
    if use == "glu_train":
        y, h = ts.group_glu_fwd(s["x"], s["w"], groups, want_h=True)
        return {"y": y, "h": h, "dh": ts.group_glu_dgrad(s["dy"], s["w2"], s["h"], groups)}
    if use == "glu":
        return {"y": ts.group_glu_fwd(s["x"], s["w"], groups)[0]}
    res = {"y": ts.group_fwd(s["x"], s["w"], groups)}
    if use == "train":
        res["dx"], res["dw"] = ts.group_dgrad(s["dy"], s["w"], groups), ts.group_wgrad(s["x"], s["dy"], groups)
    return res


def _combine_own(s, ts):
    res = {"out": ts.combine_fwd(s["y"], s["place"], s["gates"])}
    if s["case"]["train"]:
        res["dy"], res["dgates"] = ts.combine_bwd(s["dout"], s["y"], s["place"], s["gates"])
    return {k: res[k] for k in ("out", "dgates", "dy") if k in res}


def run(state):
    kind = state["case"]["kind"]
    if own:
        from convolution_voxelised_point_amd import ts
        return {"rope": _rope_own, "route": _route_own, "group": _group_own, "combine": _combine_own}[kind](state, ts)
    return {"rope": _rope_plain, "route": _route_plain, "group": _group_plain, "combine": _combine_plain}[kind](state)


# ---------------------------------------------------------------- the definitions in fp64
def _rope_exact(s):
    """The rotation as a product of complex numbers, the gradients by differentiating it."""
    c, pairs = s["case"], _pairs(s["case"])
    p = sum(pairs)
    angle, at = [], 0
    for a, m in enumerate(pairs):
        angle.append(s["coords"][:, a + 1, None].double() * s["freqs"][None, at:at + m].double())
        at += m
    angle = torch.cat(angle, 1)
    phase = torch.polar(torch.ones_like(angle), angle)[:, None]
    res = {}
    for name in ("q", "k"):
        x = s[name].double().requires_grad_(c["train"])
        y, w = x, None
        if c["norm"]:
            w = s["w" + name].double().requires_grad_(c["train"])
            y = x / torch.sqrt((x * x).sum(2, keepdim=True) / c["d"] + EPS) * w
        parts = y[..., :2 * p].unflatten(2, (p, 2) if c["interleaved"] else (2, p)).movedim(3 if c["interleaved"] else 2, 0)
        z = torch.complex(parts[0], parts[1]) * phase
        turned = torch.stack([z.real, z.imag], 3 if c["interleaved"] else 2).flatten(2)
        y = torch.cat([turned, y[..., 2 * p:]], 2)
        res[name] = y.detach()
        if c["train"]:
            got = torch.autograd.grad(y, (x, w) if c["norm"] else (x,), s["d" + name].double())
            if c["norm"]:
                res["dw" + name] = got[1]
            res["d" + name] = got[0]
    return res


def _route_exact(s):
    c = s["case"]
    z, top, e = s["logits"].double(), c["top"], c["experts"]
    experts = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
    leaf = z.clone().requires_grad_(c["train"])
    best = leaf.gather(1, experts)
    gates = torch.softmax(leaf, 1).gather(1, experts) if c["over_all"] else torch.softmax(best, 1)
    n = z.shape[0]
    key = experts * n + torch.arange(n, device="cuda")[:, None]  # expert by expert, by row within one
    ordered = key.reshape(-1).sort().values
    starts = torch.searchsorted(ordered, torch.arange(e + 1, device="cuda") * n)
    res = {"experts": experts, "gates": gates.detach(), "starts": starts, "rows": ordered % n, "place": torch.searchsorted(ordered, key)}
    if c["train"]:
        res["dlogits"] = torch.autograd.grad(gates, leaf, s["dgates"].double())[0]
    return res


def _group_exact(s):
    c, use = s["case"], s["case"]["use"]
    rows, p, cout = s["rows"].long(), s["rows"].numel(), s["case"]["cout"]

    def silu(h):
        return h[:, :cout] * torch.sigmoid(h[:, :cout]) * h[:, cout:]
    new = lambda width: torch.empty(p, width, dtype=torch.float64, device="cuda")  # noqa: E731
    y = new(cout)
    res = {"y": y}
    if use == "glu_train":
        res["h"], res["dh"] = new(2 * cout), new(2 * cout)
    if use == "train":
        res["dx"], res["dw"] = new(c["cin"]), torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        a, b = s["host"][e], s["host"][e + 1]
        if a == b:
            continue
        x, w = s["x"].double()[rows[a:b]], s["w"][e].double()
        h = torch.mm(x, w)
        y[a:b] = silu(h) if use.startswith("glu") else h
        if use == "glu_train":
            res["h"][a:b] = h
            leaf = s["h"][a:b].double().requires_grad_()
            res["dh"][a:b] = torch.autograd.grad(torch.mm(silu(leaf), s["w2"][e].double()), leaf, s["dy"][a:b].double())[0]
        if use == "train":
            dy = s["dy"][a:b].double()
            res["dx"][a:b] = torch.mm(w, dy.t().contiguous()).t()
            res["dw"][e] = torch.mm(dy.t().contiguous(), x).t()
    return res


def _combine_exact(s):
    c = s["case"]
    y, gates, place = s["y"].double(), s["gates"].double(), s["place"].long()
    out = torch.zeros(c["n"], c["c"], dtype=torch.float64, device="cuda")
    for j in range(place.shape[1]):
        out += gates[:, j, None] * y[place[:, j]]
    res = {"out": out}
    if c["train"]:
        d = s["dout"].double()
        res["dgates"] = torch.stack([(d * y[place[:, j]]).sum(1) for j in range(place.shape[1])], 1)
        dy = torch.empty_like(y)
        for j in range(place.shape[1]):
            dy[place[:, j]] = gates[:, j, None] * d
        res["dy"] = dy
    return res


def exact(case, seed):
    return {"rope": _rope_exact, "route": _route_exact, "group": _group_exact, "combine": _combine_exact}[case["kind"]](prepare(case, seed))
