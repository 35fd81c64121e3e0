"""Cases of the voxel-transformer operators: attention within sets of voxels
(forward and backward), the residual root-mean-square norm with its 8-bit
output, and activation checkpoints in 8 bits with the weight gradient that
reads them.

``run`` computes a case either in plain torch operations in fp32 (``own`` is
false) or through the framework's calls (``own`` is true); ``exact`` gives the
same outputs from the definitions in fp64.

8-bit checkpoint: blocks of 32 consecutive channels of a row share a quantum
2^(floor(log2 max|x|) - 6) (at least 2^-126); a value is held as the integer
clamp(rint(x / quantum), -127, 127) and stands for integer * quantum.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def _attn(name, train, dtype, sets, lq, lk, hq, hk, d, cap=0.0, bias=False, ragged=True):
    return {"name": name, "kind": "attn", "train": train, "dtype": dtype, "sets": sets, "lq": lq, "lk": lk, "hq": hq,
            "hk": hk, "d": d, "cap": cap, "bias": bias, "ragged": ragged}


def _norm(name, train, dtype, n, c, residual, q8):
    return {"name": name, "kind": "norm", "train": train, "dtype": dtype, "n": n, "c": c, "residual": residual, "q8": q8}


def _ckpt(name, use, dtype, n, cin, cout, k, ndim, density):
    return {"name": name, "kind": "ckpt", "use": use, "dtype": dtype, "n": n, "cin": cin, "cout": cout, "k": k,
            "ndim": ndim, "density": density}


def listed():
    return [
        # one object query (8 heads on 2 shared key-value heads) over every voxel of a LiDAR scene: serving a detector
        _attn("query_over_scene", False, "f16", 1, 1, 102835, 8, 2, 64, bias=True, ragged=False),
        # a handful of pixel images, about 39 pixels each: the smallest call, where latency counts
        _attn("pixels_few", False, "f16", 8, 39, 39, 2, 2, 16),
        # a LiDAR scene cut into windows of about 100 voxels, inference
        _attn("windows", False, "bf16", 1024, 100, 100, 4, 4, 32, bias=True),
        # four scenes downsampled to 4096 voxels each, attention over the whole scene with capped scores
        _attn("scenes_capped", False, "f16", 4, 4096, 4096, 8, 8, 64, cap=10.0, ragged=False),
        # the training scenes (304,878 voxels) cut into windows: forward and backward
        _attn("train_windows", True, "bf16", 2400, 127, 127, 4, 4, 32, bias=True),
        # two downsampled scenes of about 8192 voxels, shared key-value heads, cap and distance bias: the largest
        _attn("train_scenes", True, "bf16", 2, 8192, 8192, 8, 4, 64, cap=10.0, bias=True),
        # object queries of 13 scenes over their voxels, odd head width, empty scenes among them
        _attn("train_queries", True, "f16", 13, 37, 1000, 6, 3, 40, cap=10.0, bias=True),
        # one image's pixels through a norm with 8-bit output: latency
        _norm("norm_few", False, "f16", 39, 64, True, "y"),
        # the training scenes: norm of the residual stream, its 8-bit checkpoint, and the backward pass from it
        _norm("norm_train", True, "bf16", 304878, 128, True, "h"),
        # a LiDAR scene in fp32 with a channel count that is no multiple of anything
        _norm("norm_odd", True, "f32", 102835, 77, True, "none"),
        # the training scenes: 8-bit checkpoint of a layer's input and the weight gradient from it (kernel 3, 128 channels)
        _ckpt("ckpt_train", "wgrad", "bf16", 304878, 128, 128, 3, 3, 0.04),
        # pixel tracks, 8 channels, kernel 3 in 2-D
        _ckpt("ckpt_pixels", "wgrad", "f16", 160798, 8, 8, 3, 2, 0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "norm", "ckpt"])
    if kind == "attn":
        hk = rng.choice([1, 2, 3, 4, 8])
        hq = hk * rng.choice([1, 1, 2, 4]) if hk < 8 else hk
        c = _attn("", rng.random() < 0.5, rng.choice(["f16", "bf16"]), 1, 1, 1, hq, hk, rng.choice([16, 24, 32, 40, 64, 80, 128]),
                  cap=rng.choice([0.0, 10.0]), bias=rng.random() < 0.6)
        form = rng.choice(["windows", "scenes", "queries"])
        if form == "windows":
            c["lq"] = c["lk"] = _log(rng, 8, 500)
            c["sets"] = max(1, _log(rng, 8, 200000) // c["lq"])
        elif form == "scenes":
            c["lq"] = c["lk"] = _log(rng, 300, 6000)
            c["sets"] = rng.randint(1, 2)
        else:
            c["sets"], c["lq"] = rng.randint(1, 6), _log(rng, 1, 200)
            c["lk"] = _log(rng, 100, 20000)
            c["ragged"] = rng.random() < 0.7
        # no more products than the largest listed case has
        while c["sets"] * c["lq"] * c["lk"] * c["hq"] * max(c["d"], 64) * (14 if c["train"] else 4) > 2 * 8192 ** 2 * 8 * 64 * 13:
            c["lk"] = max(1, c["lk"] // 2)
            c["lq"] = min(c["lq"], c["lk"])
    elif kind == "norm":
        c = _norm("", rng.random() < 0.6, rng.choice(["f16", "bf16", "f32"]), _log(rng, 1, 300000), _log(rng, 8, 512),
                  rng.random() < 0.7, rng.choice(["none", "y", "h"]))
        if rng.random() < 0.5:
            c["c"] = max(8, c["c"] // 8 * 8)
        if c["train"] and c["q8"] == "y":
            c["q8"] = "h"
    else:
        ndim = rng.choice([2, 3])
        c = _ckpt("", rng.choice(["wgrad", "wgrad", "unpack"]), rng.choice(["f16", "bf16"]), _log(rng, 100, 250000),
                  rng.choice([8, 16, 24, 32, 48, 64, 96, 128]), rng.choice([8, 16, 24, 32, 48, 64, 96, 128]), rng.choice([1, 3]),
                  ndim, 0.3 if ndim == 2 else 0.04)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _lengths(case):
    """Voxels (queries, keys) of each set: the same for every seed.  Ragged sets are 0.25 to 1.75 times the mean;
    every 11th has no voxels (queries over other voxels keep their queries there)."""
    s, lq, lk = case["sets"], case["lq"], case["lk"]
    if not case["ragged"]:
        return np.full(s, lq, np.int64), np.full(s, lk, np.int64)
    i = np.arange(s)
    f = 0.25 + 1.5 * np.modf((i + 1) * 0.6180339887498949)[0]
    k = np.where(i % 11 == 7, 0, np.maximum(1, np.rint(lk * f))).astype(np.int64)
    if lq == lk:
        return k, k
    g = 0.25 + 1.5 * np.modf((i + 1) * 0.7548776662466927)[0]
    return np.maximum(1, np.rint(lq * g)).astype(np.int64), k


def _grid(case):
    """Sides (batch, then spatial) of the grid whose cells a share `density` holds a voxel."""
    cells = max(case["n"], int(case["n"] / case["density"])) + 1
    if case["ndim"] == 2:
        return [-(-cells // 4096), 64, 64]
    side = math.isqrt(-(-cells // 32)) + 1
    return [1, side, side, 32]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["kind"] == "attn":
        lq, lk = _lengths(case)
        nq, nk, hq, hk, d = int(lq.sum()), int(lk.sum()), case["hq"], case["hk"], case["d"]
        s["q_starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lq)])).cuda()
        s["k_starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lk)])).cuda()
        s["longest"] = (int(lq.max()), int(lk.max()))
        s["same"] = case["lq"] == case["lk"]
        s["q"], s["k"], s["v"] = normal(nq, hq, d, scale=2.0), normal(nk, hk, d), normal(nk, hk, d)
        s["slopes"] = s["q_coords"] = s["k_coords"] = None
        if case["bias"]:
            side = max(4, round((8 * case["lk"]) ** (1 / 3)))  # an eighth of a set's box is filled
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
            s["k_coords"] = torch.randint(0, side, (nk, 4), generator=g, device="cuda", dtype=torch.int32)
            s["q_coords"] = s["k_coords"] if s["same"] else torch.randint(0, side, (nq, 4), generator=g, device="cuda", dtype=torch.int32)
        if case["train"]:
            s["dout"] = normal(nq, hq, d)
    elif case["kind"] == "norm":
        n, c = case["n"], case["c"]
        s["x"] = normal(n, c)
        s["residual"] = normal(n, c, scale=3.0) if case["residual"] else None
        s["w"] = normal(c, scale=0.2, dtype=torch.float32) + 1.0
        if case["train"]:
            s["dy"] = normal(n, c)
            s["dh"] = normal(n, c) if case["residual"] else None
    else:
        n, sides = case["n"], _grid(case)
        cells = torch.randperm(math.prod(sides), generator=g, device="cuda")[:n].sort().values
        coords, rest = [], cells
        for side in reversed(sides):
            coords.append(rest % side)
            rest = rest // side
        coords = torch.stack(coords[::-1], 1).to(torch.int32).contiguous()
        s["x"] = torch.relu(normal(n, case["cin"]))  # what a layer takes: the activations of the one before
        s["dy"] = normal(n, case["cout"])
        if case["use"] == "wgrad" and own:  # the map a training step keeps beside the scene
            from convolution_voxelised_point_amd import ts
            s["map"] = ts.build_kmap(coords, ts.HashTable(coords, 2.0), case["k"], 1, ts.TS_KMAP_PAIRS)
        elif case["use"] == "wgrad":
            s["nbr"] = _neighbours(coords, sides, case["k"])
    return s


def _neighbours(coords, sides, k):
    """[n][k^D] row of the voxel at each kernel offset, n where there is none."""
    n, r = coords.shape[0], (k - 1) // 2
    pad = [sides[0]] + [v + 2 * r for v in sides[1:]]
    step = [math.prod(pad[i + 1:]) for i in range(len(pad))]
    at = ((coords.long() + torch.tensor([0] + [r] * (len(sides) - 1), device="cuda")) * torch.tensor(step, device="cuda")).sum(1)
    table = torch.full((math.prod(pad),), n, dtype=torch.int64, device="cuda")
    table[at] = torch.arange(n, device="cuda")
    delta = torch.cartesian_prod(*[torch.arange(-r, k - r) for _ in sides[1:]]).reshape(k ** (len(sides) - 1), -1)
    move = (delta * torch.tensor(step[1:])).sum(1).cuda()
    return table[at[:, None] + move[None, :]]


def work(case):
    e = BYTES[case["dtype"]]
    if case["kind"] == "attn":
        lq, lk = _lengths(case)
        nq, nk, hq, hk, d = int(lq.sum()), int(lk.sum()), case["hq"], case["hk"], case["d"]
        pairs = int((lq * lk).sum()) * hq
        rows, keys = (4, 4) if case["train"] else (2, 2)
        b = (rows * nq * hq + keys * nk * hk) * d * e + nq * hq * 4 + 16 * (case["sets"] + 1)
        b += 16 * (nk if lq is lk else nq + nk) if case["bias"] else 0
        return {"bytes": b, "flops": pairs * d * (14 if case["train"] else 4)}
    if case["kind"] == "norm":
        n, c = case["n"], case["c"]
        full = n * c * e
        eight = n * c + n * -(-c // BLOCK)
        b = full * (3 if case["residual"] else 1) + full + 4 * c  # x, residual, h; y
        b += n * 4 if case["train"] else 0
        if case["q8"] == "y":
            b += eight + full  # the 8-bit output, and the values it stands for
        if case["train"]:
            b += full * (3 if case["residual"] else 2) + (2 * eight if case["q8"] == "h" else 0) + 4 * c
        return {"bytes": b, "flops": n * c * (16 if case["train"] else 6)}
    n, cin, cout = case["n"], case["cin"], case["cout"]
    kvol = case["k"] ** case["ndim"]
    if case["use"] == "unpack":
        return {"bytes": n * cin * 2 * e + 2 * n * (cin + -(-cin // BLOCK)), "flops": 4 * n * cin}
    pairs = n * (1 + (kvol - 1) * case["density"])
    return {"bytes": n * (cin * e + cin + -(-cin // BLOCK) + cout * e) + 8 * pairs + 4 * kvol * cin * cout,
            "flops": 2 * pairs * cin * cout}


# ---------------------------------------------------------------- plain forms (fp32)
def _padded(x, starts, longest):
    """[sets][longest][...] of packed rows, zeros past each set's end, and which rows are a set's own."""
    at = starts[:-1, None] + torch.arange(longest, device="cuda")[None, :]
    real = at < starts[1:, None]
    x = x[at.clamp(max=x.shape[0] - 1)].float()
    return torch.where(real.reshape(real.shape + (1,) * (x.dim() - 2)), x, 0.0), real


def _packed(x, starts, n):
    """Rows of [sets][longest][...] back in packed order."""
    row = torch.arange(n, device="cuda")
    of = torch.searchsorted(starts, row, right=True) - 1
    return x[of, row - starts[of]]


def _attn_plain(s):
    c = s["case"]
    dt, hq, hk, d, cap = DT[c["dtype"]], c["hq"], c["hk"], c["d"], c["cap"]
    grp, (lq, lk) = hq // hk, s["longest"]
    nq, nk, sets = s["q"].shape[0], s["k"].shape[0], c["sets"]
    qs, ks = s["q_starts"], s["k_starts"]

    def rows(x):  # [sets][longest][hq][d] -> [sets * hk][grp * longest][d]
        return x.reshape(sets, lq, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(sets * hk, grp * lq, d)

    def unrows(x):
        return x.reshape(sets, hk, grp, lq, d).permute(0, 3, 1, 2, 4).reshape(sets, lq, hq, d)

    def keys(x):
        return x.permute(0, 2, 1, 3).reshape(sets * hk, lk, d)

    def unkeys(x):
        return x.reshape(sets, hk, lk, d).permute(0, 2, 1, 3)

    q, _ = _padded(s["q"], qs, lq)
    k, real = _padded(s["k"], ks, lk)
    v, _ = _padded(s["v"], ks, lk)
    q, k, v = rows(q), keys(k), keys(v)
    scale = 1.0 / math.sqrt(d)
    t = (q @ k.transpose(1, 2).contiguous()) * scale
    if cap:
        t = torch.tanh(t / cap)
        z = (t * cap).reshape(sets, hk, grp, lq, lk)
    else:
        z = t.reshape(sets, hk, grp, lq, lk)
    if c["bias"]:
        qc, _ = _padded(s["q_coords"][:, 1:], qs, lq)
        kc, _ = _padded(s["k_coords"][:, 1:], ks, lk)
        dist = (qc[:, :, None, :] - kc[:, None, :, :]).square().sum(3).sqrt()
        z = z - s["slopes"].reshape(1, hk, grp, 1, 1) * dist[:, None, None]
    real = real[:, None, None, None, :]
    z = torch.where(real, z, -torch.inf)
    top = z.amax(4, keepdim=True)
    p = torch.where(real, torch.exp(z - torch.where(top > -torch.inf, top, 0.0)), 0.0)
    p = (p / p.sum(4, keepdim=True).clamp(min=1e-30)).reshape(sets * hk, grp * lq, lk)
    out = p @ v
    res = {"out": _packed(unrows(out), qs, nq).to(dt)}
    if c["train"]:
        do = rows(_padded(s["dout"], qs, lq)[0])
        dp = do @ v.transpose(1, 2).contiguous()
        ds = p * (dp - (do * out).sum(2, keepdim=True))
        if cap:
            ds = ds * (1.0 - t * t)
        ds = ds * scale
        res["dq"] = _packed(unrows(ds @ k), qs, nq).to(dt)
        res["dk"] = _packed(unkeys(ds.transpose(1, 2).contiguous() @ q), ks, nk).to(dt)
        res["dv"] = _packed(unkeys(p.transpose(1, 2).contiguous() @ do), ks, nk).to(dt)
    return res


def _held(x):
    """The fp32 values that the 8-bit checkpoint of x stands for."""
    n, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % BLOCK)).reshape(n, -1, BLOCK)
    top = x.abs().amax(2, keepdim=True)
    e = ((top.view(torch.int32) >> 23) - 6).clamp(min=1)  # biased exponent of the quantum
    quantum, inverse = (e << 23).view(torch.float32), ((254 - e) << 23).view(torch.float32)
    return (torch.round(x * inverse).clamp(-127, 127) * quantum).reshape(n, -1)[:, :c]


def _norm_plain(s):
    c = s["case"]
    dt = DT[c["dtype"]]
    x, w = s["x"].float(), s["w"]
    res = {}
    if c["residual"]:
        x = (x + s["residual"].float()).to(dt)
        res["h"] = x
        x = x.float()
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x * rstd * w
    res["y"] = y.to(dt)
    if c["q8"] == "y":
        res["y8"] = _held(y).to(dt)
    if c["train"]:
        x = _held(x) if c["q8"] == "h" else x
        dy, xn = s["dy"].float(), x * rstd
        g = dy * w
        dx = rstd * (g - xn * (g * xn).mean(1, keepdim=True))
        res["dx"] = (dx + s["dh"].float() if c["residual"] else dx).to(dt)
        res["dw"] = (dy * xn).sum(0)
    return res


def _ckpt_plain(s):
    c = s["case"]
    x = _held(s["x"].float())
    if c["use"] == "unpack":
        return {"x": x.to(DT[c["dtype"]])}
    n, kvol = x.shape[0], s["nbr"].shape[1]
    x = torch.nn.functional.pad(x, (0, 0, 0, 1))[s["nbr"]].reshape(n, -1)
    return {"dw": (x.t() @ s["dy"].float()).reshape(kvol, c["cin"], c["cout"])}


# ---------------------------------------------------------------- the framework's calls
def _attn_own(s, ts):
    c = s["case"]
    options = dict(k_starts=None if s["same"] else s["k_starts"], cap=c["cap"], slopes=s["slopes"], q_coords=s["q_coords"],
                   k_coords=s["k_coords"])
    out, lse = ts.attn_fwd(s["q"], s["k"], s["v"], s["q_starts"], **options)
    if not c["train"]:
        return {"out": out}
    dq, dk, dv = ts.attn_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, s["q_starts"], **options)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _norm_own(s, ts):
    c = s["case"]
    r = ts.norm_fwd(s["x"], s["w"], residual=s["residual"], eps=EPS, want_rstd=c["train"], y8=c["q8"] == "y", h8=c["q8"] == "h")
    res = {"y": r.y}
    if c["residual"]:
        res["h"] = r.h
    if c["q8"] == "y":
        res["y8"] = ts.act_unpack(r.y8, s["x"].dtype)
    if c["train"]:
        res["dx"], res["dw"] = ts.norm_bwd(s["dy"], r.h8 if c["q8"] == "h" else r.h, s["w"], r.rstd, dh=s["dh"])
    return res


def _ckpt_own(s, ts):
    packed = ts.act_pack(s["x"])
    if s["case"]["use"] == "unpack":
        return {"x": ts.act_unpack(packed, s["x"].dtype)}
    return {"dw": ts.conv_wgrad_act8(s["map"], packed, s["dy"])}


def run(state):
    kind = state["case"]["kind"]
    if own:
        from convolution_voxelised_point_amd import ts
        return {"attn": _attn_own, "norm": _norm_own, "ckpt": _ckpt_own}[kind](state, ts)
    return {"attn": _attn_plain, "norm": _norm_plain, "ckpt": _ckpt_plain}[kind](state)


# ---------------------------------------------------------------- the definitions in fp64
def _attn_exact(s):
    """Set by set, the gradients by differentiating the definition."""
    c = s["case"]
    hq, hk, d = c["hq"], c["hk"], c["d"]
    leaf = {n: s[n].double().requires_grad_(c["train"]) for n in ("q", "k", "v")}
    qs, ks = s["q_starts"].tolist(), s["k_starts"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    grads = {n: torch.zeros_like(t) for n, t in leaf.items()}
    for i in range(c["sets"]):
        a, b = slice(qs[i], qs[i + 1]), slice(ks[i], ks[i + 1])
        if qs[i] == qs[i + 1] or ks[i] == ks[i + 1]:
            continue
        q, k, v = (leaf[n][r].detach().requires_grad_(c["train"]) for n, r in (("q", a), ("k", b), ("v", b)))
        grp = torch.arange(hq, device="cuda") // (hq // hk)
        z = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0)[grp]) / d ** 0.5
        if c["cap"]:
            z = c["cap"] * torch.tanh(z / c["cap"])
        if c["bias"]:
            far = s["q_coords"][a, 1:].double()[:, None] - s["k_coords"][b, 1:].double()[None]
            z = z - s["slopes"].double()[:, None, None] * torch.linalg.vector_norm(far, dim=2)
        o = torch.matmul(torch.softmax(z, 2), v.transpose(0, 1)[grp]).transpose(0, 1)
        out[a] = o.detach()
        if c["train"]:
            got = torch.autograd.grad(o, (q, k, v), s["dout"][a].double())
            for (n, r), t in zip((("q", a), ("k", b), ("v", b)), got):
                grads[n][r] = t
    res = {"out": out}
    if c["train"]:
        res.update(dq=grads["q"], dk=grads["k"], dv=grads["v"])
    return res


def _held_exact(x):
    res = torch.empty_like(x)
    for b in range(0, x.shape[1], BLOCK):
        part = x[:, b:b + BLOCK]
        e = torch.frexp(part.abs().max(1, keepdim=True).values).exponent - 7  # max = m * 2^(e + 7), 0.5 <= m < 1
        quantum = ((e.clamp(min=-126).long() + 1023) << 52).view(torch.float64)  # exactly 2^e: ties decide on it
        res[:, b:b + BLOCK] = torch.clamp(torch.round(part / quantum), -127, 127) * quantum
    return res


def _norm_exact(s):
    c = s["case"]
    h = s["x"].double()
    res = {}
    if c["residual"]:
        h = h + s["residual"].double()
        res["h"] = h
        h = h.to(DT[c["dtype"]]).double()  # the stream is kept in its type: what follows takes the rounded sum
    w = s["w"].double()
    r = 1 / (torch.sum(h * h, 1, keepdim=True) / c["c"] + EPS).sqrt()
    res["y"] = h * r * w
    if c["q8"] == "y":
        res["y8"] = _held_exact(res["y"])
    if c["train"]:
        if c["q8"] == "h":
            h = _held_exact(h)
        dy = s["dy"].double()
        inner = torch.sum(dy * w * h, 1, keepdim=True)
        res["dx"] = r * dy * w - h * r ** 3 * inner / c["c"] + (s["dh"].double() if c["residual"] else 0)
        res["dw"] = torch.sum(dy * h * r, 0)
    return res


def _ckpt_exact(s):
    c = s["case"]
    x = _held_exact(s["x"].double())
    if c["use"] == "unpack":
        return {"x": x}
    dy, dw = s["dy"].double(), []
    for o in range(s["nbr"].shape[1]):
        rows = torch.nonzero(s["nbr"][:, o] < x.shape[0])[:, 0]
        dw.append(x[s["nbr"][rows, o]].t() @ dy[rows])
    return {"dw": torch.stack(dw)}


def exact(case, seed):
    return {"attn": _attn_exact, "norm": _norm_exact, "ckpt": _ckpt_exact}[case["kind"]](prepare(case, seed))
