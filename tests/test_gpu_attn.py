"""GPU parity of attention within packed sets (forward and backward) against a
plain fp64 implementation, set by set.

Tolerances, element by element, from the kernels' roundings (u = 2^-11 fp16,
2^-8 bf16; all else is fp32):
  scores      |dz| <= (d + 16) 2^-24 scale sum|q||k| + cap 2^-21 + distances 2^-22
  p           relative 2 |dz| (score and lse), then u for the product's operand
  out         u |out| + sum_j p_j |v_j| (u + 2|dz|)
  ds          u |ds| + 2|dz| |ds| + p (d 2^-24 sum|do||v| + sum|do| err(out)), the
              last term from delta = sum do * out with the rounded out
  dq, dk, dv  u |result| + the errors of ds or p times the other operand
fp16 also drops 2^-25 per operand, and per result, below its normal range."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}


def reference(q, k, v, qs, ks, scale, cap=0.0, slopes=None, qc=None, kc=None, dout=None, dtype=torch.float16):
    """fp64 results and elementwise error bounds, dicts of out, lse (and dq, dk, dv)."""
    u, tiny = U[dtype], TINY[dtype]
    q, k, v = (t.double().cpu() for t in (q, k, v))
    nq, hq, d = q.shape
    grp = hq // k.shape[1]
    ref = {"out": torch.zeros_like(q), "lse": torch.full((nq, hq), -math.inf, dtype=torch.float64)}
    tol = {"out": torch.zeros_like(q), "lse": torch.zeros((nq, hq), dtype=torch.float64)}
    if dout is not None:
        dout = dout.double().cpu()
        for n, t in (("dq", q), ("dk", k), ("dv", v)):
            ref[n], tol[n] = torch.zeros_like(t), torch.zeros_like(t)
    qs, ks = [int(x) for x in qs], [int(x) for x in ks]
    for s in range(len(qs) - 1):
        a, b = slice(qs[s], qs[s + 1]), slice(ks[s], ks[s + 1])
        if qs[s] == qs[s + 1] or ks[s] == ks[s + 1]:
            continue
        for h in range(hq):
            qi, kj, vj = q[a, h], k[b, h // grp], v[b, h // grp]
            raw = scale * qi @ kj.T
            z = cap * torch.tanh(raw / cap) if cap else raw
            dz = (d + 16) * 2.0 ** -24 * scale * (qi.abs() @ kj.abs().T) + cap * 2.0 ** -21
            if slopes is not None:
                far = (qc[a, None, 1:].double().cpu() - kc[None, b, 1:].double().cpu()).square().sum(2).sqrt()
                z = z - float(slopes[h]) * far
                dz = dz + abs(float(slopes[h])) * far * 2.0 ** -22
            lse = torch.logsumexp(z, 1, keepdim=True)
            p = torch.where(torch.isfinite(lse), torch.exp(z - lse), 0.0)
            out = p @ vj
            ep = p * (u + 2 * dz) + tiny
            eo = u * out.abs() + 1.05 * (ep @ vj.abs()) + tiny + 1e-30
            ref["out"][a, h], tol["out"][a, h] = out, eo
            ref["lse"][a, h] = lse[:, 0]
            tol["lse"][a, h] = 2 * dz.amax(1) + 2.0 ** -20 * (1 + lse[:, 0].abs())
            if dout is None:
                continue
            do = dout[a, h]
            dp = do @ vj.T
            flat = 1 - torch.tanh(raw / cap) ** 2 if cap else torch.ones_like(raw)
            inner = dp - (do * out).sum(1, keepdim=True)
            ds = p * inner * flat
            edelta = (do.abs() * eo).sum(1, keepdim=True)
            eds = u * ds.abs() + 2 * dz * ds.abs() + p * flat * (2 * d * 2.0 ** -24 * (do.abs() @ vj.abs().T) + edelta)
            eds = eds + p * inner.abs() * 2.0 ** -21 + tiny
            for n, r, t, e in (("dq", a, ds @ kj * scale, eds @ kj.abs() * scale),):
                ref[n][r, h] = t
                tol[n][r, h] = u * t.abs() + 1.05 * e + tiny + 1e-30
            kh = h // grp
            ref["dk"][b, kh] += ds.T @ qi * scale
            tol["dk"][b, kh] += 1.05 * (eds.T @ qi.abs()) * scale
            ref["dv"][b, kh] += p.T @ do
            tol["dv"][b, kh] += 1.05 * (ep.T @ do.abs())
    if dout is not None:
        for n in ("dk", "dv"):
            tol[n] = tol[n] + u * ref[n].abs() + tiny + 1e-30
    return ref, tol


def check(got, ref, tol, what):
    for n, g in got.items():
        g = g.double().cpu()
        r, t = ref[n], tol[n]
        if n == "lse":
            assert torch.equal(torch.isinf(r), torch.isinf(g)), f"{what} lse: rows without keys"
            g, r, t = g[torch.isfinite(r)], r[torch.isfinite(r)], t[torch.isfinite(r)]
        bad = ~((g - r).abs() <= t)
        assert not bad.any(), (f"{what} {n}: {int(bad.sum())} of {bad.numel()} over tolerance, worst "
                               f"{float(((g - r).abs() / t).nan_to_num(math.inf)[bad].max()):.3g} times it")


def lengths(rng, sets, mean):
    return [int(rng.integers(0, 2 * mean + 1)) for _ in range(sets)]


def starts(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int64, device="cuda")


# name, dtype, query lengths, key lengths (None: the same rows), hq, hk, d, cap, slopes, ndim
CASES = [
    ("one_row_one_key", "f16", [1], None, 1, 1, 16, 0.0, False, 3),
    ("windows_bf16", "bf16", [70, 0, 1, 64, 65, 63, 129, 3], None, 4, 4, 32, 0.0, True, 3),
    ("windows_capped_f16", "f16", [17, 200, 16, 15], None, 2, 2, 64, 5.0, True, 2),
    ("shared_heads", "f16", [33, 100], [250, 77], 8, 2, 64, 0.0, False, 3),
    ("odd_group_odd_width", "bf16", [9, 40], [130, 61], 6, 2, 33, 4.0, True, 3),
    ("width_1", "f16", [20], None, 3, 3, 1, 0.0, False, 3),
    ("width_7", "bf16", [50, 5], None, 2, 1, 7, 0.0, True, 2),
    ("width_40", "f16", [37, 30], [300, 129], 6, 3, 40, 10.0, True, 3),
    ("width_100", "bf16", [77], [131], 2, 2, 100, 0.0, True, 3),
    ("width_128", "f16", [130, 1], None, 2, 1, 128, 10.0, True, 3),
    ("one_query_long", "f16", [1], [5000], 8, 2, 64, 0.0, True, 3),
    ("one_query_long_128", "bf16", [1, 1], [3001, 2], 4, 1, 128, 10.0, False, 3),
    ("few_queries_long", "bf16", [3, 2], [2600, 0], 5, 1, 24, 0.0, False, 3),
    ("tile_queries_long", "f16", [40], [3000], 1, 1, 32, 3.0, False, 3),
    ("long_rows_few_keys", "bf16", [4000], [5], 2, 2, 64, 0.0, True, 3),
    ("queries_without_keys", "f16", [5, 7, 3], [0, 10, 0], 2, 2, 16, 0.0, False, 3),
    ("keys_without_queries", "bf16", [0, 7], [20, 10], 2, 2, 16, 0.0, False, 3),
    ("many_sets", "f16", None, None, 2, 2, 16, 0.0, False, 3),
    ("long_two_columns", "bf16", [1500], None, 64, 64, 16, 0.0, False, 3),
    ("long_two_columns_64", "f16", [1100], None, 64, 64, 48, 6.0, True, 3),
]


def build(case, seed=0):
    name, dt, lq, lk, hq, hk, d, cap, bias, ndim = case
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16}[dt]
    rng = np.random.default_rng(seed + sum(map(ord, name)))
    if lq is None:
        lq = lengths(rng, 300, 5)
    n, m = sum(lq), sum(lq if lk is None else lk)
    gen = torch.Generator().manual_seed(seed + len(name))
    t = lambda r, h, s: (torch.randn(r, h, d, generator=gen) * s).to(dtype).cuda()  # noqa: E731
    q, k, v, dout = t(n, hq, 2.0), t(m, hk, 1.0), t(m, hk, 1.0), t(n, hq, 1.0)
    opt = dict(cap=cap)
    if bias:
        opt["slopes"] = torch.tensor([2.0 ** -(1 + h % 6) for h in range(hq)], device="cuda")
        c = lambda r: torch.randint(-20, 40, (r, ndim + 1), generator=gen, dtype=torch.int32).cuda()  # noqa: E731
        opt["q_coords"] = c(n)
        opt["k_coords"] = c(m) if lk is not None else None
    qs = starts(lq)
    ks = None if lk is None else starts(lk)
    return dtype, q, k, v, dout, qs, ks, opt


def ref_of(dtype, q, k, v, qs, ks, opt, dout=None, scale=None):
    qc = opt.get("q_coords")
    kc = opt.get("k_coords")
    return reference(q, k, v, qs.tolist(), (qs if ks is None else ks).tolist(), scale or 1 / q.shape[2] ** 0.5,
                     opt["cap"], opt.get("slopes"), qc, qc if kc is None else kc, dout, dtype)


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_attention(ts, case):
    dtype, q, k, v, dout, qs, ks, opt = build(case)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = ts.attn_fwd(q, k, v, qs, ks, err_flags=flags, **opt)
    dq, dk, dv = ts.attn_bwd(dout, q, k, v, out, lse, qs, ks, err_flags=flags, **opt)
    ref, tol = ref_of(dtype, q, k, v, qs, ks, opt, dout)
    check({"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, ref, tol, case[0])
    assert int(flags) == 0
    # the same bits again
    out2, lse2 = ts.attn_fwd(q, k, v, qs, ks, **opt)
    again = ts.attn_bwd(dout, q, k, v, out2, lse2, qs, ks, **opt)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), again))


@pytest.mark.parametrize("case", [CASES[1], CASES[7], CASES[4]], ids=lambda c: c[0])
def test_gradient_against_differences(ts, case):
    """<grad, direction> against central differences of the fp64 forward."""
    dtype, q, k, v, dout, qs, ks, opt = build(case, seed=5)
    out, lse = ts.attn_fwd(q, k, v, qs, ks, **opt)
    grads = ts.attn_bwd(dout, q, k, v, out, lse, qs, ks, **opt)
    _, tol = ref_of(dtype, q, k, v, qs, ks, opt, dout)
    gen = torch.Generator().manual_seed(3)
    h = 1e-5
    for n, (i, g) in zip(("dq", "dk", "dv"), enumerate(grads)):
        base = [q.double().cpu(), k.double().cpu(), v.double().cpu()]
        way = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        side = []
        for s in (h, -h):
            x = list(base)
            x[i] = base[i] + s * way
            r, _ = ref_of(dtype, *x, qs, ks, opt)
            side.append(float((r["out"] * dout.double().cpu()).sum()))
        got = float((g.double().cpu() * way).sum())
        # elementwise bounds along the direction; the difference itself is good to h^2
        bound = float((tol[n] * way.abs()).sum()) + 1e-6 * abs(got) + 1e-5
        assert abs(got - (side[0] - side[1]) / (2 * h)) <= bound, (n, got, side, bound)


@pytest.mark.parametrize("d", [32, 40, 33])
def test_columns_of_one_matrix(ts, d):
    """q, k, v as columns of one projected matrix, rows a stride apart, also
    where that leaves them unaligned."""
    n, h = 150, 3
    gen = torch.Generator().manual_seed(d)
    for pad in (0, 1, 8):
        m = torch.randn(n, 3 * h * d + pad, generator=gen).half().cuda()
        q, k, v = (m[:, i * h * d:(i + 1) * h * d].unflatten(1, (h, d)) for i in range(3))
        qs = starts([100, 50])
        dout = torch.randn(n, h, d, generator=gen).half().cuda()
        out, lse = ts.attn_fwd(q, k, v, qs)
        dq, dk, dv = ts.attn_bwd(dout, q, k, v, out, lse, qs)
        assert dq.stride(0) == m.shape[1]
        ref, tol = ref_of(torch.float16, q, k, v, qs, None, {"cap": 0.0}, dout)
        check({"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, ref, tol, f"columns d={d} pad={pad}")
        # a gradient of out that is not dense
        wide = torch.randn(n, 2 * h * d, generator=gen).half().cuda()[:, :h * d].unflatten(1, (h, d))
        a = ts.attn_bwd(wide, q, k, v, out, lse, qs)
        b = ts.attn_bwd(wide.contiguous(), q, k, v, out, lse, qs)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_outside_every_set(ts):
    """Starts that leave rows at both ends uncovered (buffers with spare rows):
    zeros there, and NaN in them reaches no other row."""
    n, h, d = 200, 2, 32
    gen = torch.Generator().manual_seed(1)
    q, k, v, dout = (torch.randn(n, h, d, generator=gen).half().cuda() for _ in range(4))
    for t in (q, k, v, dout):
        t[:10] = math.nan
        t[150:] = math.inf
    qs = torch.tensor([10, 60, 60, 150], device="cuda")
    out, lse = ts.attn_fwd(q, k, v, qs)
    dq, dk, dv = ts.attn_bwd(dout, q, k, v, out, lse, qs)
    spare = torch.cat([torch.arange(10), torch.arange(150, n)]).cuda()
    for t in (out, dq, dk, dv):
        assert (t[spare] == 0).all()
    assert (lse[spare] == -math.inf).all()
    inner = slice(10, 150)
    ref, tol = reference(q[inner], k[inner], v[inner], [0, 50, 50, 140], [0, 50, 50, 140], d ** -0.5, dout=dout[inner])
    got = {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    check({n_: t[inner] for n_, t in got.items()}, ref, tol, "inner rows")


def test_neighbouring_sets_do_not_leak(ts):
    """A set's NaN, and tiles that end inside it, leave the sets beside it alone."""
    lq, h, d = [5, 70, 3, 64, 10], 2, 64
    gen = torch.Generator().manual_seed(2)
    q, k, v, dout = (torch.randn(sum(lq), h, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(4))
    qs = starts(lq)
    clean = ts.attn_fwd(q, k, v, qs)
    clean = (clean[0], *ts.attn_bwd(dout, q, k, v, *clean, qs))
    for t in (q, k, v):
        t[75:78] = math.nan  # the third set
    bad = ts.attn_fwd(q, k, v, qs)
    bad = (bad[0], *ts.attn_bwd(dout, q, k, v, *bad, qs))
    rest = torch.cat([torch.arange(75), torch.arange(78, sum(lq))]).cuda()
    for a, b in zip(clean, bad):
        assert torch.equal(a[rest], b[rest])
        assert b[75:78].isnan().all()


def test_infinite_scores(ts):
    """-inf scores drop their keys; a row of nothing else is a row without keys."""
    d = 16
    q = torch.zeros(2, 1, d, dtype=torch.float16, device="cuda")
    k = torch.zeros(40, 1, d, dtype=torch.float16, device="cuda")
    v = torch.randn(40, 1, d, generator=torch.Generator().manual_seed(1)).half().cuda()
    q[:, :, 0] = 1.0
    k[:, 0, 0] = -math.inf
    k[7, 0, 0] = 0.0
    qs, ks = torch.tensor([0, 2], device="cuda"), torch.tensor([0, 40], device="cuda")
    out, lse = ts.attn_fwd(q, k, v, qs, ks)
    assert torch.equal(out[0, 0], v[7, 0]) and float(lse[0, 0]) == 0.0
    k[7, 0, 0] = -math.inf
    out, lse = ts.attn_fwd(q, k, v, qs, ks)
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = ts.attn_bwd(torch.ones_like(q), q, k, v, out, lse, qs, ks)
    assert (dv == 0).all()


def test_large_scores_and_rising_maxima(ts):
    """Scores far beyond exp's range whose maximum rises from tile to tile."""
    n, d = 700, 32
    q = torch.ones(3, 1, d, dtype=torch.bfloat16, device="cuda") * 4
    k = (torch.linspace(-20, 20, n, device="cuda")[:, None, None] * torch.ones(1, 1, d, device="cuda")).to(torch.bfloat16)
    v = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    dout = torch.randn(3, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    qs, ks = torch.tensor([0, 3], device="cuda"), torch.tensor([0, n], device="cuda")
    for kk in (k, k.flip(0).contiguous()):
        out, lse = ts.attn_fwd(q, kk, v, qs, ks)
        got = dict(zip(("dq", "dk", "dv"), ts.attn_bwd(dout, q, kk, v, out, lse, qs, ks)), out=out, lse=lse)
        ref, tol = ref_of(torch.bfloat16, q, kk, v, qs, ks, {"cap": 0.0}, dout)
        check(got, ref, tol, "rising")


def test_far_coordinates(ts):
    """Distances over the whole packable range, whose squares pass 24 bits."""
    n, h, d = 130, 2, 32
    gen = torch.Generator().manual_seed(4)
    q, k, v, dout = (torch.randn(n, h, d, generator=gen).half().cuda() for _ in range(4))
    c = torch.randint(-32768, 32768, (n, 4), generator=gen, dtype=torch.int32)
    c[1::2, 1:] = c[::2, 1:] + torch.randint(-2, 3, (n // 2, 3), generator=gen, dtype=torch.int32)  # near pairs far out
    opt = dict(cap=0.0, slopes=torch.tensor([1e-4, 1.0], device="cuda"), q_coords=c.cuda())
    qs = starts([n])
    out, lse = ts.attn_fwd(q, k, v, qs, **opt)
    got = dict(zip(("dq", "dk", "dv"), ts.attn_bwd(dout, q, k, v, out, lse, qs, **opt)), out=out, lse=lse)
    ref, tol = ref_of(torch.float16, q, k, v, qs, None, opt, dout)
    check(got, ref, tol, "far")


def test_empty(ts):
    z = lambda n, h=2: torch.zeros(n, h, 16, dtype=torch.float16, device="cuda")  # noqa: E731
    no = torch.zeros(1, dtype=torch.int64, device="cuda")  # no sets
    out, lse = ts.attn_fwd(z(0), z(0), z(0), no)
    assert out.shape == (0, 2, 16) and lse.shape == (0, 2)
    q = z(3) + 1
    out, lse = ts.attn_fwd(q, z(0), z(0), torch.tensor([0, 3], device="cuda"), torch.tensor([0, 0], device="cuda"))
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = ts.attn_bwd(q, q, z(0), z(0), out, lse, torch.tensor([0, 3], device="cuda"),
                             torch.tensor([0, 0], device="cuda"))
    assert (dq == 0).all() and dk.shape[0] == 0
    dq, dk, dv = ts.attn_bwd(z(0), z(0), q, q, z(0), lse[:0], torch.tensor([0, 0], device="cuda"),
                             torch.tensor([0, 3], device="cuda"))
    assert (dk == 0).all() and (dv == 0).all()
    out, lse = ts.attn_fwd(q, q, q, no)  # rows, but no set
    assert (out == 0).all()


def test_bad_starts_raise_the_flag(ts):
    q = torch.randn(64, 1, 16, generator=torch.Generator().manual_seed(1)).half().cuda()
    for bad in ([0, 40, 30, 64], [0, 65], [-1, 64], [5, 3]):
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        s = torch.tensor(bad, device="cuda")
        ts.attn_fwd(q, q, q, s, err_flags=flags)
        assert int(flags) == ts.TS_FLAG_RANGE, bad
    for good in ([0, 64], [0, 0, 64, 64], [3, 60]):
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        ts.attn_fwd(q, q, q, torch.tensor(good, device="cuda"), err_flags=flags)
        assert int(flags) == 0, good


def test_other_stream(ts):
    """A call on a stream that is not the current one."""
    dtype, q, k, v, dout, qs, ks, opt = build(CASES[10])
    ref = ts.attn_fwd(q, k, v, qs, ks, **opt)
    refb = ts.attn_bwd(dout, q, k, v, *ref, qs, ks, **opt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = ts.attn_fwd(q, k, v, qs, ks, stream=s, **opt)
        back = ts.attn_bwd(dout, q, k, v, *got, qs, ks, stream=s, **opt)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *back), (*ref, *refb)))


def test_refusals(ts):
    h = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    s = torch.tensor([0, 8], device="cuda")
    q = h(8, 4, 16)

    def refused(status, *a, **kw):
        with pytest.raises(ts.TsError) as e:
            ts.attn_fwd(*a, **kw)
        assert e.value.status == status

    refused(ts.TS_ERR_UNSUPPORTED, q.float(), q.float(), q.float(), s)
    refused(ts.TS_ERR_UNSUPPORTED, h(8, 1, 136), h(8, 1, 136), h(8, 1, 136), s)
    refused(ts.TS_ERR_INVALID_ARG, q, h(8, 3, 16), h(8, 3, 16), s)         # 3 does not divide 4
    refused(ts.TS_ERR_INVALID_ARG, q, h(9, 4, 16), h(9, 4, 16), s)         # other keys, no k_starts
    refused(ts.TS_ERR_INVALID_ARG, q, q, h(8, 4, 24), s)
    refused(ts.TS_ERR_INVALID_ARG, q, q, q.bfloat16(), s)
    refused(ts.TS_ERR_INVALID_ARG, q, q, q, s.int())
    refused(ts.TS_ERR_INVALID_ARG, q, q, q, s, cap=-1.0)
    refused(ts.TS_ERR_INVALID_ARG, q, q, q, s, cap=math.nan)
    refused(ts.TS_ERR_INVALID_ARG, q, q, q, s, scale=math.inf)
    refused(ts.TS_ERR_INVALID_ARG, q, q, q, s, slopes=torch.zeros(4, device="cuda"))
    refused(ts.TS_ERR_INVALID_ARG, q.transpose(1, 2), q.transpose(1, 2), q.transpose(1, 2), s)
    refused(ts.TS_ERR_INVALID_ARG, q[:1].expand(8, 4, 16), q, q, s)        # rows that share their memory
    refused(ts.TS_ERR_INVALID_ARG, q.cpu(), q, q, s)
    at = ts.attn_args(q, h(9000, 4, 16), h(9000, 4, 16), s, torch.tensor([0, 9000], device="cuda"))
    assert ts.ts_attn_workspace_bytes(at, False) > 0
    with pytest.raises(ts.TsError):  # no workspace
        ts.ts_attn_fwd(at, q, h(9000, 4, 16), h(9000, 4, 16), torch.empty_like(q), torch.empty(8, 4, device="cuda"))


@pytest.mark.parametrize("nq,cap", [(1, 0.0), (1, 6.0), (40, 0.0)])
def test_one_key_has_no_score_gradient(ts, nq, cap):
    """With one key a softmax is constant: dq and dk are 0.  The sum of p (dp - delta) that a row's delta is
    corrected by is formed in fp32, p = exp(z - lse) is 1 to 2^-19 (z, lse below 32) and dp below |dout| |v|, so what
    is left of ds is below 2^-18 |dout| |v|; from the rounded out alone it would be 2^-12 of it."""
    d, n = 32, 50
    g = torch.Generator("cuda").manual_seed(77)
    q, dout = (torch.randn(n * nq, 1, d, generator=g, device="cuda").half() for _ in range(2))
    k, v = (torch.randn(n, 1, d, generator=g, device="cuda").half() for _ in range(2))
    qs = torch.arange(0, n * nq + 1, nq, device="cuda")
    ks = torch.arange(0, n + 1, device="cuda")
    out, lse = ts.attn_fwd(q, k, v, qs, ks, cap=cap)
    dq, dk, _ = ts.attn_bwd(dout, q, k, v, out, lse, qs, ks, cap=cap)
    largest = float(dout.float().norm(dim=2).max() * v.float().norm(dim=2).max())
    bar = 2.0 ** -18 * largest * d ** -0.5
    assert float(dq.float().abs().max()) <= bar * float(k.float().abs().max()) + 2.0 ** -25
    assert float(dk.float().abs().max()) <= nq * bar * float(q.float().abs().max()) + 2.0 ** -25


def test_offsets_past_32_bits(ts):
    """Rows 2^20 elements apart, 3000 of them (6 GiB a tensor): the bits of the same rows side by side."""
    n, hq, hk, d, stride = 3000, 4, 2, 32, 1 << 20
    g = torch.Generator("cuda").manual_seed(55)
    dense = [torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for h in (hq, hk, hk, hq)]
    far = [torch.empty(n * stride, dtype=torch.bfloat16, device="cuda").as_strided(t.shape, (stride, d, 1)) for t in dense]
    for t, s in zip(far, dense):
        t.copy_(s)
    starts = torch.tensor([0, 40, 2900, n], device="cuda")
    results = []
    for q, k, v, dout in (dense, far):
        out, lse = ts.attn_fwd(q, k, v, starts)
        results.append((out, lse, *ts.attn_bwd(dout, q, k, v, out, lse, starts)))
    for a, b in zip(*results):
        assert torch.equal(a, b)
