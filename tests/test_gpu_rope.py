"""GPU parity of the query and key rotation with its norm, forward and backward,
against plain fp64 implementations; gradients also against differences.

Tolerances from the roundings, E = 2^-24 (fp32), u the result's type (0, 2^-11, 2^-8):
a sum of m terms is off by at most m E of the sum of their magnitudes, sine and cosine
by 2 E, and each of the few products around them by E of itself.  So with d terms in
the norm: results by u |y| + (d + 16) E of the magnitudes that enter them."""
import numpy as np
import pytest
import torch

import bench
from helpers import U_OUT

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol, what):
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), f"{what}: {(~(err <= tol)).sum()} of {err.size} over tolerance, worst {np.nanmax(err / tol):.3g} times it"


def turn(x, angle, il, sign=1.0):
    """x [n][h][d] turned by angle [n][P], and what its results' magnitudes are bounded by."""
    p, out, mag = angle.shape[1], x.copy(), np.abs(x)
    a = np.arange(p) * 2 if il else np.arange(p)
    b = a + 1 if il else a + p
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None] * sign
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return out, mag


def angles(coords, freqs, pairs):
    axis = np.repeat(np.arange(len(pairs)), pairs) + 1
    return coords.cpu().numpy()[:, axis].astype(np.float64) * freqs.cpu().numpy().astype(np.float64)


def check(ts, dt, q, k, coords, freqs, pairs, wq, wk, il, dq, dk, eps=1e-6, **kw):
    u = U_OUT[DT[dt]]
    tiny = 2.0 ** -25 if dt == "f16" else 1e-37
    angle = angles(coords, freqs, pairs) if sum(pairs) else np.zeros((q.shape[0], 0))
    y = ts.rope_fwd(q, k, coords, freqs, pairs, wq=wq, wk=wk, eps=eps, interleaved=il, **kw)
    r = ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, wq=wq, wk=wk, eps=eps, interleaved=il, **kw)
    for what, x, w, got, g, dx, dw in (("q", q, wq, y[0], dq, r.dq, r.dwq), ("k", k, wk, y[1], dk, r.dk, r.dwk)):
        if x is None:
            assert got is None and dx is None and dw is None
            continue
        x, g = f64(x), f64(g)
        n, h, d = x.shape
        ww = np.ones(d) if w is None else f64(w)
        rstd = 1.0 if w is None else 1 / np.sqrt((x * x).mean(2, keepdims=True) + eps)
        ref, mag = turn(x * rstd * ww, angle, il)
        close(got, ref, u * np.abs(ref) + (d + 16) * E * mag + tiny, what)
        g, gmag = turn(g, angle, il, -1.0)
        if w is None:
            assert dw is None
            close(dx, g, u * np.abs(g) + 16 * E * gmag + tiny, "d" + what)
            continue
        xn = x * rstd
        ref = rstd * (g * ww - xn * (g * ww * xn).mean(2, keepdims=True))
        mag = rstd * (gmag * np.abs(ww) + np.abs(xn) * (gmag * np.abs(ww * xn)).mean(2, keepdims=True))
        close(dx, ref, u * np.abs(ref) + (2 * d + 32) * E * mag + tiny, "d" + what)
        close(dw, (g * xn).sum((0, 1)), (n * h + d + 32) * E * (gmag * np.abs(xn)).sum((0, 1)) + tiny, "dw" + what)
    return y, r


def inputs(dt, n, hq, hk, d, pairs, norm=True, seed=0, reach=3000):
    g = torch.Generator().manual_seed(seed + 1000 * n + d)
    dtype = DT[dt]
    m = (torch.randn(n, hq + 2 * hk, d, generator=g) * 2).to(dtype).cuda()
    q, k, _ = m.split((hq, hk, hk), 1)
    coords = torch.randint(-reach, reach, (n, len(pairs) + 1), generator=g, dtype=torch.int32).cuda()
    freqs = torch.cat([10.0 ** (-torch.arange(p) / max(p, 1)) for p in pairs]).cuda() if sum(pairs) else None
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).cuda() if norm else None for _ in range(2))
    dq, dk = (torch.randn(n, h, d, generator=g).to(dtype).cuda() for h in (hq, hk))
    return q, k if hk else None, coords, freqs, pairs, wq, wk if hk else None, dq, dk if hk else None


SHAPES = [  # n, hq, hk, d, pairs
    (1, 1, 1, 1, (0, 0)), (3, 2, 1, 2, (1, 0)), (5, 1, 2, 3, (0, 1)), (39, 2, 2, 16, (4, 4)), (39, 2, 2, 16, (3, 3, 2)),
    (257, 3, 1, 17, (4, 2, 2)), (100, 4, 2, 24, (4, 4, 4)), (65, 6, 3, 40, (6, 6, 4)), (70, 8, 8, 64, (11, 11, 10)),
    (33, 5, 1, 77, (38, 0)), (31, 3, 3, 80, (14, 13, 13)), (41, 2, 1, 96, (0, 0, 0)), (20, 16, 4, 128, (22, 21, 21)),
    (9, 1, 1, 128, (0, 0, 1)), (9, 2, 2, 127, (1, 2, 3)), (300, 1, 0, 32, (5, 5)), (2, 700, 3, 8, (2, 2)), (0, 4, 2, 32, (8, 8)),
    (7, 3, 2, 10, (2, 1)), (1300, 1, 1, 16, (4, 4)), (40000, 4, 4, 32, (6, 6, 4)), (12000, 1, 1, 18, (3, 3, 3)),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("il", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope(ts, shape, il, dt):
    n, hq, hk, d, pairs = shape
    for norm in (True, False):
        q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs(dt, n, hq, hk, d, pairs, norm)
        check(ts, dt, q, k, coords, freqs, pairs, wq, wk, il, dq, dk)


@pytest.mark.parametrize("n", [2, 1500, 70000])
@pytest.mark.parametrize("il,d,pairs", [(False, 4, (1, 0)), (False, 5, (0, 0, 1)), (True, 2, (0, 1)), (True, 3, (1, 0))])
def test_one_pair(ts, n, il, d, pairs):
    """A head with a single pair of channels to turn, in tiles of one row and of many."""
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs("f32", n, 2, 1, d, pairs)
    check(ts, "f32", q, k, coords, freqs, pairs, wq, wk, il, dq, dk)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("il", [False, True])
def test_single_channel(ts, dt, il):
    """Heads of one channel, which have no pair: many rows, and what lies around the results stays."""
    n = 1500
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs(dt, n, 3, 2, 1, (0, 0))
    y, r = check(ts, dt, q, k, coords, freqs, pairs, wq, wk, il, dq, dk)
    for f, want in ((lambda into: ts.rope_fwd(q, k, coords, freqs, pairs, wq=wq, wk=wk, interleaved=il, into=into), y),
                    (lambda into: ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, wq=wq, wk=wk, interleaved=il, into=into), (r.dq, r.dk))):
        band = torch.full((n + 2, 9, 1), 7.0, dtype=DT[dt], device="cuda")
        f((band[1:-1, 1:4], band[1:-1, 5:7]))
        assert torch.equal(band[1:-1, 1:4], want[0]) and torch.equal(band[1:-1, 5:7], want[1])
        band[1:-1, 1:4], band[1:-1, 5:7] = 7.0, 7.0
        assert (band == 7).all()


@pytest.mark.parametrize("reach", [2 ** 15, 2 ** 31 - 1])
def test_far_positions(ts, reach):
    """Angles of positions over all of int32: the reference's own product is off by 2^-53 of an angle of up to
    2^31 and the kernel's by twice that more, 2^-20 in all at the largest, which is added to sine's and cosine's error."""
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs("f32", 200, 2, 2, 32, (8, 8), True, 5, reach)
    y = ts.rope_fwd(q, k, coords, freqs, pairs)
    angle = angles(coords, freqs, pairs)
    for x, got in ((q, y[0]), (k, y[1])):
        ref, mag = turn(f64(x), angle, False)
        close(got, ref, (16 * E + 4 * 2.0 ** -53 * reach) * mag, "far")


def test_special_values(ts):
    """A row of zeros, infinite and NaN elements, and tiny ones with eps 0: as the formulas have it, and other rows are
    not touched by them."""
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs("f32", 60, 2, 1, 32, (8, 8))
    q = q.clone()
    want = ts.rope_fwd(q, k, coords, freqs, pairs, wq=wq, wk=wk)[0]
    q[3], q[5, 0, 7], q[8, 1, 31] = 0.0, float("nan"), float("inf")
    got = ts.rope_fwd(q, k, coords, freqs, pairs, wq=wq, wk=wk)[0]
    assert (got[3] == 0).all() and got[5, 0].isnan().all() and got[8, 1, 31].isnan()
    for r, h in ((5, 0), (8, 1)):
        got[r, h] = want[r, h]
    got[3] = want[3]
    assert torch.equal(got, want)
    small = (q[:2] * 1e-17).contiguous()
    r = check(ts, "f32", small, None, coords[:2].contiguous(), freqs, pairs, wq, None, False, dq[:2], None, eps=0.0)
    assert r[0][0].abs().max() > 0.1


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("d,pairs", [(32, (6, 6, 4)), (26, (3, 3, 3)), (40, (10, 10))])
def test_in_place_and_columns(ts, d, pairs, il):
    """Written over q and k within the projected matrix (the values beside them stay), gradients over dq and dk."""
    n, hq, hk = 333, 4, 2
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs("bf16", n, hq, hk, d, pairs)
    kw = dict(wq=wq, wk=wk, interleaved=il)
    want = ts.rope_fwd(q, k, coords, freqs, pairs, **kw)
    grads = ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, **kw)
    again = ts.rope_bwd(dq.clone(), dk.clone(), q, k, coords, freqs, pairs, **kw)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))  # the same bits on every run
    wide = torch.randn(n, hq + 2 * hk, d, device="cuda").bfloat16()
    gq, gk, gv = wide.split((hq, hk, hk), 1)
    gq.copy_(dq)
    gk.copy_(dk)
    beside = gv.clone()
    got = ts.rope_bwd(gq, gk, q, k, coords, freqs, pairs, into=(gq, gk), **kw)
    assert torch.equal(gq, grads.dq) and torch.equal(gk, grads.dk) and torch.equal(gv, beside)
    assert torch.equal(got.dwq, grads.dwq) and torch.equal(got.dwk, grads.dwk)
    m = torch.empty(n, hq + 2 * hk, d, device="cuda", dtype=torch.bfloat16)
    a, b, c = m.split((hq, hk, hk), 1)
    a.copy_(q)
    b.copy_(k)
    c.copy_(beside)
    ts.rope_fwd(a, b, coords, freqs, pairs, into=(a, b), **kw)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, beside)


def test_rows_past_32_bit_offsets(ts):
    """Rows further apart than 2^31 elements in all: the last ones are read and written where they lie."""
    n, stride = 5, 1 << 29
    m = torch.empty((n - 1) * stride + 64, device="cuda", dtype=torch.float16)
    q = m.as_strided((n, 2, 32), (stride, 32, 1))
    data = torch.randn(n, 2, 32, device="cuda").half()
    q.copy_(data)
    coords = torch.arange(n * 3, device="cuda", dtype=torch.int32).view(n, 3)
    freqs = ts.rope_freqs((8, 8))
    w = torch.full((32,), 1.5, device="cuda")
    want = ts.rope_fwd(data, None, coords, freqs, (8, 8), wq=w)[0]
    ts.rope_fwd(q, None, coords, freqs, (8, 8), wq=w, into=(q, None))
    assert torch.equal(q, want)


def test_gradient_against_differences(ts):
    """Central differences in fp32: step h = 2^-6 on values of about 1 with third derivatives of at most about 10
    leaves h^2 10 / 6 = 4e-4 and 2^-24 * 64 terms * 8 / h = 2e-3 relative to a loss of terms of about 1."""
    q, _, coords, freqs, pairs, wq, _, dq, _ = inputs("f32", 4, 1, 0, 16, (4, 4), reach=20)
    q, h = q.contiguous(), 2.0 ** -6
    loss = lambda x, w: float((ts.rope_fwd(x, None, coords, freqs, pairs, wq=w)[0].double() * dq.double()).sum())
    r = ts.rope_bwd(dq, None, q, None, coords, freqs, pairs, wq=wq)
    for at in range(0, q.numel(), 7):
        e = torch.zeros_like(q).view(-1)
        e[at] = h
        e = e.view_as(q)
        assert abs((loss(q + e, wq) - loss(q - e, wq)) / (2 * h) - float(r.dq.reshape(-1)[at])) < 5e-3
    for at in range(16):
        e = torch.zeros_like(wq)
        e[at] = h
        assert abs((loss(q, wq + e) - loss(q, wq - e)) / (2 * h) - float(r.dwq[at])) < 5e-3


def test_scores_depend_on_differences_only(ts):
    """What the rotation is for: moving every voxel by the same vector leaves the products of queries and keys."""
    q, k, coords, freqs, pairs, wq, wk, *_ = inputs("f32", 50, 2, 2, 32, (6, 6, 4), reach=100)
    moved = coords + torch.tensor([0, 1000, -777, 31], device="cuda", dtype=torch.int32)
    score = lambda c: torch.matmul(*(f(t) for f, t in zip((lambda a: a.double().transpose(0, 1), lambda b: b.double().permute(1, 2, 0).contiguous()),
                                                          ts.rope_fwd(q, k, c, freqs, pairs, wq=wq, wk=wk))))
    a, b = score(coords), score(moved)
    assert float((a - b).abs().max()) <= 64 * 64 * E * float(a.abs().max())


def test_stream_and_graph(ts):
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs("bf16", 5000, 4, 2, 32, (6, 6, 4))
    kw = dict(wq=wq, wk=wk)
    flat = lambda y, r: [*y, *r]
    want = flat(ts.rope_fwd(q, k, coords, freqs, pairs, **kw), ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, **kw))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = flat(ts.rope_fwd(q, k, coords, freqs, pairs, stream=side, **kw), ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, stream=side, **kw))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    held = []

    def step():
        held[:] = flat(ts.rope_fwd(q, k, coords, freqs, pairs, **kw), ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, **kw))
    graph = bench.capture([step])
    for _ in range(3):
        for t in held:
            t.fill_(-7)
        torch.randn(512, 512, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_refusals(ts):
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs("f16", 20, 2, 1, 32, (8, 8))
    bad = [dict(pairs=(9, 8)), dict(pairs=(-1, 8)), dict(pairs=(8,)), dict(coords=coords.long()), dict(coords=coords[:-1]),
           dict(freqs=freqs[:-1]), dict(freqs=None), dict(k=k.float()), dict(k=k[:-1]), dict(q=q.transpose(0, 1)),
           dict(wq=wq[:-1]), dict(wq=wq.half()), dict(eps=-1.0), dict(eps=float("nan")), dict(into=(None, None)),
           dict(into=(q.float(), k)), dict(q=q.cpu())]
    for change in bad:
        args = dict(dict(q=q, k=k, coords=coords, freqs=freqs, pairs=pairs, wq=wq, wk=wk), **change)
        with pytest.raises(ts.TsError):
            ts.rope_fwd(**args)
        with pytest.raises(ts.TsError):
            ts.rope_bwd(dq, dk, **args)
    with pytest.raises(ts.TsError):
        ts.rope_bwd(dq, None, q, k, coords, freqs, pairs)
    wide = torch.zeros(4, 1, 136, device="cuda")
    with pytest.raises(ts.TsError) as e:
        ts.rope_fwd(wide, None, None, None, (0, 0))
    assert e.value.status == ts.TS_ERR_UNSUPPORTED
