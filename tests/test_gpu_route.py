"""GPU parity of the router and of the combining sum, forward and backward, against
plain fp64 implementations.  Experts, starts, rows and places are exact.

Tolerances, E = 2^-24: a gate is exp of a difference d of two logits over a sum of m such
terms: off by (|d| + m + 8) E of itself (the difference is rounded once, exp is off by 2 E);
sums of m products by (m + 8) E of their magnitudes; results by u of themselves besides."""
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


def route(z, top):
    """experts, starts, rows, place of logits z [n][e] in fp64."""
    n, e = z.shape
    order = np.argsort(-z, axis=1, kind="stable")[:, :top]
    none = np.take_along_axis(z, order, 1) == -np.inf
    experts = np.where(none, -1, order)
    flat = np.where(none, e, order).reshape(-1)
    by = np.argsort(flat, kind="stable")
    starts = np.searchsorted(flat[by], np.arange(e + 1))
    rows = np.where(flat[by] == e, -1, by // top)
    place = np.empty(n * top, np.int64)
    place[by] = np.arange(n * top)
    return experts, starts, rows, np.where(none, -1, place.reshape(n, top))


def check(ts, z, top, over_all):
    zz = f64(z)
    n, e = zz.shape
    r = ts.route_fwd(z, top, over_all=over_all)
    experts, starts, rows, place = route(zz, top)
    for got, ref in ((r.experts, experts), (r.starts, starts), (r.rows, rows), (r.place, place)):
        assert np.array_equal(got.cpu().numpy(), ref)
    picked = experts >= 0
    best = np.take_along_axis(zz, np.maximum(experts, 0), 1)
    with np.errstate(invalid="ignore"):
        far = np.where(picked, best - best[:, :1], 0.0)
        p = np.exp(zz - best[:, :1]) if over_all else np.where(picked, np.exp(far), 0.0)
    p = np.where(picked[:, :1], p, 0.0)
    total = np.maximum(p.sum(1, keepdims=True), 1e-300)
    gates = np.where(picked, np.exp(far), 0.0) / total
    close(r.gates, gates, gates * (np.abs(far) + e + 16) * E + 1e-40, "gates")
    dg = torch.randn(n, top, generator=torch.Generator().manual_seed(n + e), dtype=torch.float32).cuda()
    d = ts.route_bwd(dg, z, r, over_all=over_all)
    g = np.where(picked, f64(dg), 0.0)
    inner, size = (gates * g).sum(1, keepdims=True), (gates * np.abs(g)).sum(1, keepdims=True)
    ref, mag = np.zeros_like(zz), np.zeros_like(zz)
    at = np.nonzero(picked)
    ref[at[0], experts[at]] = (gates * (g if over_all else g - inner))[at]
    mag[at[0], experts[at]] = (gates * (np.abs(g) + size))[at]
    if over_all:
        ref -= p / total * inner
        mag += p / total * size
    spread = np.abs(np.where(np.isfinite(zz), zz - np.where(picked[:, :1], best[:, :1], 0.0), 0.0)).max() if n else 0.0
    u = U_OUT[z.dtype]
    close(d, ref, u * np.abs(ref) + mag * (2 * spread + 2 * e + 2 * top + 32) * E + (2.0 ** -25 if z.dtype == torch.float16 else 1e-37), "dlogits")
    return r


SHAPES = [(1, 1, 1), (1, 8, 2), (39, 8, 2), (40, 7, 7), (1000, 9, 1), (5, 512, 16), (129, 512, 16), (64, 65, 3), (3000, 16, 16),
          (2048, 31, 1), (2049, 32, 1), (20011, 64, 2), (9000, 200, 8), (30000, 3, 2), (70000, 8, 1), (0, 8, 2)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_route(ts, shape, dt):
    n, e, top = shape
    g = torch.Generator().manual_seed(n + 7 * e + top)
    z = (2 * torch.randn(n, e, generator=g)).to(DT[dt])
    lean = z + torch.linspace(3, -3, e).to(DT[dt])
    for over_all in (False, True):
        check(ts, z.cuda(), top, over_all)
        check(ts, lean.cuda(), top, over_all)


@pytest.mark.parametrize("n", [50, 6000])
@pytest.mark.parametrize("over_all", [False, True])
def test_ties_and_masks(ts, n, over_all):
    """Equal logits (0 and -0 among them), experts that are never picked, rows that nothing is left of."""
    e, top = 20, 4
    g = torch.Generator().manual_seed(n)
    z = torch.randint(-2, 3, (n, e), generator=g).float()
    z[z == 0] *= torch.where(torch.rand(int((z == 0).sum()), generator=g) < 0.5, 1.0, -1.0)
    check(ts, z.cuda(), top, over_all)
    z[:, 3] = z[:, 11] = -torch.inf
    z[::7] = -torch.inf
    z[3::7, 2:] = -torch.inf
    z[5::7] = torch.finfo(torch.float32).min
    r = check(ts, z.cuda(), top, over_all)
    assert (r.experts[0] == -1).all() and (r.gates[0] == 0).all() and (r.experts[3, 2:] == -1).all()
    assert int(r.starts[-1]) < n * top and (r.rows[int(r.starts[-1]):] == -1).all()
    check(ts, torch.full((n, e), -torch.inf).cuda(), top, over_all)


def test_nan_and_infinity(ts):
    """They rank as largest and make their own row's gates NaN, no other's."""
    z = torch.randn(300, 12)
    want = ts.route_fwd(z.cuda(), 2)
    z[4, 5], z[9, 7] = float("nan"), float("inf")
    for over_all in (False, True):
        r = ts.route_fwd(z.cuda(), 2, over_all=over_all)
        assert int(r.experts[4, 0]) == 5 and int(r.experts[9, 0]) == 7
        assert r.gates[4].isnan().all() and r.gates[9].isnan().any()
        rest = [i for i in range(300) if i not in (4, 9)]
        assert not r.gates[rest].isnan().any() and torch.equal(r.experts[rest], want.experts[rest])


def test_route_stream_and_graph(ts):
    z, dg = torch.randn(20000, 24, device="cuda"), torch.randn(20000, 3, device="cuda")
    few, dfew = z[:100].contiguous(), dg[:100].contiguous()

    def both():
        r, s = ts.route_fwd(z, 3), ts.route_fwd(few, 3, over_all=True)
        return [*r, *s, ts.route_bwd(dg, z, r), ts.route_bwd(dfew, few, s, over_all=True)]
    want, held = both(), []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ts.route_fwd(z, 3, stream=side)
    back = ts.route_bwd(dg, z, got, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(back, want[10])

    def step():
        held[:] = both()
    graph = bench.capture([step])
    for _ in range(3):
        for t in held:
            t.fill_(-7)
        torch.randn(512, 512, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


# ---------------------------------------------------------------- the combining sum
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(1, 1, 1), (37, 2, 64), (100, 3, 77), (65, 5, 8), (33, 16, 33), (50, 2, 512), (40, 4, 520),
                                   (11, 6, 2100), (9000, 2, 128), (20, 9, 7), (0, 2, 16)], ids=str)
def test_combine(ts, shape, dt):
    n, top, c = shape
    g = torch.Generator().manual_seed(n * 31 + c)
    dtype, u = DT[dt], U_OUT[DT[dt]]
    p = n * top + 3
    place = torch.randperm(p, generator=g)[:n * top].int().view(n, top)
    if n > 1:
        place[torch.rand(n, top, generator=g) < 0.2] = -1
        place[1] = -1
    y, dout = (torch.randn(m, c, generator=g).to(dtype) for m in (p, n))
    gates = torch.randn(n, top, generator=g)
    used = place >= 0
    at = torch.where(used, place, 0).long()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    tiny = 2.0 ** -25 if dt == "f16" else 1e-37
    for w in (gates, None):
        full = np.where(used.numpy(), f64(w) if w is not None else 1.0, 0.0)[:, :, None]
        ref = (full * f64(y)[at.numpy()]).sum(1)
        mag = np.abs(full * f64(y)[at.numpy()]).sum(1)
        got = ts.combine_fwd(y.cuda(), place.cuda(), None if w is None else w.cuda(), err_flags=flags)
        close(got, ref, u * np.abs(ref) + (top + 2) * E * mag + tiny, "out")
    mark = torch.full((p, c), 9.0, dtype=dtype, device="cuda")
    dy, dgates = ts.combine_bwd(dout.cuda(), y.cuda(), place.cuda(), gates.cuda(), err_flags=flags, into=mark.clone())
    ref = np.full((p, c), 9.0)
    ref[at[used].numpy()] = (f64(gates)[:, :, None] * f64(dout)[:, None])[used.numpy()]
    close(dy, ref, u * np.abs(ref) + E * np.abs(ref) + tiny, "dy")
    prod = np.where(used.numpy()[:, :, None], f64(dout)[:, None] * f64(y)[at.numpy()], 0.0)
    close(dgates, prod.sum(2), (c + 8) * E * np.abs(prod).sum(2) + 1e-37, "dgates")
    over = y.cuda()
    dy2, dgates2 = ts.combine_bwd(dout.cuda(), over, place.cuda(), gates.cuda(), into=over)  # over the grouped rows themselves
    named = at[used].cuda()
    assert torch.equal(dy2[named], dy[named]) and torch.equal(dgates, dgates2) and int(flags) == 0


def test_combine_places_out_of_range(ts):
    """Raised as a flag, counted as nothing."""
    y, d = torch.randn(10, 16, device="cuda"), torch.randn(3, 16, device="cuda")
    place = torch.tensor([[0, 10], [-2, 3], [2 ** 31 - 1, -1]], device="cuda", dtype=torch.int32)
    gates = torch.ones(3, 2, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ts.combine_fwd(y, place, gates, err_flags=flags)
    assert int(flags) == ts.TS_FLAG_RANGE
    assert torch.equal(out, torch.stack([y[0], y[3], torch.zeros(16, device="cuda")]))
    flags.zero_()
    dy, dg = ts.combine_bwd(d, y, place, gates, err_flags=flags, into=torch.zeros_like(y))
    assert int(flags) == ts.TS_FLAG_RANGE and torch.equal(dy[[0, 3]], d[:2])
    assert (dy[[1, 2, 4, 5, 6, 7, 8, 9]] == 0).all()
    assert (dg.reshape(-1)[[1, 2, 4, 5]] == 0).all()
    assert torch.equal(ts.combine_fwd(y, place, gates), out)  # without a flag word


def test_combine_past_32_bit_offsets(ts):
    """Grouped rows behind 2^31 elements."""
    c, p = 65536, 33000
    y = torch.empty(p, c, device="cuda", dtype=torch.float16)
    last = torch.randn(2, c, device="cuda").half()
    y[-2:] = last
    place = torch.tensor([[p - 1, p - 2]], device="cuda", dtype=torch.int32)
    gates = torch.tensor([[1.0, 0.0]], device="cuda")
    assert torch.equal(ts.combine_fwd(y, place, gates)[0], last[1])
    d = torch.randn(1, c, device="cuda").half()
    dy, _ = ts.combine_bwd(d, y, place, gates, into=y)
    assert torch.equal(dy[-1], d[0]) and (dy[-2] == 0).all()


def test_refusals(ts):
    z = torch.randn(20, 8, device="cuda")
    r = ts.route_fwd(z, 2)
    dg = torch.randn(20, 2, device="cuda")
    for f in (lambda: ts.route_fwd(z, 0), lambda: ts.route_fwd(z, 9), lambda: ts.route_fwd(z.t(), 2), lambda: ts.route_fwd(z.long(), 2),
              lambda: ts.route_fwd(z.cpu(), 2), lambda: ts.route_bwd(dg[:-1], z, r), lambda: ts.route_bwd(dg.half(), z, r),
              lambda: ts.route_fwd(torch.randn(4, 513, device="cuda"), 2), lambda: ts.route_fwd(torch.randn(4, 100, device="cuda"), 17)):
        with pytest.raises(ts.TsError):
            f()
    y = torch.randn(40, 16, device="cuda")
    for f in (lambda: ts.combine_fwd(y, r.place.long(), r.gates), lambda: ts.combine_fwd(y, r.place, r.gates[:-1]),
              lambda: ts.combine_fwd(y.t(), r.place, r.gates), lambda: ts.combine_fwd(y, r.place.view(-1), None),
              lambda: ts.combine_bwd(y, y, r.place, r.gates), lambda: ts.combine_bwd(y[:20].half(), y, r.place, r.gates),
              lambda: ts.combine_bwd(y[:20], y, r.place, r.gates, into=y[:20])):
        with pytest.raises(ts.TsError):
            f()
