"""GPU parity of the products grouped by expert, forward, backward and with silu(a) b, against
plain fp64 implementations.

Tolerances, E = 2^-24, u the result's type (2^-11, 2^-8): products of 16-bit values are exact
in fp32, a sum of K of them is off by at most (K + 8) E of the sum of their magnitudes, and the
result by u of itself.  silu has a slope of at most 1.1 and is formed with an error of 8 E of itself."""
import numpy as np
import pytest
import torch

import bench
from helpers import U_OUT

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -24


def close(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} over tolerance, worst {float((err / tol).nan_to_num(1e9).max()):.3g} "
                                 f"times it, first at {torch.nonzero(bad)[0].tolist()}")


def silu(a):
    return a * torch.sigmoid(a)


class Case:
    def __init__(self, ts, dt, lens, cin, cout, gather=True, before=0, behind=0, seed=0):
        self.ts, self.dt, self.u, self.tiny = ts, DT[dt], U_OUT[DT[dt]], 2.0 ** -25 if dt == "f16" else 1e-37
        g = torch.Generator("cuda").manual_seed(seed + cin * 7 + cout)
        self.e, self.cin, self.cout = len(lens), cin, cout
        self.host = np.cumsum([before] + list(lens)).tolist()
        self.p = self.host[-1] + behind
        n = max(self.p // 2, 1) if gather else self.p
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(self.dt)
        self.x, self.w, self.wg = normal(n, cin), normal(self.e, cin, cout), normal(self.e, cin, 2 * cout)
        self.dy, self.h = normal(self.p, cout), normal(self.p, 2 * cin)
        rows = torch.randint(0, n, (self.p,), generator=g, device="cuda", dtype=torch.int32) if gather else None
        self.groups = ts.Groups(torch.tensor(self.host, device="cuda"), rows)
        self.xg = self.x if rows is None else self.x[rows.long()]
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def product(self, x, w):
        """Grouped x W and the sums of magnitudes, zeros where no group owns."""
        y = torch.zeros(self.p, w.shape[2], dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(y)
        for e in range(self.e):
            a, b = self.host[e], self.host[e + 1]
            y[a:b] = x[a:b].double() @ w[e].double()
            mag[a:b] = x[a:b].double().abs() @ w[e].double().abs()
        return y, mag

    def check(self, what=("fwd", "glu", "dgrad", "glu_dgrad", "wgrad")):
        ts, u, tiny, f = self.ts, self.u, self.tiny, dict(err_flags=self.flags)
        wt = self.w.transpose(1, 2).contiguous()
        if "fwd" in what:
            y, mag = self.product(self.xg, self.w)
            close(ts.group_fwd(self.x, self.w, self.groups, **f), y, u * y.abs() + (self.cin + 8) * E * mag + tiny, "y")
        if "glu" in what:
            h, mag = self.product(self.xg, self.wg)
            err = (self.cin + 8) * E * mag
            (a, b), (ea, eb) = h.chunk(2, 1), err.chunk(2, 1)
            y = silu(a) * b
            tol = 1.1 * ea * (b.abs() + eb) + silu(a).abs() * eb + 8 * E * y.abs()
            got, kept = ts.group_glu_fwd(self.x, self.wg, self.groups, want_h=True, **f)
            close(got, y, u * y.abs() + tol + tiny, "silu(a) b")
            close(kept, h, u * h.abs() + err + tiny, "h")
            alone, none = ts.group_glu_fwd(self.x, self.wg, self.groups, **f)
            assert none is None and torch.equal(alone, got)
        if "dgrad" in what or "glu_dgrad" in what:
            d, mag = self.product(self.dy, wt)
            ed = (self.cout + 8) * E * mag
            if "dgrad" in what:
                close(ts.group_dgrad(self.dy, self.w, self.groups, **f), d, u * d.abs() + ed + tiny, "dx")
            if "glu_dgrad" in what:
                a, b = self.h.double().chunk(2, 1)
                s = torch.sigmoid(a)
                ref = torch.cat([d * b * s * (1 + a * (1 - s)), d * a * s], 1)
                tol = torch.cat([1.1 * ed * b.abs() + 16 * E * (d * b).abs() * (1 + a.abs()), ed * a.abs() + 16 * E * (d * a).abs()], 1)
                got = ts.group_glu_dgrad(self.dy, self.w, self.h, self.groups, **f)
                close(got, ref, u * ref.abs() + tol + tiny, "dh")
                over = self.h.clone()
                assert torch.equal(ts.group_glu_dgrad(self.dy, self.w, over, self.groups, into=over), got)
        if "wgrad" in what:
            dw = ts.group_wgrad(self.x, self.dy, self.groups, **f)
            for e in range(self.e):
                a, b = self.host[e], self.host[e + 1]
                x, dy = self.xg[a:b].double().t().contiguous(), self.dy[a:b].double()
                close(dw[e], x @ dy, (b - a + 8) * E * (x.abs() @ dy.abs()) + 1e-37, f"dw[{e}]")
            assert torch.equal(ts.group_wgrad(self.x, self.dy, self.groups), dw)
        assert int(self.flags) == 0
        return self


CASES = [  # rows of each group, cin, cout
    ([1], 1, 1), ([2], 8, 8), ([1, 0, 1], 32, 64), ([0, 0], 64, 64), ([3, 5, 0, 7], 40, 24), ([17, 15, 16], 77, 133),
    ([1] * 70, 64, 128), ([0] * 129 + [2], 33, 65), ([48, 60, 33], 256, 192), ([30, 18, 24], 128, 512),
    ([128, 127, 129, 0, 1, 300], 64, 128), ([100, 200], 72, 136), ([90, 110], 31, 129), ([513, 600], 256, 256),
    ([600, 0, 1500], 264, 520), ([1025], 512, 256), ([777, 999], 100, 300), ([5000, 3], 128, 16), ([9001], 96, 40),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}_{c[1]}_{c[2]}")
def test_group(ts, case, dt):
    lens, cin, cout = case
    Case(ts, dt, lens, cin, cout).check()
    Case(ts, dt, lens, cin, cout, gather=False, before=3, behind=150).check()


LONG = [  # long runs of the weight gradient, and many of them; many groups of many rows
    ([9000, 0, 4100, 300], 264, 520, ("wgrad",)), ([40000, 7, 23000], 256, 256, ("wgrad",)),
    ([5, 0, 900] * 90, 512, 512, ("wgrad",)), ([700, 0, 1200] * 24, 64, 256, ("fwd", "glu", "wgrad")),
    ([700, 0, 1200] * 24, 256, 64, ("dgrad", "glu_dgrad")),
    # many groups of few rows and many columns
    ([1, 0, 3, 9] * 16, 128, 1024, ("fwd", "glu")), ([20, 0, 3, 9] * 16, 77, 1029, ("fwd", "glu")),
    ([1, 0, 3, 9] * 16, 1024, 128, ("dgrad", "glu_dgrad")), ([1, 0, 3, 9] * 16, 1029, 77, ("dgrad", "glu_dgrad")),
    ([50000, 0, 30000], 515, 517, ("wgrad",)), ([50000, 30000], 1024, 1024, ("wgrad",)), ([70000, 30000], 128, 1024, ("wgrad",)),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("case", LONG, ids=lambda c: f"{len(c[0])}x{max(c[0])}_{c[1]}_{c[2]}")
def test_long_groups(ts, case, dt):
    lens, cin, cout, what = case
    Case(ts, dt, lens, cin, cout).check(what)
    Case(ts, dt, lens, cin, cout, gather=False, before=70, behind=300).check(what)


def test_long_groups_with_bad_rows_and_starts(ts):
    c = Case(ts, "bf16", [40000, 0, 23000], 256, 256)
    c.groups.rows[::1000], c.groups.rows[c.p - 1] = -1, c.x.shape[0]
    c.xg = c.xg.clone()
    c.xg[::1000], c.xg[c.p - 1] = 0, 0
    dw = ts.group_wgrad(c.x, c.dy, c.groups, err_flags=c.flags)
    assert int(c.flags) == ts.TS_FLAG_RANGE
    for e in range(c.e):
        a, b = c.host[e], c.host[e + 1]
        x, dy = c.xg[a:b].double().t().contiguous(), c.dy[a:b].double()
        close(dw[e], x @ dy, (b - a + 8) * E * (x.abs() @ dy.abs()) + 1e-37, f"dw[{e}]")
    for starts in ([0, 50000, 20, 63000], [0, 63000, 0, 63000], [-5, 10 ** 12, 3, 63000]):
        c.flags.zero_()
        ts.group_wgrad(c.x, c.dy, ts.Groups(torch.tensor(starts, device="cuda"), c.groups.rows.clamp(0, 10)), err_flags=c.flags)
        assert int(c.flags) == ts.TS_FLAG_RANGE


@pytest.mark.parametrize("n", [0, 5, 70, 1200])
def test_rows_without_a_group(ts, n):
    """All rows before or behind the groups: zeros, and no gradient."""
    for before, behind in ((n, 0), (0, n)):
        c = Case(ts, "bf16", [0, 0, 0], 64, 96, gather=False, before=before, behind=behind).check()
        assert (ts.group_wgrad(c.x, c.dy, c.groups) == 0).all()
        if n:
            assert (ts.group_fwd(c.x, c.w, c.groups) == 0).all()


@pytest.mark.parametrize("d", [0, 4])
def test_matrices_that_are_not_16_byte_aligned(ts, d):
    """Columns that are multiples of 8, but bases that are not."""
    c = Case(ts, "f16", [70, 300], 64, 64)

    def moved(t):
        m = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        v = m[1 + d:1 + d + t.numel()].view(t.shape)
        v.copy_(t)
        return v
    c.x, c.w, c.wg, c.dy, c.h = (moved(t) for t in (c.x, c.w, c.wg, c.dy, c.h))
    c.check()


@pytest.mark.parametrize("lens,cin,cout", [([2, 3], 64, 64), ([600, 700], 256, 256), ([200, 90], 64, 64), ([200, 90], 63, 61)])
def test_rows_out_of_range(ts, lens, cin, cout):
    """Read as zeros, with the flag; the others as ever."""
    c = Case(ts, "bf16", lens, cin, cout)
    want = ts.group_fwd(c.x, c.w, c.groups)
    c.groups.rows[1], c.groups.rows[c.p - 1] = -1, c.x.shape[0]
    got = ts.group_fwd(c.x, c.w, c.groups, err_flags=c.flags)
    assert int(c.flags) == ts.TS_FLAG_RANGE
    assert (got[[1, c.p - 1]] == 0).all()
    got[[1, c.p - 1]] = want[[1, c.p - 1]]
    assert torch.equal(got, want)
    c.flags.zero_()
    c.xg = c.xg.clone()
    c.xg[[1, c.p - 1]] = 0
    dw = ts.group_wgrad(c.x, c.dy, c.groups, err_flags=c.flags)
    assert int(c.flags) == ts.TS_FLAG_RANGE
    for e in range(c.e):
        a, b = c.host[e], c.host[e + 1]
        x, dy = c.xg[a:b].double().t().contiguous(), c.dy[a:b].double()
        close(dw[e], x @ dy, (b - a + 8) * E * (x.abs() @ dy.abs()) + 1e-37, f"dw[{e}]")


@pytest.mark.parametrize("starts", [[0, 50, 40, 60], [-5, 10, 20, 60], [0, 10, 20, 10 ** 12], [60, 0, 60, 0], [-2 ** 62, 2 ** 62, -1, 2 ** 62]])
@pytest.mark.parametrize("rows", [60, 3000])
def test_bad_starts(ts, starts, rows):
    """Raise the flag, and nothing outside the buffers is touched (a band around the results stays)."""
    c = Case(ts, "f16", [rows, 0, 0], 64, 64, gather=False)
    bad = ts.Groups(torch.tensor(starts, device="cuda"))
    for f in (lambda: ts.group_fwd(c.x, c.w, bad, err_flags=c.flags), lambda: ts.group_dgrad(c.dy, c.w, bad, err_flags=c.flags),
              lambda: ts.group_wgrad(c.x, c.dy, bad, err_flags=c.flags)):
        c.flags.zero_()
        f()
        assert int(c.flags) == ts.TS_FLAG_RANGE


def test_infinities_stay_in_their_rows(ts):
    for lens in ([3, 4], [300, 200]):
        c = Case(ts, "bf16", lens, 64, 128, gather=False)
        want = ts.group_fwd(c.x, c.w, c.groups)
        c.x[2, 5] = float("nan")
        got = ts.group_fwd(c.x, c.w, c.groups)
        assert got[2].isnan().all()
        got[2] = want[2]
        assert torch.equal(got, want)


def test_past_32_bit_offsets(ts):
    """Grouped rows and weights behind 2^31 elements; x as large as that."""
    cin, cout, p = 64, 32768, 70000
    w = torch.zeros(2, cin, cout, device="cuda", dtype=torch.bfloat16)
    w[:, :, -64:] = torch.randn(2, cin, 64, device="cuda").bfloat16()
    x = torch.randn(p, cin, device="cuda").bfloat16()
    y = ts.group_fwd(x, w, ts.Groups(torch.tensor([0, 10, p], device="cuda")))
    ref = x[-300:].double() @ w[1, :, -64:].double()
    close(y[-300:, -64:], ref, 2.0 ** -8 * ref.abs() + 72 * E * (x[-300:].double().abs() @ w[1, :, -64:].double().abs()), "y")
    assert (y[-300:, :-64] == 0).all()
    rows = torch.tensor([p - 1, p - 2, 5], device="cuda", dtype=torch.int32)  # y itself read by rows
    w2 = torch.zeros(1, cout, 8, device="cuda", dtype=torch.bfloat16)
    w2[0, -8:] = torch.eye(8, device="cuda")
    z = ts.group_fwd(y, w2, ts.Groups(torch.tensor([0, 3], device="cuda"), rows))
    assert torch.equal(z, y[rows.long(), -8:])
    many = torch.zeros(130, 4096, 4096, device="cuda", dtype=torch.float16)
    many[-1] = torch.eye(4096, device="cuda")
    starts = torch.zeros(131, dtype=torch.int64, device="cuda")
    starts[-1] = 5
    x = torch.randn(5, 4096, device="cuda").half()
    assert torch.equal(ts.group_fwd(x, many, ts.Groups(starts)), x) and torch.equal(ts.group_dgrad(x, many, ts.Groups(starts)), x)


def test_stream_and_graph(ts):
    cases = [Case(ts, "bf16", lens, cin, cout) for lens, cin, cout in (([2, 1, 3], 128, 256), ([700, 900], 256, 256), ([150, 90], 77, 40))]

    def every(stream=None):
        out = []
        for c in cases:
            out += [ts.group_fwd(c.x, c.w, c.groups, stream=stream), *ts.group_glu_fwd(c.x, c.wg, c.groups, True, stream=stream),
                    ts.group_dgrad(c.dy, c.w, c.groups, stream=stream), ts.group_glu_dgrad(c.dy, c.w, c.h, c.groups, stream=stream),
                    ts.group_wgrad(c.x, c.dy, c.groups, stream=stream)]
        return out
    want, held = every(), []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = every(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    def step():
        held[:] = every()
    graph = bench.capture([step])
    for _ in range(3):
        for t in held:
            t.fill_(-7)
        torch.randn(512, 512, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_refusals(ts):
    c = Case(ts, "f16", [30, 40], 32, 48)
    g, bad = c.groups, [
        lambda g: ts.group_fwd(c.x, c.w.float(), g), lambda g: ts.group_fwd(c.x, c.w[:1], g), lambda g: ts.group_fwd(c.x[:, :24].contiguous(), c.w, g),
        lambda g: ts.group_fwd(c.x.t(), c.w, g), lambda g: ts.group_fwd(c.x, c.w.transpose(1, 2), g), lambda g: ts.group_fwd(c.x.cpu(), c.w, g),
        lambda g: ts.group_fwd(c.x.float(), c.w.float(), g), lambda g: ts.group_fwd(c.x, c.w, ts.Groups(g.starts.int(), g.rows)),
        lambda g: ts.group_fwd(c.x, c.w, ts.Groups(g.starts, g.rows.long())), lambda g: ts.group_fwd(c.x, c.w, ts.Groups(g.starts[:1], g.rows)),
        lambda g: ts.group_glu_fwd(c.x, torch.cat([c.w, c.w[:, :, :1]], 2), g), lambda g: ts.group_dgrad(c.dy[:, :40].contiguous(), c.w, g),
        lambda g: ts.group_glu_dgrad(c.dy, c.w, c.h[:-1], g), lambda g: ts.group_glu_dgrad(c.dy, c.w, c.h, g, into=c.dy),
        lambda g: ts.group_wgrad(c.x, c.dy[:-1], g), lambda g: ts.group_wgrad(c.x, c.dy.bfloat16(), g),
        lambda g: ts.group_wgrad(c.x, c.dy, ts.Groups(g.starts)),
    ]
    for f in bad:
        with pytest.raises(ts.TsError):
            f(g)
