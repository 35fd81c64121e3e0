"""Products grouped by expert after bad starts and row numbers: results, kept halves and the workspace lie in
larger buffers, and what is around them stays as it was."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

MARGIN = 1 << 14  # elements on either side: more than a tile's rows of these widths


class Band:
    """A dense tensor of `shape` in the middle of a buffer whose other elements are marked."""

    def __init__(self, shape, dtype, mark):
        self.n, self.mark = 1, mark
        for s in shape:
            self.n *= s
        self.all = torch.full((self.n + 2 * MARGIN,), mark, dtype=dtype, device="cuda")
        self.t = self.all[MARGIN:MARGIN + self.n].view(shape)

    def stays(self):
        return bool((self.all[:MARGIN] == self.mark).all()) and bool((self.all[MARGIN + self.n:] == self.mark).all())


def bad_starts(e, n):
    """Starts of e groups of n rows that decrease, leave the range, overlap, or are any numbers at all."""
    g = torch.Generator().manual_seed(e + n)
    for cut in ([0, n, 0], [0, n * 4 // 5, n // 3], [-5, n // 6, n // 3], [0, n // 6, 10 ** 12], [n, 0, n], [-2 ** 62, 2 ** 62, -1], [3, n, n // 2]):
        yield cut + [n] * (e - 2)
    yield [0, n] * ((e + 1) // 2) + [n] * ((e + 1) % 2)  # the whole of them, over and over
    for _ in range(3):
        yield torch.randint(-n // 4, n + n // 4, (e + 1,), generator=g).tolist()


CASES = [  # rows, groups, cin, cout: few rows an expert, tiles of 128, 192 and 256 rows, rows that are no whole 16 bytes, more than 64 groups
    (60, 3, 64, 64), (90, 3, 77, 133), (3000, 3, 64, 128), (3000, 3, 77, 133), (2100, 3, 264, 520), (45600, 72, 256, 264),
    (700, 70, 72, 40), (63000, 3, 256, 256), (9000, 66, 31, 65),
]


@pytest.mark.parametrize("gather", [False, True], ids=["", "rows"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_nothing_around_the_results_changes(ts, case, gather):
    n, e, cin, cout = case
    g = torch.Generator("cuda").manual_seed(n)
    dt, n_src = torch.bfloat16, n // 2
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, w, wg, dy, h = normal(n_src if gather else n, cin), normal(e, cin, cout), normal(e, cin, 2 * cout), normal(n, cout), normal(n, 2 * cin)
    rows = torch.randint(-3, n_src + 3, (n,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    y, glu, kept = (Band((n, c), dt, -77.0) for c in (cout, cout, 2 * cout))
    dx, dh, dw = Band((n, cin), dt, -77.0), Band((n, 2 * cin), dt, -77.0), Band((e, cin, cout), torch.float32, -77.0)
    for starts in bad_starts(e, n):
        at = torch.tensor(starts, device="cuda")
        assert at.numel() == e + 1
        groups = ts.TsGroups(e, n, at.data_ptr(), rows.data_ptr() if gather else None, n_src if gather else 0)
        ref = ctypes.byref(groups)
        size = ts._lib_group_wgrad_workspace_bytes(ref, cin, cout)
        ws = Band((size // 4,), torch.float32, -77.0)
        dh.t.copy_(h)
        p = [t.data_ptr() for t in (x, w, wg, dy, h, flags)]
        for call in (
                lambda: ts._lib_group_fwd(ref, p[0], cin, p[1], cout, ts.TS_BF16, 0, y.t.data_ptr(), None, p[5], stream),
                lambda: ts._lib_group_fwd(ref, p[0], cin, p[2], cout, ts.TS_BF16, 1, glu.t.data_ptr(), kept.t.data_ptr(), p[5], stream),
                lambda: ts._lib_group_bwd_dgrad(ref, p[3], cout, p[1], cin, ts.TS_BF16, None, dx.t.data_ptr(), p[5], stream),
                lambda: ts._lib_group_bwd_dgrad(ref, p[3], cout, p[1], cin, ts.TS_BF16, dh.t.data_ptr(), dh.t.data_ptr(), p[5], stream),
                lambda: ts._lib_group_bwd_wgrad(ref, p[0], cin, p[3], cout, ts.TS_BF16, dw.t.data_ptr(), ws.t.data_ptr(), size, p[5], stream)):
            flags.zero_()
            assert call() == 0
            assert int(flags) == ts.TS_FLAG_RANGE, starts
        for band, what in ((y, "y"), (glu, "silu(a) b"), (kept, "h"), (dx, "dx"), (dh, "dh"), (dw, "dw"), (ws, "workspace")):
            assert band.stays(), (what, starts)
