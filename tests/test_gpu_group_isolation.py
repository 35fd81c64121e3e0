"""Products grouped by expert: a value that is no number reaches the results it enters and no others, whatever lies
beside it in memory; and rows of x behind 2^31 elements, read by number."""
import pytest
import torch

from test_gpu_group import E, Case, close

pytestmark = pytest.mark.gpu

NAN = float("nan")
CASES = [  # few rows and many, whole accesses and rows that are none, a last step that is not full, runs of the weight gradient
    ([5, 9, 1], 77, 133), ([30, 44, 20], 77, 133), ([40, 80, 35], 5, 3), ([3, 2, 7], 40, 24), ([300, 200, 90], 77, 133), ([300, 77, 200], 3, 6),
    ([300, 200, 90], 64, 128), ([300, 201, 90], 72, 136), ([600, 777, 1500], 264, 520), ([3000, 20001, 100], 256, 256), ([3000, 20001, 100], 261, 259),
]


def same_but(got, want, where, what):
    """Not a number at the True places of `where`, the same bits at the others."""
    assert bool(got[where].isnan().all()), what
    assert torch.equal(torch.where(where, 0.0, got), torch.where(where, 0.0, want)), what


@pytest.mark.parametrize("gather", [False, True], ids=["", "rows"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_values_stay_in_their_rows_and_columns(ts, case, gather):
    lens, cin, cout = case
    c = Case(ts, "bf16", lens, cin, cout, gather=False)
    a, b, p = c.host[1], c.host[2], c.p
    rows = torch.arange(p - 1, -1, -1, device="cuda", dtype=torch.int32) if gather else None
    c.groups = ts.Groups(c.groups.starts, rows)
    src = rows.long() if gather else torch.arange(p, device="cuda")  # where grouped row p of x lies
    at = torch.tensor([a, b - 1], device="cuda")                     # the first and the last row of the middle expert
    mine = torch.zeros(p, 1, dtype=torch.bool, device="cuda")
    mine[at] = True
    middle = torch.zeros(p, 1, dtype=torch.bool, device="cuda")
    middle[a:b] = True

    def ends(width):
        m = torch.zeros(1, width, dtype=torch.bool, device="cuda")
        m[0, [0, -1]] = True
        return m
    x, dy, h = c.x.clone(), c.dy.clone(), c.h.clone()
    for col in (0, -1):
        x[src[at], col] = dy[at, col] = NAN
    # a row of x or dy: its row of the result
    y, (s, kept) = ts.group_fwd(c.x, c.w, c.groups), ts.group_glu_fwd(c.x, c.wg, c.groups, True)
    dx, dh = ts.group_dgrad(c.dy, c.w, c.groups), ts.group_glu_dgrad(c.dy, c.w, c.h, c.groups)
    every = lambda t: torch.ones(1, t.shape[1], dtype=torch.bool, device="cuda")  # noqa: E731
    same_but(ts.group_fwd(x, c.w, c.groups), y, mine & every(y), "y by x")
    s1, kept1 = ts.group_glu_fwd(x, c.wg, c.groups, True)
    same_but(s1, s, mine & every(s), "silu(a) b by x")
    same_but(kept1, kept, mine & every(kept), "h by x")
    same_but(ts.group_dgrad(dy, c.w, c.groups), dx, mine & every(dx), "dx by dy")
    same_but(ts.group_glu_dgrad(dy, c.w, c.h, c.groups), dh, mine & every(dh), "dh by dy")
    # an element of h: its own two gradients
    for col in (0, cin - 1, cin, 2 * cin - 1):
        h[at, col] = NAN
    both = torch.cat([ends(cin), ends(cin)], 1)
    same_but(ts.group_glu_dgrad(c.dy, c.w, h, c.groups), dh, mine & both, "dh by h")
    # a column of an expert's weights (a row, for the gradient): its column of that expert's rows
    w, wg = c.w.clone(), c.wg.clone()
    w[1, -1, [0, -1]] = NAN
    wg[1, -1, [0, cout - 1, cout, 2 * cout - 1]] = NAN
    same_but(ts.group_fwd(c.x, w, c.groups), y, middle & ends(cout), "y by w")
    s1, kept1 = ts.group_glu_fwd(c.x, wg, c.groups, True)
    same_but(s1, s, middle & ends(cout), "silu(a) b by w")
    same_but(kept1, kept, middle & torch.cat([ends(cout), ends(cout)], 1), "h by w")
    w = c.w.clone()
    w[1, [0, -1], -1] = NAN
    same_but(ts.group_dgrad(c.dy, w, c.groups), dx, middle & ends(cin), "dx by w")
    same_but(ts.group_glu_dgrad(c.dy, w, c.h, c.groups), dh, middle & both, "dh by w")
    # the weight gradient: rows and columns of that expert's, and nothing of its neighbours'
    dw = ts.group_wgrad(c.x, c.dy, c.groups)
    mine = torch.zeros_like(dw, dtype=torch.bool)
    mine[1] = ends(cin).t() | torch.zeros(1, cout, dtype=torch.bool, device="cuda")
    same_but(ts.group_wgrad(x, c.dy, c.groups), dw, mine, "dw by x")
    mine[1] = ends(cout) | torch.zeros(cin, 1, dtype=torch.bool, device="cuda")
    same_but(ts.group_wgrad(c.x, dy, c.groups), dw, mine, "dw by dy")


@pytest.mark.parametrize("n_src", [32767, 32769])
def test_rows_looked_up_behind_32_bit_offsets(ts, n_src):
    """The last rows of an x of just under 2^31 elements (byte offsets up to 2^32) and of one of more."""
    cin, cout, p = 65536, 8, 300
    g = torch.Generator("cuda").manual_seed(n_src)
    x = torch.zeros(n_src, cin, device="cuda", dtype=torch.bfloat16)
    x[-p:] = torch.randn(p, cin, generator=g, device="cuda").bfloat16()
    w, dy = torch.randn(2, cin, cout, generator=g, device="cuda").bfloat16(), torch.randn(p, cout, generator=g, device="cuda").bfloat16()
    rows = n_src - 1 - torch.randperm(p, generator=g, device="cuda").int()
    cut = 140
    groups = ts.Groups(torch.tensor([0, cut, p], device="cuda"), rows)
    y, dw = ts.group_fwd(x, w, groups), ts.group_wgrad(x, dy, groups)
    xg = x[rows.long()].double()
    for e, (a, b) in enumerate(((0, cut), (cut, p))):
        ref = xg[a:b] @ w[e].double()
        close(y[a:b], ref, 2.0 ** -8 * ref.abs() + (cin + 8) * E * (xg[a:b].abs() @ w[e].double().abs()), f"y[{e}]")
        xt = xg[a:b].t().contiguous()
        close(dw[e], xt @ dy[a:b].double(), (b - a + 8) * E * (xt.abs() @ dy[a:b].double().abs()) + 1e-37, f"dw[{e}]")
