"""Host-side checks of the entry points of rotation, routing, grouped products and the combining
sum (no GPU needed): size queries, and bad arguments refused before anything is launched."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "convolution_voxelised_point_amd", "libts.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libts.so not built")

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first, or has nothing to do
BIG = 1 << 60


@pytest.fixture(scope="module")
def ts():
    from convolution_voxelised_point_amd import ts as mod
    return mod


def rope(ts, **changes):
    fields = dict(dtype=ts.TS_F16, d=32, ndim=3, pairs=(6, 6, 4), interleaved=0, eps=1e-6, n=100, coords=0x1000, freqs=0x1000)
    fields.update(changes)
    fields["pairs"] = (ctypes.c_int32 * 3)(*fields["pairs"])
    return ts.TsRope(**fields)


def heads(ts, **changes):
    fields = dict(heads=4, x_stride=256, y_stride=128, dy_stride=128, dx_stride=256, x=0x1000, w=0x1000, y=0x1000, dy=0x1000, dx=0x1000,
                  dw=0x1000)
    fields.update(changes)
    return ts.TsRopeHeads(**fields)


def rope_calls(ts, r, q, k):
    a, b, c = (None if s is None else ctypes.byref(s) for s in (r, q, k))
    return ts._lib_rope_fwd(a, b, c, None), ts._lib_rope_bwd(a, b, c, FAKE, BIG, None)


BAD_ROPE = [
    (dict(dtype=3), "INVALID_ARG"), (dict(d=0), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"), (dict(ndim=1), "INVALID_ARG"),
    (dict(ndim=4), "INVALID_ARG"), (dict(eps=-1e-6), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(pairs=(-1, 6, 4)), "INVALID_ARG"), (dict(pairs=(6, 6, 5)), "INVALID_ARG"),
    (dict(pairs=(2 ** 31 - 1, 2 ** 31 - 1, 2)), "INVALID_ARG"), (dict(coords=None), "INVALID_ARG"), (dict(freqs=None), "INVALID_ARG"),
    (dict(d=129, pairs=(8, 8, 8)), "UNSUPPORTED"), (dict(n=1 << 30), "UNSUPPORTED"),
]


@pytest.mark.parametrize("changes,want", BAD_ROPE, ids=[str(b[0]) for b in BAD_ROPE])
def test_rope_refuses(ts, changes, want):
    r = rope(ts, **changes)
    status = getattr(ts, "TS_ERR_" + want)
    assert rope_calls(ts, r, heads(ts), heads(ts)) == (status, status)
    if "n" not in changes:
        assert ts._lib_rope_workspace_bytes(ctypes.byref(r), 4, 4) == 0


def test_rope_heads(ts):
    bad, r = ts.TS_ERR_INVALID_ARG, rope(ts)
    assert rope_calls(ts, None, heads(ts), None) == (bad, bad)
    for side in (0, 1):
        pair = lambda h: (h, heads(ts)) if side == 0 else (heads(ts), h)  # noqa: E731
        for change in (dict(heads=-1), dict(x=None), dict(x_stride=127)):
            assert rope_calls(ts, r, *pair(heads(ts, **change))) == (bad, bad), change
        for change in (dict(y=None), dict(y_stride=127)):
            assert rope_calls(ts, r, *pair(heads(ts, **change)))[0] == bad, change
        for change in (dict(dy=None), dict(dx=None), dict(dw=None), dict(dy_stride=127), dict(dx_stride=127)):
            assert rope_calls(ts, r, *pair(heads(ts, **change)))[1] == bad, change
        assert rope_calls(ts, r, *pair(heads(ts, heads=65536, x_stride=1 << 22, y_stride=1 << 22, dy_stride=1 << 22, dx_stride=1 << 22))) == \
            (ts.TS_ERR_UNSUPPORTED,) * 2
    need = ts._lib_rope_workspace_bytes(ctypes.byref(r), 4, 2)
    assert need >= 2 * 32 * 4 and need % 4 == 0
    q = ctypes.byref(heads(ts))
    for ws, n in ((None, BIG), (FAKE, ts._lib_rope_workspace_bytes(ctypes.byref(r), 4, 0) - 1)):
        assert ts._lib_rope_bwd(ctypes.byref(r), q, None, ws, n, None) == bad
    # nothing to do
    assert ts._lib_rope_workspace_bytes(ctypes.byref(rope(ts, n=0)), 4, 4) == 0
    assert rope_calls(ts, r, None, None) == (0, 0)
    assert rope_calls(ts, r, heads(ts, heads=0, x=None, y=None), None) == (0, 0)
    # the largest sizes answer without overflow
    assert 0 < ts._lib_rope_workspace_bytes(ctypes.byref(rope(ts, n=(1 << 31) - 1, d=128, pairs=(20, 20, 20))), 65535, 65535) < 1 << 24


@pytest.mark.parametrize("n", [1, 1 << 20, (1 << 21) - 1, 1 << 21, 1 << 40, (1 << 63) - 1])
def test_rope_workspace_of_any_length(ts, n):
    """Two sides' shares of dw from at most 1024 blocks, of 2048 channels or more."""
    for h, d in ((1, 1), (4, 32), (65535, 128)):
        blocks = min(-(-n * h * d // 2048), 1024)
        pairs = (0, 0, 0) if d == 1 else (6, 6, 4)
        assert ts._lib_rope_workspace_bytes(ctypes.byref(rope(ts, n=n, d=d, pairs=pairs)), h, 0) == 2 * blocks * d * 4


def test_route_refuses(ts):
    bad, no = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    out = [FAKE] * 5
    for n, e, dt, top, want in ((-1, 8, 1, 2, bad), (8, 0, 1, 1, bad), (8, 8, 3, 2, bad), (8, 8, 1, 0, bad), (8, 8, 1, 9, bad),
                                (8, 513, 1, 2, no), (8, 64, 1, 17, no), (1 << 30, 8, 1, 2, no)):
        assert ts._lib_route_fwd(FAKE, n, e, dt, top, 0, *out, FAKE, BIG, None) == want
        assert ts._lib_route_bwd(FAKE, FAKE, FAKE, FAKE, n, e, dt, top, 1, FAKE, None) == want
        if dt != 3:
            assert ts._lib_route_workspace_bytes(n, e, top) == 0
    for i in range(6):                                     # logits, experts, gates, starts, rows, place
        args = [FAKE] * 6
        args[i] = None
        assert ts._lib_route_fwd(args[0], 8, 8, 1, 2, 0, *args[1:], FAKE, BIG, None) == bad, i
    for i in range(5):                                     # dgates, logits, experts, gates, dlogits
        args = [FAKE] * 5
        args[i] = None
        assert ts._lib_route_bwd(*args[:4], 8, 8, 1, 2, 1, args[4], None) == bad, i
    assert ts._lib_route_workspace_bytes(8, 8, 2) == 0     # one block does it
    need = ts._lib_route_workspace_bytes(300000, 64, 2)
    assert 65 * 4 < need <= 1 << 21
    for ws, n in ((None, need), (FAKE, need - 1)):
        assert ts._lib_route_fwd(FAKE, 300000, 64, 1, 2, 0, *out, ws, n, None) == bad
    assert ts._lib_route_bwd(None, None, None, None, 0, 8, 1, 2, 1, None, None) == 0
    for n, e in (((1 << 31) - 1, 512), ((1 << 31) - 1, 1), (2 ** 20, 512)):
        assert 0 < ts._lib_route_workspace_bytes(n, e, 1) < 1 << 22


def test_combine_refuses(ts):
    bad = ts.TS_ERR_INVALID_ARG

    def fwd(y=FAKE, p=20, place=FAKE, gates=FAKE, n=10, top=2, c=8, dt=1, out=FAKE):
        return ts._lib_combine_fwd(y, p, place, gates, n, top, c, dt, out, None, None)

    def bwd(dout=FAKE, y=FAKE, p=20, place=FAKE, gates=FAKE, n=10, top=2, c=8, dt=1, dy=FAKE, dgates=FAKE):
        return ts._lib_combine_bwd(dout, y, p, place, gates, n, top, c, dt, dy, dgates, None, None)
    for change in (dict(p=-1), dict(p=1 << 31), dict(n=-1), dict(n=1 << 31), dict(top=0), dict(c=0), dict(c=65537), dict(dt=3), dict(y=None),
                   dict(place=None)):
        assert fwd(**change) == bad and bwd(**change) == bad, change
    assert fwd(out=None) == bad
    for name in ("dout", "gates", "dy", "dgates"):
        assert bwd(**{name: None}) == bad, name
    assert fwd(n=0, y=None, place=None, out=None) == 0 and bwd(n=0, y=None, place=None, dout=None) == 0


def groups(ts, **changes):
    fields = dict(n_groups=4, n_rows=100, starts=0x1000, rows=0x1000, n_src=50)
    fields.update(changes)
    return ts.TsGroups(**fields)


def group_calls(ts, g, cin=32, cout=64, dt=1, x=FAKE, w=FAKE, y=FAKE, dy=FAKE, ws=FAKE, n=BIG):
    r = None if g is None else ctypes.byref(g)
    return (ts._lib_group_fwd(r, x, cin, w, cout, dt, 0, y, None, None, None), ts._lib_group_bwd_dgrad(r, dy, cout, w, cin, dt, None, y, None, None),
            ts._lib_group_bwd_wgrad(r, x, cin, dy, cout, dt, y, ws, n, None, None))


BAD_GROUPS = [
    (dict(n_groups=0), {}, "INVALID_ARG"), (dict(n_rows=-1), {}, "INVALID_ARG"), (dict(n_rows=1 << 31), {}, "INVALID_ARG"),
    (dict(starts=None), {}, "INVALID_ARG"), (dict(n_src=-1), {}, "INVALID_ARG"), (dict(n_src=1 << 31), {}, "INVALID_ARG"),
    ({}, dict(cin=0), "INVALID_ARG"), ({}, dict(cout=0), "INVALID_ARG"), ({}, dict(cin=65537), "INVALID_ARG"), ({}, dict(cout=65537), "INVALID_ARG"),
    ({}, dict(dt=5), "INVALID_ARG"), ({}, dict(dt=0), "UNSUPPORTED"), (dict(n_groups=4097), {}, "UNSUPPORTED"),
]


@pytest.mark.parametrize("changes,call,want", BAD_GROUPS, ids=[f"{a}{b}" for a, b, _ in BAD_GROUPS])
def test_groups_refuse(ts, changes, call, want):
    status = getattr(ts, "TS_ERR_" + want)
    assert group_calls(ts, groups(ts, **changes), **call) == (status,) * 3


def test_groups_of_too_many_tiles(ts):
    assert group_calls(ts, groups(ts, n_rows=(1 << 31) - 1), cin=65536, cout=65536, n=0) == (ts.TS_ERR_UNSUPPORTED,) * 3
    assert group_calls(ts, groups(ts, n_groups=4096, n_rows=1 << 20), cin=65536, cout=65536, n=0) == (ts.TS_ERR_UNSUPPORTED,) * 3


def test_group_pointers_and_workspace(ts):
    bad, g = ts.TS_ERR_INVALID_ARG, groups(ts)
    assert group_calls(ts, None) == (bad,) * 3
    assert group_calls(ts, g, w=None)[:2] == (bad, bad)
    assert group_calls(ts, g, y=None) == (bad,) * 3
    assert group_calls(ts, g, dy=None)[1:] == (bad, bad)
    f, _, d = group_calls(ts, g, x=None)
    assert (f, d) == (bad, bad)
    ref = ctypes.byref(g)
    assert ts._lib_group_fwd(ref, FAKE, 32, FAKE, 64, 1, 0, FAKE, FAKE, None, None) == bad  # h without glu
    need = ts._lib_group_wgrad_workspace_bytes(ref, 32, 64)
    assert need >= 4 * 32 * 64 * 4
    for ws, n in ((None, need), (FAKE, need - 1)):
        assert group_calls(ts, g, ws=ws, n=n)[2] == bad
    assert ts._lib_group_wgrad_workspace_bytes(None, 32, 64) == 0
    assert ts._lib_group_wgrad_workspace_bytes(ctypes.byref(groups(ts, n_groups=0)), 32, 64) == 0
    # a run never has fewer than 256 rows, nor are there more than one partial sum a run and group
    for rows, e, cin, cout in ((1, 1, 1, 1), (10 ** 6, 8, 128, 128), (10 ** 6, 8, 1024, 4096), (2 ** 31 - 1, 3, 64, 64), (5000, 4096, 256, 256), ((1 << 31) - 1, 4, 65536, 65536)):
        size = ts._lib_group_wgrad_workspace_bytes(ctypes.byref(groups(ts, n_rows=rows, n_groups=e)), cin, cout)
        assert e * cin * cout * 4 <= size <= (rows // 256 + e) * cin * cout * 4
    # nothing to do
    none = groups(ts, n_rows=0)
    assert group_calls(ts, none, x=None, dy=None)[:2] == (0, 0)


def test_binding_refuses_host_tensors(ts):
    """The binding's own checks come before the library is called."""
    import torch
    x, w, p = torch.zeros(4, 8).half(), torch.zeros(2, 8, 8).half(), torch.zeros(4, 2, dtype=torch.int32)
    starts = torch.zeros(3, dtype=torch.int64)
    for f in (lambda: ts.group_fwd(x, w, ts.Groups(starts)), lambda: ts.group_dgrad(x, w, ts.Groups(starts)),
              lambda: ts.group_wgrad(x, x, ts.Groups(starts)), lambda: ts.group_glu_fwd(x, w, ts.Groups(starts)),
              lambda: ts.route_fwd(x, 2), lambda: ts.combine_fwd(x, p), lambda: ts.rope_fwd(x.view(4, 1, 8), None, None, None, (0, 0))):
        with pytest.raises(ts.TsError):
            f()
