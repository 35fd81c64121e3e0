"""Host-side checks of the voxel-transformer entry points (no GPU needed):
size queries, and bad arguments refused before anything is launched."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "convolution_voxelised_point_amd", "libts.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libts.so not built")

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x1002)   # not 16-byte aligned
BIG = 1 << 40


@pytest.fixture(scope="module")
def ts():
    from convolution_voxelised_point_amd import ts as mod
    return mod


def attn(ts, **changes):
    fields = dict(dtype=ts.TS_F16, hq=4, hk=2, d=32, ndim=3, scale=0.2, cap=0.0, nq=100, nk=100, n_sets=3,
                  q_stride=128, k_stride=64, v_stride=64, o_stride=128, q_starts=0x1000, k_starts=0x1000,
                  slopes=None, q_coords=None, k_coords=None)
    fields.update(changes)
    return ts.TsAttn(**fields)


BAD_ATTN = [
    (dict(dtype=7), "INVALID_ARG"),
    (dict(dtype=0), "UNSUPPORTED"),                       # fp32
    (dict(hq=0), "INVALID_ARG"),
    (dict(hk=0), "INVALID_ARG"),
    (dict(hq=3), "INVALID_ARG"),                          # not a multiple of hk
    (dict(d=0), "INVALID_ARG"),
    (dict(d=136, q_stride=1024, k_stride=512, v_stride=512, o_stride=1024), "UNSUPPORTED"),
    (dict(hq=65536 * 2, hk=2, d=1, q_stride=1 << 20, o_stride=1 << 20), "UNSUPPORTED"),
    (dict(nq=-1), "INVALID_ARG"),
    (dict(nk=-1), "INVALID_ARG"),
    (dict(n_sets=-1), "INVALID_ARG"),
    (dict(nq=1 << 30), "UNSUPPORTED"),                    # rows times heads past 31 bits
    (dict(nk=1 << 31), "UNSUPPORTED"),
    (dict(n_sets=1 << 31), "UNSUPPORTED"),
    (dict(q_stride=127), "INVALID_ARG"),
    (dict(k_stride=63), "INVALID_ARG"),
    (dict(v_stride=63), "INVALID_ARG"),
    (dict(o_stride=127), "INVALID_ARG"),
    (dict(k_stride=(1 << 23) + 8), "UNSUPPORTED"),
    (dict(scale=float("nan")), "INVALID_ARG"),
    (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(cap=-1.0), "INVALID_ARG"),
    (dict(cap=float("nan")), "INVALID_ARG"),
    (dict(scale=1e30, cap=1e-30), "INVALID_ARG"),         # scale / cap past the largest float
    (dict(cap=1025.0), "UNSUPPORTED"),
    (dict(q_starts=None), "INVALID_ARG"),
    (dict(k_starts=None, nk=99), "INVALID_ARG"),          # one list of starts: one number of rows
    (dict(slopes=0x1000), "INVALID_ARG"),                 # a slope without coordinates
    (dict(slopes=0x1000, q_coords=0x1000, ndim=4), "INVALID_ARG"),
    (dict(slopes=0x1000, q_coords=0x1000, nk=99), "INVALID_ARG"),
]


@pytest.mark.parametrize("changes,want", BAD_ATTN, ids=[str(b[0]) for b in BAD_ATTN])
def test_attention_refuses(ts, changes, want):
    at = attn(ts, **changes)
    status = getattr(ts, "TS_ERR_" + want)
    ref = ctypes.byref(at)
    assert ts._lib_attn_fwd(ref, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None, None) == status
    assert ts._lib_attn_bwd(ref, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None, None) == status
    assert ts._lib_attn_workspace_bytes(ref, 0) == 0
    assert ts._lib_attn_workspace_bytes(ref, 1) == 0


def test_attention_pointers(ts):
    bad = ts.TS_ERR_INVALID_ARG
    at = attn(ts)
    ref = ctypes.byref(at)
    assert ts._lib_attn_fwd(None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None, None) == bad
    assert ts._lib_attn_workspace_bytes(None, 0) == 0
    for i in range(5):                                     # q, k, v, out, lse
        for wrong in (None, ODD) if i < 4 else (None,):
            args = [FAKE] * 5
            args[i] = wrong
            assert ts._lib_attn_fwd(ref, *args, FAKE, BIG, None, None) == bad, (i, wrong)
    for i in range(9):                                     # q, k, v, out, lse, dout, dq, dk, dv
        for wrong in (None, ODD) if i != 4 else (None,):
            args = [FAKE] * 9
            args[i] = wrong
            assert ts._lib_attn_bwd(ref, *args, FAKE, BIG, None, None) == bad, (i, wrong)


def test_attention_workspace(ts):
    bad = ts.TS_ERR_INVALID_ARG
    sizes = lambda at: [ts._lib_attn_workspace_bytes(ctypes.byref(at), b) for b in (0, 1)]
    # short sets: nothing forward, one float per row and head (in whole 256 bytes) backward
    assert sizes(attn(ts)) == [0, 1792]
    # one row against many: the walk over the keys is split
    long = attn(ts, nq=1, nk=100000, n_sets=1)
    fwd, bwd = sizes(long)
    assert fwd > 0 and fwd % (4 * 4 * (32 + 2)) == 0 and bwd > 0
    ref = ctypes.byref(long)
    for ws, n in ((None, fwd), (FAKE, fwd - 1), (ODD, fwd)):
        assert ts._lib_attn_fwd(ref, FAKE, FAKE, FAKE, FAKE, FAKE, ws, n, None, None) == bad
    for ws, n in ((None, bwd), (FAKE, bwd - 1), (ODD, bwd)):
        assert ts._lib_attn_bwd(ref, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ws, n, None, None) == bad
    # heads of a width that is no multiple of 8 are copied: more than the same sizes at 32
    odd = sizes(attn(ts, d=31))
    assert odd[0] >= 2 * 100 * (4 + 2) * 32 * 2 and odd[1] >= 4 * 100 * (4 + 2) * 32 * 2
    # the largest sizes allowed answer without overflow
    assert min(sizes(attn(ts, nq=(1 << 29) - 1, nk=(1 << 30) - 1, d=33, q_stride=256, k_stride=128, v_stride=128,
                          o_stride=256))) > 1 << 36
    # nothing to do
    assert sizes(attn(ts, nq=0, nk=0, n_sets=0)) == [0, 0]


def test_norm_and_pack_refuse(ts):
    bad = ts.TS_ERR_INVALID_ARG
    good = ts.TsAct8(0x1000, 0x1000)
    act, half, none = ctypes.byref(good), ctypes.byref(ts.TsAct8(0x1000, None)), ctypes.byref(ts.TsAct8(None, 0x1000))
    for n, c, dt in ((-1, 8, 1), (1 << 31, 8, 1), (8, 0, 1), (8, (1 << 16) + 1, 1), (8, 8, 7)):
        assert ts._lib_act_pack(FAKE, n, c, dt, act, None) == bad
        assert ts._lib_act_unpack(act, n, c, FAKE, dt, None) == bad
        assert ts._lib_norm_fwd(FAKE, None, FAKE, n, c, 1e-6, dt, FAKE, FAKE, FAKE, None, None, None) == bad
        assert ts._lib_norm_bwd(FAKE, FAKE, None, FAKE, FAKE, None, n, c, dt, FAKE, FAKE, FAKE, BIG, None) == bad
    assert ts._lib_act_pack(None, 8, 8, 1, act, None) == bad
    for a in (None, half, none):
        assert ts._lib_act_pack(FAKE, 8, 8, 1, a, None) == bad
        assert ts._lib_act_unpack(a, 8, 8, FAKE, 1, None) == bad
    assert ts._lib_act_unpack(act, 8, 8, None, 1, None) == bad

    def fwd(x=FAKE, w=FAKE, eps=1e-6, h=None, y=FAKE, y8=None, h8=None):
        return ts._lib_norm_fwd(x, None, w, 8, 8, eps, 1, h, y, None, y8, h8, None)
    assert fwd(x=None) == bad and fwd(w=None) == bad
    assert fwd(eps=-1.0) == bad and fwd(eps=float("nan")) == bad and fwd(eps=float("inf")) == bad
    assert fwd(y=None) == bad                              # nothing asked for
    assert fwd(y8=half) == bad and fwd(h8=none) == bad

    need = ts._lib_norm_workspace_bytes(8, 8)
    assert need >= 8 * 4 and ts._lib_norm_workspace_bytes(-1, 8) == 0 and ts._lib_norm_workspace_bytes(8, 0) == 0

    def bwd(dy=FAKE, h=FAKE, h8=None, w=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, ws=FAKE, n=need):
        return ts._lib_norm_bwd(dy, h, h8, w, rstd, None, 8, 8, 1, dx, dw, ws, n, None)
    for name in ("dy", "h", "w", "rstd", "dx", "dw", "ws"):
        assert bwd(**{name: None}) == bad, name
    assert bwd(h8=act) == bad                              # h and h8: one of the two
    assert bwd(h=None, h8=half) == bad
    assert bwd(n=need - 1) == bad


def test_weight_gradient_from_8_bits_refuses(ts):
    bad = ts.TS_ERR_INVALID_ARG
    act, half = ctypes.byref(ts.TsAct8(0x1000, 0x1000)), ctypes.byref(ts.TsAct8(0x1000, None))
    km = ts.TsKmap()
    km.kvol, km.stride, km.n_in, km.n_out_cap, km.flags = 27, 1, 100, 100, ts.TS_KMAP_PAIRS
    km.fwd.n_dest_cap, km.fwd.n_tiles, km.fwd.row_mask = 100, 7, 0x3000
    need = ts._lib_conv_wgrad_act8_workspace_bytes(ctypes.byref(km), 32, 16)
    assert need > 0
    assert ts._lib_conv_wgrad_act8_workspace_bytes(None, 32, 16) == 0
    assert ts._lib_conv_wgrad_act8_workspace_bytes(ctypes.byref(km), 0, 16) == 0

    def call(m=km, x=act, cin=32, dy=FAKE, cout=16, dt=1, dw=FAKE, ws=FAKE, n=need):
        return ts._lib_conv_bwd_wgrad_act8(ctypes.byref(m) if m else None, x, cin, dy, cout, dt, dw, ws, n, None)
    assert call(m=None) == bad and call(x=None) == bad and call(x=half) == bad
    assert call(cin=0) == bad and call(cout=0) == bad and call(cin=(1 << 16) + 1) == bad
    assert call(dt=9) == bad and call(dt=0) == ts.TS_ERR_UNSUPPORTED
    assert call(dy=None) == bad and call(dw=None) == bad and call(ws=None) == bad and call(n=need - 1) == bad
    km.flags = 0
    assert call() == bad                                   # needs the pair lists
    km.flags, km.kvol = ts.TS_KMAP_PAIRS, 0
    assert call() == bad
