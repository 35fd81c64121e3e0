"""Attention within packed sets where it can go wrong at its edges: views the
library has to be given copies of, starts without rows, rows far apart,
coordinates far from the origin, the range of fp16, and rows that nothing is
left of.  The reference and its bounds are those of test_gpu_attn.py."""
import math

import pytest
import torch

from test_gpu_attn import check, reference, starts

pytestmark = pytest.mark.gpu


def half(*shape, seed, dtype=torch.float16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def test_one_row_at_any_address(ts):
    """One row of a matrix of odd width is a row like any other, wherever it begins."""
    hq, hk, d, n = 4, 2, 16, 300
    m = half(9, 97, seed=1)
    k, v = half(n, hk, d, seed=2), half(n, hk, d, seed=3)
    qs, ks = starts([1]), starts([n])
    row = lambda t, i: t[:, :hq * d].unflatten(1, (hq, d))[i:i + 1]  # noqa: E731
    for i in range(9):
        q, dout = row(m, i), row(m, 8 - i)
        out, lse = ts.attn_fwd(q, k, v, qs, ks)
        want = ts.attn_fwd(q.clone(), k, v, qs, ks)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        wide = torch.empty_like(m)
        mine = row(wide, i)
        mine.copy_(out)
        back = ts.attn_bwd(dout, q, k, v, mine, lse, qs, ks)
        for a, b in zip(back, ts.attn_bwd(dout.clone(), q.clone(), k, v, out, lse, qs, ks)):
            assert torch.equal(a, b)
        into = (row(torch.zeros_like(m), i), torch.zeros_like(k), torch.zeros_like(v))
        got = ts.attn_bwd(dout, q, k, v, mine, lse, qs, ks, into=into)
        assert all(a is b and torch.equal(a, c) for a, b, c in zip(got, into, back))
    # one key
    q = half(5, hq, d, seed=4)
    k1, v1 = (m[:, o:o + hk * d].unflatten(1, (hk, d))[3:4] for o in (0, 33))
    out, lse = ts.attn_fwd(q, k1, v1, starts([5]), starts([1]))
    assert torch.equal(out, v1.repeat_interleave(hq // hk, 1).expand(5, hq, d))


def test_bad_starts_without_query_rows(ts):
    """The flag does not need a query row to be raised."""
    q, k = half(0, 1, 16, seed=1), half(64, 1, 16, seed=2)
    lse = torch.zeros(0, 1, device="cuda")
    for qs, ks, bad in (([0, 0], [0, 65], True), ([0, 0, 0], [0, 40, 30], True), ([0, 1], [0, 64], True), ([-1, 0], [0, 64], True),
                        ([0, 0], [0, 64], False), ([0, 0, 0], [3, 3, 60], False), ([0], [64], False), ([0], [65], True)):
        args = torch.tensor(qs, device="cuda"), torch.tensor(ks, device="cuda")
        want = ts.TS_FLAG_RANGE if bad else 0
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, _ = ts.attn_fwd(q, k, k, *args, err_flags=flags)
        assert int(flags) == want and out.shape == (0, 1, 16), (qs, ks)
        flags.zero_()
        _, dk, dv = ts.attn_bwd(q, q, k, k, q, lse, *args, err_flags=flags)
        assert int(flags) == want and not dk.any() and not dv.any(), (qs, ks)
    ts.attn_fwd(q, k, k, torch.tensor([0, 0], device="cuda"), torch.tensor([0, 65], device="cuda"))  # nobody asks


@pytest.mark.parametrize("stride", [(1 << 22) + 8, 1 << 23])
def test_padded_channels_of_rows_far_apart(ts, stride):
    """Head widths between 32 and 64 are computed as 64 with zeros beside them, however far apart the rows of a tile are:
    an infinite key drops itself and no other."""
    n, d = 120, 40
    wide = torch.empty((n - 1) * stride + 2 * d, dtype=torch.float16, device="cuda")
    k, v = (wide[o:].as_strided((n, 1, d), (stride, d, 1)) for o in (0, d))
    g = torch.Generator("cuda").manual_seed(7)
    k.copy_(torch.randn(n, 1, d, generator=g, device="cuda"))
    v.copy_(torch.randn(n, 1, d, generator=g, device="cuda"))
    q = torch.randn(3, 1, d, generator=g, device="cuda").half().abs() + 0.1
    k[:20, 0, 1] = -math.inf
    qs, ks = starts([3]), starts([n])
    out, lse = ts.attn_fwd(q, k, v, qs, ks)
    rest, _ = ts.attn_fwd(q, k.clone(), v.clone(), qs, ks)
    assert torch.isfinite(out).all() and torch.equal(out, rest)
    ref, tol = reference(q, k[20:], v[20:], [0, 3], [0, n - 20], d ** -0.5)
    check({"out": out, "lse": lse}, ref, tol, "rows far apart")


@pytest.mark.parametrize("origin", [1 << 25, -(1 << 30), (1 << 30) - 100])
def test_coordinates_far_from_the_origin(ts, origin):
    """A distance depends on the coordinates' differences alone, which are exact."""
    n, h, d = 150, 2, 32
    q, k, v, dout = (half(n, h, d, seed=s) for s in range(4))
    gen = torch.Generator().manual_seed(5)
    opt = dict(slopes=torch.tensor([0.5, 1.0], device="cuda"))
    qs = starts([90, 60])
    for ndim in (2, 3):
        near = torch.randint(-40, 40, (n, ndim + 1), generator=gen, dtype=torch.int32).cuda()
        at = near + torch.tensor([0] + [origin] * ndim, dtype=torch.int32, device="cuda")
        a, b = [], []
        for c, res in ((near, a), (at, b)):
            out, lse = ts.attn_fwd(q, k, v, qs, q_coords=c, **opt)
            res += [out, lse, *ts.attn_bwd(dout, q, k, v, out, lse, qs, q_coords=c, **opt)]
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        ref, tol = reference(q, k, v, [0, 90, 150], [0, 90, 150], d ** -0.5, slopes=opt["slopes"], qc=at, kc=at, dout=dout)
        check(dict(zip(("out", "lse", "dq", "dk", "dv"), b)), ref, tol, f"origin {origin}")


@pytest.mark.parametrize("cap", [0.0, 40.0])
@pytest.mark.parametrize("nq,hk,n", [(1, 1, 500), (100, 2, 400), (1100, 64, 500)])
def test_small_probabilities_in_fp16(ts, nq, hk, n, cap):
    """Many keys 2^-26 below a row's largest are a part of its result.  A probability is rounded as an fp16 number once
    the row's largest is at least 2^7: to 2^-11 of itself, and never by more than 2^-32 of the largest.  (A capped score
    is good to cap 2^-21.)"""
    d = 16
    q = torch.zeros(nq, hk, d, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    k, v = (torch.zeros(n, hk, d, dtype=torch.float16, device="cuda") for _ in range(2))
    v[:, :, 1] = 30000.0
    for at in (0, n // 2, n - 1):
        k[:, :, 0] = 0.0
        k[at, :, 0] = 18.09375
        v[:, :, 1] = 30000.0
        v[at] = 0.0
        out, _ = ts.attn_fwd(q, k, v, starts([nq]), starts([n]), scale=1.0, cap=cap)
        top = cap * math.tanh(18.09375 / cap) if cap else 18.09375
        small = 30000.0 / (n - 1 + math.exp(top))
        want = (n - 1) * small
        bar = want * (2.0 ** -10 + 2.0 ** -18 + cap * 2.0 ** -20) + (n - 1) * 30000.0 * 2.0 ** -32
        assert float((out[:, :, 1].double() - want).abs().max()) <= bar, (at, float(out[0, 0, 1]), want)


@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_value_gradients_over_many_keys_in_fp16(ts, cap):
    """dv = p dout where p lies far below fp16's smallest number (equal scores over 3,000,000 keys): to the result's own
    rounding and that of p, 2^-11 each; exp2 and lse add less than 2^-18, a capped score cap 2^-21 (and its lse)."""
    n, d = 3_000_000, 8
    q, dout = torch.ones(1, 1, d, dtype=torch.float16, device="cuda"), torch.full((1, 1, d), 20000.0, dtype=torch.float16, device="cuda")
    k = torch.zeros(n, 1, d, dtype=torch.float16, device="cuda")
    v = torch.ones_like(k)
    qs, ks = starts([1]), starts([n])
    out, lse = ts.attn_fwd(q, k, v, qs, ks, cap=cap)
    _, _, dv = ts.attn_bwd(dout, q, k, v, out, lse, qs, ks, cap=cap)
    want = 20000.0 / n
    assert float((dv.double() - want).abs().max()) <= want * (2.0 ** -10 + 2.0 ** -18 + cap * 2.0 ** -20)
    # one key that takes everything: the largest p there is
    out, lse = ts.attn_fwd(q, k[:1], v[:1], qs, starts([1]), cap=cap)
    _, _, dv = ts.attn_bwd(dout, q, k[:1], v[:1], out, lse, qs, starts([1]), cap=cap)
    assert (dv == 20000.0).all()


# query rows, keys, hq, hk, d: the waves share the keys; one column block a wave; two
FORMS = [(3, 40, 1, 1, 16), (3, 2000, 4, 2, 40), (70, 90, 4, 2, 32), (130, 200, 2, 1, 128), (1100, 700, 64, 64, 16)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("nq,nk,hq,hk,d", FORMS, ids=str)
def test_gradients_with_infinite_keys_and_queries(ts, nq, nk, hq, hk, d, dtype):
    """Keys dropped by scores of -inf leave the gradients of the rest as if they were not there, and a row whose scores are
    all -inf has none, whatever its q and dout hold."""
    scale = d ** -0.5
    q, dout = half(nq, hq, d, seed=1, dtype=dtype), half(nq, hq, d, seed=2, dtype=dtype)
    k, v = half(nk, hk, d, seed=3, dtype=dtype), half(nk, hk, d, seed=4, dtype=dtype)
    q[:, :, 0] = q[:, :, 0].abs() + 0.1
    kept = torch.arange(nk) % 3 != 1
    kept[nk // 2:] &= torch.arange(nk // 2, nk) % 7 != 0
    k[~kept.cuda(), :, 0] = -math.inf
    qs, ks = starts([nq]), starts([nk])
    out, lse = ts.attn_fwd(q, k, v, qs, ks)
    dq, dk, dv = ts.attn_bwd(dout, q, k, v, out, lse, qs, ks)
    kn, vn = k[kept.cuda()].contiguous(), v[kept.cuda()].contiguous()
    ref, tol = reference(q, kn, vn, [0, nq], [0, int(kept.sum())], scale, dout=dout, dtype=dtype)
    got = {"out": out, "lse": lse, "dq": dq, "dk": dk[kept.cuda()], "dv": dv[kept.cuda()]}
    check(got, ref, tol, "dropped keys")
    assert (dk[~kept.cuda()] == 0).all() and (dv[~kept.cuda()] == 0).all()
    # rows that see nothing
    k, lost = kn, torch.arange(nq) % 2 == 0
    k[:, :, 0] = k[:, :, 0].abs() + 0.1
    q[lost.cuda(), :, 0] = -math.inf
    q[lost.cuda(), :, 1] = 0.0
    k[:, :, 2:] = 0.0
    q[lost.cuda(), :, 2:] = 0.0
    dout[lost.cuda()] = math.nan
    n2 = k.shape[0]
    ks = starts([n2])
    out, lse = ts.attn_fwd(q, k, vn, qs, ks)
    dq, dk, dv = ts.attn_bwd(dout, q, k, vn, out, lse, qs, ks)
    assert (out[lost.cuda()] == 0).all() and (lse[lost.cuda()] == -math.inf).all() and (dq[lost.cuda()] == 0).all()
    seen = ~lost.cuda()
    ref, tol = reference(q[seen], k, vn, [0, int(seen.sum())], [0, n2], scale, dout=dout[seen], dtype=dtype)
    got = {"out": out[seen], "lse": lse[seen], "dq": dq[seen], "dk": dk, "dv": dv}
    check(got, ref, tol, "rows without scores")


def test_infinite_keys_between_sets_and_heads(ts):
    """Head after head in one block, sets with and without dropped keys: as each set by itself."""
    n, h, d, m = 1100, 4, 32, 40
    q, k, v, dout = (half(n * m, h, d, seed=s) for s in range(4))
    q[:, :, 0] = q[:, :, 0].abs() + 0.1
    k[7 * m + 3, 1, 0] = -math.inf   # set 7, the second head
    k[9 * m + 30, :, 0] = -math.inf  # set 9, every head
    qs = starts([m] * n)
    out, lse = ts.attn_fwd(q, k, v, qs)
    whole = (out, lse, *ts.attn_bwd(dout, q, k, v, out, lse, qs))
    assert all(torch.isfinite(t).all() for t in whole)
    clean = k.clone()
    clean[clean.isinf()] = 0.0
    out, lse = ts.attn_fwd(q, clean, v, qs)
    plain = (out, lse, *ts.attn_bwd(dout, q, clean, v, out, lse, qs))
    rest = [i for i in range(n * m) if i // m not in (7, 9)]
    for a, b in zip(whole, plain):
        assert torch.equal(a[rest], b[rest])
        assert torch.equal(a[7 * m:8 * m, [0, 2, 3]], b[7 * m:8 * m, [0, 2, 3]])
    for s, drop in ((7, 3), (9, 30)):
        rows = slice(s * m, s * m + m)
        keep = [i for i in range(m) if i != drop]
        ref, tol = reference(q[rows], k[rows][keep], v[rows][keep], [0, m], [0, m - 1], d ** -0.5, dout=dout[rows])
        heads = [1] if s == 7 else [0, 1, 2, 3]
        got = dict(zip(("out", "lse", "dq", "dk", "dv"), (t[rows][keep] if i > 2 else t[rows] for i, t in enumerate(whole))))
        for name in got:
            check({name: got[name][:, heads]}, {name: ref[name][:, heads]}, {name: tol[name][:, heads]}, f"set {s}")


def test_gradients_of_columns_take_one_matrix(ts):
    """Operands that are columns of one matrix get gradients that are columns of one, no larger than it."""
    n, hq, hk, d = 200, 4, 2, 32
    qs = starts([120, 80])
    dout = half(n, hq, d, seed=1)
    heads = lambda t, *w: t.view(n, -1, d).split(w, dim=1)  # noqa: E731
    m = half(n, (hq + 2 * hk) * d, seed=2)
    q, k, v = heads(m, hq, hk, hk)
    out, lse = ts.attn_fwd(q, k, v, qs)
    want = ts.attn_bwd(dout, q.contiguous(), k.contiguous(), v.contiguous(), out, lse, qs)
    for tensors, bytes_ in (((q, k, v), m.nbytes),
                            ((q.contiguous(), k, v), q.nbytes + m.nbytes),
                            ((q.contiguous(), k.contiguous(), v.contiguous()), q.nbytes + 2 * k.nbytes)):
        got = ts.attn_bwd(dout, *tensors, out, lse, qs)
        assert all(torch.equal(a, b) and a.stride() == t.stride() for a, b, t in zip(got, want, tensors))
        held = {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in got}
        assert sum(held.values()) <= bytes_
    # the same keys as values, and columns that overlap: apart
    out, lse = ts.attn_fwd(q, k, k, qs)
    _, dk, dv = ts.attn_bwd(dout, q, k, k, out, lse, qs)
    _, dk2, dv2 = ts.attn_bwd(dout, q, k, k.clone(), out, lse, qs)
    assert torch.equal(dk, dk2) and torch.equal(dv, dv2) and not torch.equal(dk, dv)
