"""Every way the library cuts up an attention call, forward and backward,
against the fp64 implementation and bounds of test_gpu_attn.py."""
import pytest
import torch

from attn_forms import FORMS
from test_gpu_attn import build, check, ref_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS, ids=[f[0] for f in FORMS])
def test_form(ts, form):
    name, dt, lq, lk, hq, hk, d, cap, bias, _, _ = form
    dtype, q, k, v, dout, qs, ks, opt = build((name, dt, lq, lk, hq, hk, d, cap, bias, 3))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = ts.attn_fwd(q, k, v, qs, ks, err_flags=flags, **opt)
    grads = ts.attn_bwd(dout, q, k, v, out, lse, qs, ks, err_flags=flags, **opt)
    assert int(flags) == 0
    ref, tol = ref_of(dtype, q, k, v, qs, ks, opt, dout)
    check(dict(zip(("dq", "dk", "dv"), grads), out=out, lse=lse), ref, tol, name)
    again = ts.attn_bwd(dout, q, k, v, *ts.attn_fwd(q, k, v, qs, ks, **opt), qs, ks, **opt)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("form", [f for f in FORMS if f[0] in ("rows_split", "share_split", "two_shared")], ids=lambda f: f[0])
def test_lost_rows_and_dropped_keys(ts, form):
    """Infinite keys and rows without a finite score where walks are split: what is left is as without them."""
    name, dt, lq, lk, hq, hk, d, cap, bias, _, _ = form
    dtype, q, k, v, dout, qs, ks, opt = build((name, dt, lq, lk, hq, hk, d, 0.0, bias, 3))
    q[:, :, 0] = q[:, :, 0].abs() + 0.1
    k[::5, :, 0] = -torch.inf
    got = {}
    got["out"], got["lse"] = ts.attn_fwd(q, k, v, qs, ks, **opt)
    got.update(zip(("dq", "dk", "dv"), ts.attn_bwd(dout, q, k, v, got["out"], got["lse"], qs, ks, **opt)))
    assert all(torch.isfinite(got[n]).all() for n in ("out", "dq", "dk", "dv"))
    assert not got["dk"][::5].any() and not got["dv"][::5].any()
    # the reference with those keys in no set's way: the rest, packed
    keep = torch.arange(k.shape[0]) % 5 != 0
    at = keep.cumsum(0).tolist()
    cut = torch.tensor([0 if s == 0 else at[s - 1] for s in (qs if ks is None else ks).tolist()])
    kc = opt.get("k_coords")
    kc = opt["q_coords"] if kc is None else kc
    rest = dict(opt, k_coords=kc[keep.cuda()])
    ref, tol = ref_of(dtype, q, k[keep.cuda()], v[keep.cuda()], qs, cut, rest, dout)
    got["dk"], got["dv"] = got["dk"][keep.cuda()], got["dv"][keep.cuda()]
    check(got, ref, tol, f"{name}: dropped keys")
    # and queries that see nothing
    k = k.clone()
    k[:, :, 0] = torch.where(k[:, :, 0].isinf(), 1.0, k[:, :, 0].abs() + 0.1)
    k[:, :, 1:] = 0.0
    q[::3, :, 0], q[::3, :, 1:] = -torch.inf, 0.0
    dout[::3] = torch.nan
    out, lse = ts.attn_fwd(q, k, v, qs, ks, **opt)
    dq, dk, dv = ts.attn_bwd(dout, q, k, v, out, lse, qs, ks, **opt)
    assert not out[::3].any() and not dq[::3].any() and (lse[::3] == -torch.inf).all()
    q2, dout2 = q.clone(), dout.clone()
    q2[::3], dout2[::3] = 0.0, 0.0  # rows that add nothing
    out2, lse2 = ts.attn_fwd(q2, k, v, qs, ks, **opt)
    want = ts.attn_bwd(dout2, q2, k, v, out2, lse2, qs, ks, **opt)
    u = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}[dtype]  # two roundings of each term and of the result
    for g, w in zip((dk, dv), want[1:]):
        assert float((g.double() - w.double()).norm() / w.double().norm()) <= u
