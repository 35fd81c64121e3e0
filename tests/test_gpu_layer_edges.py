"""Calls of rotation, routing, products by expert and combining sum that ts.h allows beside the usual ones: results over
inputs, bases that are not aligned, nothing to read."""
import pytest
import torch

from test_gpu_rope import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("il", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("d,pairs", [(32, (6, 6, 4)), (26, (3, 3, 3)), (77, (10, 10, 10))])
def test_rotation_gradients_over_the_inputs(ts, d, pairs, il, dt):
    """dx in the place of x, within a projected matrix."""
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs(dt, 700, 4, 2, d, pairs)
    want = ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, wq=wq, wk=wk, interleaved=il)
    got = ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, wq=wq, wk=wk, interleaved=il, into=(q, k))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(q, want.dq) and torch.equal(k, want.dk)


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,e,top", [(39, 8, 2), (5000, 64, 2), (700, 77, 5), (300, 512, 16), (50, 3, 3)])
def test_logit_gradients_over_the_logits(ts, n, e, top, dt):
    z = torch.randn(n, e, device="cuda").to(dt)
    r, dg = ts.route_fwd(z, top, over_all=True), torch.randn(n, top, device="cuda")
    want = ts.route_bwd(dg, z, r, over_all=True)
    code = {torch.float32: ts.TS_F32, torch.float16: ts.TS_F16, torch.bfloat16: ts.TS_BF16}[dt]
    assert ts._lib_route_bwd(dg.data_ptr(), z.data_ptr(), r.experts.data_ptr(), r.gates.data_ptr(), n, e, code, top, 1, z.data_ptr(),
                             torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(z, want)


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [40, 9000])
def test_logits_that_are_not_16_byte_aligned(ts, n, dt):
    z = torch.randn(n, 64, device="cuda").to(dt)
    at = torch.empty(n * 64 + 1, dtype=dt, device="cuda")[1:].view(n, 64)
    at.copy_(z)
    dg = torch.randn(n, 3, device="cuda")
    for over_all in (False, True):
        want, got = ts.route_fwd(z, 3, over_all=over_all), ts.route_fwd(at, 3, over_all=over_all)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(ts.route_bwd(dg, at, got, over_all=over_all), ts.route_bwd(dg, z, want, over_all=over_all))


@pytest.mark.parametrize("p,cin,cout", [(5, 64, 64), (5, 7, 9), (400, 64, 64), (400, 7, 9), (1300, 256, 256)])
def test_products_of_no_rows_of_x(ts, p, cin, cout):
    """Every row number is out of range: zeros, and the flag."""
    g = ts.Groups(torch.tensor([0, p // 2, p], device="cuda"), torch.zeros(p, dtype=torch.int32, device="cuda"))
    x, w = torch.empty(0, cin, device="cuda").half(), torch.randn(2, cin, 2 * cout, device="cuda").half()
    for f in (lambda flag: ts.group_fwd(x, w, g, err_flags=flag), lambda flag: torch.cat(ts.group_glu_fwd(x, w, g, True, err_flags=flag), 1),
              lambda flag: ts.group_wgrad(x, torch.randn(p, cout, device="cuda").half(), g, err_flags=flag)):
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert (f(flag) == 0).all() and int(flag) == ts.TS_FLAG_RANGE


def test_combining_sum_of_no_rows(ts):
    y, place = torch.empty(0, 24, device="cuda"), torch.full((30, 2), -1, dtype=torch.int32, device="cuda")
    gates, flag = torch.full((30, 2), float("nan"), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    assert (ts.combine_fwd(y, place, gates, err_flags=flag) == 0).all()
    dy, dgates = ts.combine_bwd(torch.randn(30, 24, device="cuda"), y, place, gates, err_flags=flag)
    assert dy.shape == (0, 24) and (dgates == 0).all() and int(flag) == 0
    place[3, 1] = 0
    assert (ts.combine_fwd(y, place, gates, err_flags=flag) == 0).all() and int(flag) == ts.TS_FLAG_RANGE
