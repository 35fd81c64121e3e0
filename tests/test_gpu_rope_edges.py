"""Rotation of query and key heads where its parts must not touch each other: channels that are
not turned, beside values that are no numbers."""
import pytest
import torch

from test_gpu_rope import DT, inputs

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
PARTLY = [  # d, pairs: channels left over behind whole and cut accesses, an odd one last, one pair turned
    (40, (6, 6, 4)), (32, (3, 3, 3)), (41, (6, 6, 4)), (77, (5, 0, 6)), (24, (1, 0)), (7, (1, 1)), (128, (20, 20, 20)),
]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("il", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("shape", PARTLY, ids=str)
def test_channels_that_are_not_turned(ts, shape, il, dt):
    """An infinite or NaN value in one of them stays there, in the results and in the gradients."""
    d, pairs = shape
    q, k, coords, freqs, pairs, _, _, dq, dk = inputs(dt, 30, 2, 1, d, pairs, norm=False)
    q, dq, kw = q.clone(), dq.clone(), dict(interleaved=il)
    want = ts.rope_fwd(q, k, coords, freqs, pairs, **kw)[0]
    back = ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, **kw).dq
    at = [(i, i % 2, 2 * sum(pairs) + i % (d - 2 * sum(pairs)), (INF, -INF, NAN)[i % 3]) for i in range(30)]
    for r, h, c, v in at:
        q[r, h, c] = dq[r, h, c] = v
    y = ts.rope_fwd(q, k, coords, freqs, pairs, **kw)[0]
    g = ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, **kw).dq
    for r, h, c, v in at:
        for got, ref in ((y, want), (g, back)):
            assert torch.equal(got[r, h, c].cpu(), torch.tensor(v).to(got.dtype)) or (v != v and bool(got[r, h, c].isnan())), (r, h, c, v)
            got[r, h, c] = ref[r, h, c]
    assert torch.equal(y, want) and torch.equal(g, back)


@pytest.mark.parametrize("il", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("shape", PARTLY, ids=str)
def test_channels_that_are_not_turned_with_norm(ts, shape, il):
    """With the norm an infinite one makes the others of its head zeros (x / infinity) and itself NaN, as the formula has
    it; an infinite gradient there reaches no other channel of dw."""
    d, pairs = shape
    q, k, coords, freqs, pairs, wq, wk, dq, dk = inputs("f32", 30, 2, 1, d, pairs)
    q, dq, kw, c = q.clone(), dq.clone(), dict(wq=wq, wk=wk, interleaved=il), 2 * sum(pairs)
    dq[3, 1, c] = INF
    dw = ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, **kw).dwq
    assert not dw[c].isfinite() and dw.isfinite().sum() == d - 1
    q[5, 0, c] = INF
    y = ts.rope_fwd(q, k, coords, freqs, pairs, **kw)[0]
    assert y[5, 0, c].isnan() and (y[5, 0] == 0).sum() == d - 1


@pytest.mark.parametrize("n", [0, 30])
@pytest.mark.parametrize("hq,hk", [(0, None), (0, 0), (2, 0), (0, 1)])
def test_gradients_of_weights_without_heads(ts, hq, hk, n):
    """An empty sum is zero, whatever the memory held before."""
    d, pairs = 32, (8, 8)
    new = lambda h: None if h is None else torch.randn(n, h, d, device="cuda")  # noqa: E731
    q, k, dq, dk = new(hq), new(hk), new(hq), new(hk)
    wq, wk = torch.ones(d, device="cuda"), None if hk is None else torch.ones(d, device="cuda")
    coords, freqs = torch.ones(n, 3, dtype=torch.int32, device="cuda"), ts.rope_freqs(pairs)
    junk = [torch.full((d,), NAN, device="cuda") for _ in range(64)]
    del junk  # what the allocator hands out next
    r = ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, wq=wq, wk=wk)
    for h, dw in ((hq, r.dwq), (hk, r.dwk)):
        assert (dw is None) == (h is None) and (dw is None or bool(dw.isfinite().all()))
        assert h is None or n * h > 0 or (dw == 0).all()


@pytest.mark.parametrize("reach", [30, 1 << 20])
def test_sine_and_cosine(ts, reach):
    """Of (1, 0) the rotation returns cosine and sine themselves.  Over an eighth of a turn either way, in units of
    E = 2^-24: the angle x <= 0.79 is rounded once, by E / 2, which moves the sine by that and the cosine by 0.71 of it; the
    last addition is off by E / 2 of a result below 1.  Sine: x^3 <= 0.49 by E / 4 and its factor 1/6 by E / 16, 0.1 E in all.
    Cosine: x^2 <= 0.62 by E / 2, which moves it by 0.46 of that, and the factor of x^2 by E / 4: 0.4 E in all.  Coefficients and
    the terms left out 0.05 E, the 2^19 turns of the farthest positions 0.01 E.  So sine 1.16 E, cosine 1.32 E."""
    n, p = 200000, 16
    g = torch.Generator().manual_seed(reach)
    q = torch.zeros(n, 1, 2 * p, device="cuda")
    q[..., :p] = 1.0
    coords = torch.randint(-reach, reach + 1, (n, 3), generator=g, dtype=torch.int32)
    freqs = torch.rand(p, generator=g) * 3
    y = ts.rope_fwd(q, None, coords.cuda(), freqs.cuda(), (p // 2, p // 2))[0][:, 0].cpu().double()
    at = torch.tensor([1] * (p // 2) + [2] * (p // 2))
    angle = coords[:, at].double() * freqs.double()  # exact: 21 and 24 bits
    for got, ref in ((y[:, :p], torch.cos(angle)), (y[:, p:], torch.sin(angle))):
        assert float((got - ref).abs().max()) <= 1.4 * 2.0 ** -24
