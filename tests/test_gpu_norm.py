"""GPU parity of the residual RMS norm (forward, backward, 8-bit outputs) and of
activations in 8 bits (pack, unpack, the weight gradient that reads them)
against plain fp64 implementations.

Tolerances from the roundings (u = 0, 2^-11, 2^-8 for fp32, fp16, bf16; a sum of
m fp32 terms is off by at most m 2^-24 of the sum of their magnitudes): given with
each check.  h, and packing and unpacking, are exact."""
import math

import numpy as np
import pytest
import torch

import oracle
from convolution_voxelised_point_amd import synth
from helpers import U_OUT, assert_feature_close, dev

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -24


def held(x: np.ndarray):
    """(codes, scales, values) of the 8-bit form of x [n][c], in fp64."""
    n, c = x.shape
    nb = -(-c // 32)
    codes, scales, vals = np.zeros((n, c), np.int8), np.zeros((n, nb), np.uint8), np.zeros((n, c))
    for b in range(nb):
        p = x[:, 32 * b:32 * b + 32]
        with np.errstate(invalid="ignore"):
            top = np.abs(p).max(1)
        bad = ~np.isfinite(p).all(1)
        _, e = np.frexp(np.where(bad, 1.0, top))
        e = np.where(top > 0, e - 1 - 6 + 127, 1)
        e = np.maximum(e, 1)
        q = np.ldexp(1.0, e - 127)[:, None]
        with np.errstate(invalid="ignore"):
            k = np.clip(np.rint(np.where(bad[:, None], 0.0, p) / q), -127, 127)
        codes[:, 32 * b:32 * b + 32] = k
        scales[:, b] = np.where(bad, 255, e)
        vals[:, 32 * b:32 * b + 32] = np.where(bad[:, None], np.nan, k * q)
    return codes, scales, vals


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol, what):
    bad = ~(np.abs(f64(got) - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} over tolerance, worst {np.nanmax(np.abs(f64(got) - ref) / tol):.3g} times it"


SHAPES = [(1, 1), (1, 8), (3, 7), (39, 64), (257, 32), (100, 31), (65, 33), (70, 77), (1000, 128), (33, 100), (20, 256),
          (19, 300), (9, 512), (11, 520), (5, 1024), (7, 1030), (3, 2048), (4, 2049), (6, 2600), (2, 8200)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm(ts, shape, dt):
    n, c = shape
    dtype, u = DT[dt], U_OUT[DT[dt]]
    gen = torch.Generator().manual_seed(n * 10007 + c)
    x, res, dy, dh = ((torch.randn(n, c, generator=gen) * s).to(dtype).cuda() for s in (1.0, 3.0, 1.0, 1.0))
    w = (1 + 0.3 * torch.randn(c, generator=gen)).cuda()
    w[c // 2] = 0.0
    for residual in (None, res):
        r = ts.norm_fwd(x, w, residual=residual, eps=1e-5, y8=True, h8=True)
        h = x if residual is None else (x.float() + residual.float()).to(dtype)
        assert torch.equal(r.h, h)
        hh, ww = f64(h), f64(w)
        rstd = 1 / np.sqrt((hh * hh).mean(1, keepdims=True) + 1e-5)
        y = hh * rstd * ww
        ey = np.abs(y) * (c + 16) * E
        close(r.rstd, rstd[:, 0], rstd[:, 0] * (c + 8) * E, "rstd")
        close(r.y, y, u * np.abs(y) + ey + (2.0 ** -25 if dt == "f16" else 0) + 1e-30, "y")
        codes, scales, vals = held(hh)
        assert np.array_equal(r.h8.codes.cpu().numpy(), codes) and np.array_equal(r.h8.scales.cpu().numpy(), scales)
        # y8: half a quantum, a whole one past 127 quanta, and what y itself is off by
        quantum = np.repeat(np.ldexp(1.0, held(y)[1].astype(int) - 127), 32, axis=1)[:, :c]
        close(ts.act_unpack(r.y8, torch.float32), y, quantum * np.where(np.abs(y) > 127 * quantum, 1.0, 0.5) + ey + 1e-30, "y8")
        for grad_h in (None, dh):
            for kept, hv in ((r.h, hh), (r.h8, vals)):
                dx, dw = ts.norm_bwd(dy, kept, w, r.rstd, dh=grad_h)
                xn, d = hv * rstd, f64(dy)
                g = d * ww
                ref = rstd * (g - xn * (g * xn).mean(1, keepdims=True))
                size = rstd * (np.abs(g) + np.abs(xn) * np.abs(g * xn).mean(1, keepdims=True))
                if grad_h is not None:
                    ref = ref + f64(dh)
                tiny = 2.0 ** -25 if dt == "f16" else 1e-30
                close(dx, ref, u * np.abs(ref) + size * 2 * (c + 16) * E + np.abs(ref) * 2 * E + tiny, "dx")
                close(dw, (d * xn).sum(0), (n + c + 16) * E * np.abs(d * xn).sum(0) + 1e-30, "dw")


def test_norm_gradient_against_differences(ts):
    n, c, h = 6, 40, 1e-6
    gen = torch.Generator().manual_seed(9)
    x, dy, way = (torch.randn(n, c, generator=gen) for _ in range(3))
    w, wayw = 1 + 0.3 * torch.randn(c, generator=gen), torch.randn(c, generator=gen)
    r = ts.norm_fwd(x.cuda(), w.cuda(), eps=1e-5)
    dx, dw = ts.norm_bwd(dy.cuda(), r.h, w.cuda(), r.rstd)

    def loss(x, w):
        y = x / (x.square().mean(1, keepdim=True) + 1e-5).sqrt() * w
        return float((y * dy.double()).sum())

    X, W = x.double(), w.double()
    for got, step in ((float((dx.cpu().double() * way).sum()), lambda s: loss(X + s * way.double(), W)),
                      (float((dw.cpu().double() * wayw).sum()), lambda s: loss(X, W + s * wayw.double()))):
        # fp32 results against a difference good to about 1e-9
        assert abs(got - (step(h) - step(-h)) / (2 * h)) <= 1e-4 * max(1.0, abs(got))


def test_norm_views_and_in_place(ts):
    """Unaligned rows, and outputs over the inputs."""
    n, c = 50, 64
    for c in (64, 2304):
        gen = torch.Generator().manual_seed(4)
        base = torch.randn(n * c + 3, generator=gen).half().cuda()
        w = torch.randn(c + 1, generator=gen).cuda()[1:]
        res, dy = torch.randn(n, c, generator=gen).half().cuda(), torch.randn(n, c, generator=gen).half().cuda()
        for off in (0, 1, 3):
            x = base[off:off + n * c].view(n, c)
            a = ts.norm_fwd(x, w, residual=res, h8=True)
            b = ts.norm_fwd(x.clone(), w.clone(), residual=res, h8=True)
            assert torch.equal(a.y, b.y) and torch.equal(a.h, b.h) and torch.equal(a.h8.codes, b.h8.codes)
        x = base[:n * c].view(n, c).clone()
        y, rstd = torch.empty_like(x), torch.empty(n, device="cuda")
        keep = res.clone()
        ts.ts_norm_fwd(x, keep, w, 1e-6, h=keep, y=x, rstd=rstd)
        assert torch.equal(x, ts.norm_fwd(base[:n * c].view(n, c), w, residual=res).y)
        assert torch.equal(keep, (base[:n * c].view(n, c).float() + res.float()).half())
        ref, refw = ts.norm_bwd(dy, keep, w, rstd, dh=res)
        dw, ws = torch.empty(c, device="cuda"), torch.empty(ts.ts_norm_workspace_bytes(n, c), dtype=torch.uint8, device="cuda")
        grad = dy.clone()
        ts.ts_norm_bwd(grad, keep, None, w, rstd, res, grad, dw, ws)
        assert torch.equal(grad, ref) and torch.equal(dw, refw)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (100, 31), (65, 33), (300, 128), (40, 8), (17, 520)], ids=str)
def test_pack_and_unpack(ts, shape, dt):
    n, c = shape
    rng = np.random.default_rng(n + c)
    x = rng.standard_normal((n, c)) * 2.0 ** rng.integers(-12, 12, (n, 1))
    x[rng.random((n, c)) < 0.2] = 0.0
    xs = torch.from_numpy(x).to(DT[dt])
    if n > 10:
        xs[3] = 0.0
        xs[4, c // 2] = math.nan
        xs[5, c // 3] = -math.inf
        xs[6] = torch.finfo(DT[dt]).max
        xs[7] = torch.finfo(DT[dt]).tiny
        xs[8] = torch.finfo(DT[dt]).smallest_normal / 4  # below the normal range
        xs[9] = 127.75 if dt != "bf16" else 127.5        # rounds past 127 quanta
    codes, scales, vals = held(xs.double().numpy())
    a = ts.act_pack(xs.cuda())
    assert np.array_equal(a.codes.cpu().numpy(), codes) and np.array_equal(a.scales.cpu().numpy(), scales)
    for out in (DT[dt], torch.float32):
        got = ts.act_unpack(a, out).double().cpu().numpy()
        assert np.array_equal(got, vals, equal_nan=True)
    # packing what was read back changes nothing
    again = ts.act_pack(ts.act_unpack(a, DT[dt]))
    ok = np.isfinite(vals)
    assert np.array_equal(ts.act_unpack(again, torch.float32).double().cpu().numpy()[ok], vals[ok])


def test_pack_unaligned(ts):
    base = torch.randn(1000 * 64 + 5, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for off in (1, 3, 5):
        x = base[off:off + 64000].view(1000, 64)
        a, b = ts.act_pack(x), ts.act_pack(x.clone())
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    codes = torch.zeros(64 * 64 + 1, dtype=torch.int8, device="cuda")[1:].view(64, 64)
    a = ts.Act8(codes, torch.zeros(64, 2, dtype=torch.uint8, device="cuda"))
    ts.ts_act_pack(base[:4096].view(64, 64), a)
    assert torch.equal(ts.act_unpack(a, torch.bfloat16), ts.act_unpack(ts.act_pack(base[:4096].view(64, 64)), torch.bfloat16))


WGRAD = [
    # name, coords, ksize, stride, cin, cout, dtype
    ("subm_64_64", synth.make("lidar", scale=0.02).coords, 3, 1, 64, 64, "f16"),
    ("subm_128_128", synth.make("train", scale=0.005).coords, 3, 1, 128, 128, "bf16"),
    ("subm_192_160", synth.random_coords(41, 700, 3, 2, 12), 3, 1, 192, 160, "bf16"),
    ("pix_8_8", synth.random_coords(42, 3000, 2, 3, 50), 3, 1, 8, 8, "f16"),
    ("odd_13_21", synth.random_coords(43, 600, 3, 2, 11), 3, 1, 13, 21, "bf16"),
    ("mixed_24_48", synth.random_coords(44, 900, 3, 1, 14), 3, 1, 24, 48, "f16"),
    ("mixed_40_8", synth.random_coords(45, 900, 3, 1, 14), 1, 1, 40, 8, "bf16"),
    ("down_32_64", synth.make("down", scale=0.01).coords, 2, 2, 32, 64, "f16"),
    ("one_row", np.array([[0, 1, 2, 3]], np.int32), 3, 1, 16, 16, "f16"),
]


@pytest.mark.parametrize("case", WGRAD, ids=[c[0] for c in WGRAD])
def test_weight_gradient_from_8_bits(ts, case):
    name, c, k, s, cin, cout, dt = case
    cd = dev(c)
    tab = ts.HashTable(cd, 2.0)
    if s == 1:
        km = ts.build_kmap(cd, tab, k, 1, ts.TS_KMAP_PAIRS)
        oc = c
    else:
        out, n_out, otab = ts.strided_support(cd, s)
        km = ts.build_kmap(cd, tab, k, s, ts.TS_KMAP_PAIRS, out_coords=out, n_out=n_out, out_table=otab)
        oc = oracle.strided_support(c, s)
    tr = oracle.kmap(c, oc, k, s)
    x = torch.relu(synth.normal(51, (c.shape[0], cin), 1.0, dt))
    dy = torch.zeros(km.s.n_out_cap, cout, dtype=DT[dt])
    dy[:oc.shape[0]] = synth.normal(52, (oc.shape[0], cout), 1.0, dt)
    a = ts.act_pack(x.cuda())
    dw = ts.conv_wgrad_act8(km, a, dy.cuda())
    vals = torch.from_numpy(held(x.double().numpy())[2]).to(DT[dt])  # exact
    ref = oracle.conv_wgrad(tr, vals, dy[:oc.shape[0]], k ** (c.shape[1] - 1))
    # products of 16-bit values summed in fp32: the bound of fp32 features
    assert_feature_close(dw, ref, torch.float32, f"{name} weight gradient from 8 bits")
    assert torch.equal(dw, ts.conv_wgrad_act8(km, a, dy.cuda()))


def test_refusals(ts):
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    x, w = z(4, 16), z(16, dt=torch.float32)
    rstd = z(4, dt=torch.float32)
    a8 = ts.act_pack(x)
    for call in (lambda: ts.norm_fwd(x, w.half()), lambda: ts.norm_fwd(x, w[:8]), lambda: ts.norm_fwd(x, w, residual=x[:2]),
                 lambda: ts.norm_fwd(x, w, residual=x.float()), lambda: ts.norm_fwd(x.t(), w), lambda: ts.norm_fwd(x, w, eps=-1.0),
                 lambda: ts.norm_fwd(x, w, eps=math.nan), lambda: ts.norm_fwd(x, w, want_y=False), lambda: ts.norm_fwd(x.cpu(), w),
                 lambda: ts.norm_bwd(x, x[:2], w, rstd), lambda: ts.norm_bwd(x, x, w, rstd[:2]),
                 lambda: ts.norm_bwd(x, ts.act_pack(z(4, 32)), w, rstd), lambda: ts.norm_bwd(x, x, w, rstd, dh=x.float()),
                 lambda: ts.ts_norm_bwd(x, x, a8, w, rstd, None, x, w, torch.empty(9999, dtype=torch.uint8, device="cuda")),
                 lambda: ts.ts_norm_bwd(x, x, None, w, rstd, None, x, w, None),
                 lambda: ts.act_pack(x[0]), lambda: ts.act_pack(x.int()), lambda: ts.act_unpack(a8, torch.int8),
                 lambda: ts.act_unpack(ts.Act8(a8.codes, a8.scales[:2]), torch.float16)):
        with pytest.raises(ts.TsError) as e:
            call()
        assert e.value.status == ts.TS_ERR_INVALID_ARG
    c = dev(synth.random_coords(1, 4, 3, 1, 9))
    km = ts.build_kmap(c, ts.HashTable(c, 2.0), 3, 1, ts.TS_KMAP_PAIRS)
    with pytest.raises(ts.TsError) as e:
        ts.conv_wgrad_act8(km, a8, x.float())
    assert e.value.status == ts.TS_ERR_UNSUPPORTED
    for bad in (lambda: ts.conv_wgrad_act8(km, ts.act_pack(z(5, 16)), x), lambda: ts.conv_wgrad_act8(km, a8, x[:2]),
                lambda: ts.conv_wgrad_act8(ts.build_kmap(c, ts.HashTable(c, 2.0), 3, 1, 0), a8, x)):
        with pytest.raises(ts.TsError) as e:
            bad()
        assert e.value.status == ts.TS_ERR_INVALID_ARG


def test_empty(ts):
    x, w = torch.zeros(0, 16, dtype=torch.float16, device="cuda"), torch.ones(16, device="cuda")
    r = ts.norm_fwd(x, w, residual=x, y8=True, h8=True)
    dx, dw = ts.norm_bwd(x, r.h8, w, r.rstd)
    assert dx.shape == (0, 16) and (dw == 0).all()
    assert ts.act_unpack(ts.act_pack(x), torch.float16).shape == (0, 16)


def test_more_than_2_31_elements(ts):
    """The last rows of a matrix of 2^31 elements and more are those of the same rows by themselves."""
    n, c, last = (1 << 24) + 1000, 128, 1500
    x = torch.zeros((n, c), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(56)
    x[-last:] = torch.randn(last, c, generator=g, device="cuda").bfloat16()
    w = torch.rand(c, generator=g, device="cuda") + 0.5
    whole, part = (ts.norm_fwd(t, w, y8=True) for t in (x, x[-last:]))
    assert torch.equal(whole.y[-last:], part.y) and torch.equal(whole.rstd[-last:], part.rstd)
    assert torch.equal(whole.y8.codes[-last:], part.y8.codes) and torch.equal(whole.y8.scales[-last:], part.y8.scales)
    dx, dw = ts.norm_bwd(whole.y, x, w, whole.rstd)
    dx_part, _ = ts.norm_bwd(part.y, x[-last:], w, part.rstd)
    assert torch.equal(dx[-last:], dx_part)
    packed = ts.act_pack(x)
    values = ts.act_unpack(packed, torch.bfloat16)
    assert torch.equal(values[-last:], ts.act_unpack(ts.act_pack(x[-last:]), torch.bfloat16))
    assert not values[:-last].any()
