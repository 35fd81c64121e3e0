"""How far attention's results are from 64 bits, against what rounding the exact
results to their type would cost (both as norms over the whole tensor).

One 16-bit rounding of a product's operand adds an independent error of the
same size: sqrt(2) of the last rounding where many of them average, so 1.5
bounds it.  Operands of two parts, and a delta without a rounding, leave 2^-8
of that; scores, sums and exponentials are good to about 2^-18 of a result
against 2^-13 that rounding to fp16 costs: 1.1."""
import pytest
import torch

from test_gpu_attn import build, ref_of

pytestmark = pytest.mark.gpu

FEW = [
    ("one_query", [1], [700], 8, 2, 64, 0.0, True),
    ("one_query_few_keys", [1], [7], 4, 4, 40, 0.0, False),
    ("two_rows_sharp", [1, 1], [141, 90], 1, 1, 16, 0.0, True),
    ("four_queries", [4, 2], [141, 30], 3, 3, 64, 0.0, True),
    ("queries_128", [3, 12], [150, 500], 2, 1, 128, 0.0, True),
    ("capped", [5, 9, 0], [176, 400, 3], 6, 3, 24, 6.0, True),
    ("many_keys", [2], [9000], 4, 2, 32, 0.0, False),
    ("small_windows", [39, 20, 64, 65, 1, 90], None, 2, 2, 16, 0.0, True),
]
MANY = [
    ("narrow_windows", [70, 127, 33, 180, 65, 12, 90] * 6, None, 4, 4, 16, 0.0, True),
    ("narrow_shared", [176, 150], None, 16, 4, 16, 0.0, False),
    ("narrow_24", [114, 80, 100], None, 8, 4, 24, 0.0, True),
    ("narrow_split", [500], [2100], 6, 3, 16, 0.0, True),
    ("narrow_two_columns", [1024], None, 32, 32, 24, 0.0, True),
    ("narrow_capped", [400, 300], None, 4, 4, 16, 8.0, True),
    ("windows_32", [127, 90, 200, 40] * 4, None, 4, 4, 32, 0.0, True),
    ("scene_64", [900], None, 4, 2, 64, 0.0, True),
    ("scene_128", [600], None, 4, 4, 128, 7.0, False),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case,few", [(c, True) for c in FEW] + [(c, False) for c in MANY], ids=[c[0] for c in FEW + MANY])
def test_errors_against_the_last_rounding(ts, case, few, dt):
    name, lq, lk, hq, hk, d, cap, bias = case
    assert (sum(lq) * hq <= 2048) == few
    dtype, q, k, v, dout, qs, ks, opt = build((name, dt, lq, lk, hq, hk, d, cap, bias, 3))
    out, lse = ts.attn_fwd(q, k, v, qs, ks, **opt)
    got = dict(zip(("dq", "dk", "dv"), ts.attn_bwd(dout, q, k, v, out, lse, qs, ks, **opt)), out=out)
    ref, _ = ref_of(dtype, q, k, v, qs, ks, opt, dout)
    for n, t in got.items():
        exact = ref[n]
        last = float((exact.to(dtype).double() - exact).norm())
        bar = 1.1 if few or (n == "dq" and d < 32 and cap == 0) else 1.5
        err = float((t.double().cpu() - exact).norm())
        assert err <= bar * last, f"{name} {n}: {err / last:.3f} times the last rounding's error"
