"""How attention calls are cut up (no GPU needed): the rules of csrc/attn_plan.h,
compiled by themselves, give each call of attn_forms.py the plan it is there
for, so that a change of the rules cannot leave a form of the kernels without
its parity test unnoticed."""
import os
import shutil
import subprocess

import pytest

from attn_forms import FORMS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_voxelised_point_amd", "csrc")
GXX = shutil.which("g++")

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "attn_plan.h"
int main() {
  long long nq, nk, sets;
  int hq, hk, d;
  while (std::scanf("%lld %lld %lld %d %d %d", &nq, &nk, &sets, &hq, &hk, &d) == 6) {
    for (const ts::AttnPlan& p : {ts::plan_fwd(nq, nk, sets, hq, hk, d), ts::plan_dq(nq, nk, sets, hq, hk, d),
                                  ts::plan_dkv(nq, nk, sets, hq, hk, d)})
      std::printf("%d %d %d %d %d ", p.bm, p.nc, p.heads, p.splits, p.share_keys);
    std::printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if GXX is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run([GXX, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def ask(*calls):
        lines = "".join(" ".join(map(str, c)) + "\n" for c in calls)
        out = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, check=True, timeout=60).stdout
        rows = [list(map(int, line.split())) for line in out.splitlines()]
        return [(r[:5], r[5:10], r[10:]) for r in rows]
    return ask


@pytest.mark.parametrize("form", FORMS, ids=[f[0] for f in FORMS])
def test_forms_have_their_plans(plans, form):
    name, _, lq, lk, hq, hk, d, _, _, keys, rows = form
    lk = lq if lk is None else lk
    fwd, dq = keys if isinstance(keys[0], tuple) else (keys, keys)
    got_plans, = plans((sum(lq), sum(lk), len(lq), hq, hk, d))
    for got, (nc, heads, splits, share) in zip(got_plans, (fwd, dq, rows)):
        assert got[1:] == [nc, heads, splits, int(share)], name
        assert got[0] == (16 if share else 64 * nc)


def test_plans_hold_over_the_range(plans):
    """Whatever the sizes: forms that exist, splits that the join takes, no more blocks than a launch may have."""
    calls = [(nq, nk, sets, hk * grp, hk, d)
             for nq in (0, 1, 17, 1000, 100_000, (1 << 31) - 1) for nk in (0, 1, 300, 100_000, (1 << 31) - 1)
             for sets in (0, 1, 13, 5000, 1 << 20) for hk, grp in ((1, 1), (4, 2), (3, 1)) for d in (1, 32, 33, 64, 128)
             if nq * hk * grp < 1 << 31 and nk * hk < 1 << 31]
    for call, (fwd, dq, rows) in zip(calls, plans(*calls)):
        for bm, nc, heads, splits, share in (fwd, dq, rows):
            assert nc in (1, 2) and heads in (1, 2, 4) and heads <= call[4] and 1 <= splits <= 512, call
            assert bm == (16 if share else 64 * nc) and (nc == 1 or not share), call
            assert call[5] <= 64 or (nc == 1 and not share), call
            assert heads == 1 or (nc == 1 and not share and call[5] <= 64), call
        assert not rows[4], call
