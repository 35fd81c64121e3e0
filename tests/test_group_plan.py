"""How the products grouped by expert are done (no GPU needed): the rules of csrc/group_plan.h, compiled by
themselves, give each call of group_forms.py the form it is there for, and no form is without one, so that no
instance of the kernels is without its parity test."""
import os
import shutil
import subprocess

import pytest

from group_forms import FORMS, ROWWISE, FEW16, FEW16_LOOSE, FEW32, FEW32_LOOSE, LARGE, LOOSE, MIDDLE, SMALL

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_voxelised_point_amd", "csrc")
GXX = shutil.which("g++")

PROGRAM = r"""
#include <cstdio>
#include "group_plan.h"
int main() {
  int op, glu, aligned, e, cin, cout;
  long long rows, looked_up;
  while (std::scanf("%d %d %d %lld %d %d %d %lld", &op, &glu, &aligned, &rows, &e, &cin, &cout, &looked_up) == 8) {
    const ts::GroupForm f = ts::group_form(static_cast<ts::GroupOp>(op), glu, aligned, rows, e, cin, cout, looked_up);
    const int chunk = ts::group_chunk(rows, e, cin, cout);
    std::printf("%d %d %d %d %d %lld\n", f.few, f.rows, f.cols, f.whole, chunk, static_cast<long long>(ts::group_chunks(rows, e, chunk)));
  }
}
"""
OPS = {"fwd": (0, 0), "glu": (0, 1), "dgrad": (1, 0), "glu_dgrad": (1, 1), "wgrad": (2, 0)}


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    if GXX is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run([GXX, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def ask(*calls):
        """Of (product, aligned, rows, groups, cin, cout, rows looked up): the form, rows of a run of dW, and runs at most."""
        lines = "".join(" ".join(map(str, (*OPS[c[0]], *c[1:]))) + "\n" for c in calls)
        out = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, check=True, timeout=60).stdout
        rows = [list(map(int, line.split())) for line in out.splitlines()]
        return [((bool(r[0]), r[1], r[2], bool(r[3])), r[4], r[5]) for r in rows]
    return ask


@pytest.mark.parametrize("case", FORMS, ids=lambda c: c[0])
def test_calls_have_their_forms(forms, case):
    _, lens, cin, cout, what = case
    for looked_up in (0, sum(lens) // 2):
        for op, want in what.items():
            assert forms((op, 1, sum(lens), len(lens), cin, cout, looked_up))[0][0] == want, op


def test_no_form_is_missing():
    got = {(op, form) for *_, what in FORMS for op, form in what.items()}
    assert got == {(op, form) for op in ROWWISE for form in (FEW16, FEW16_LOOSE, FEW32, FEW32_LOOSE, LOOSE, SMALL, MIDDLE, LARGE)} | \
        {("wgrad", form) for form in (LOOSE, SMALL, LARGE)}


def test_forms_hold_over_the_range(forms):
    """Whatever the sizes: a form that is built, whole accesses only where rows allow them, and runs that 32 bits number."""
    built = {form for *_, what in FORMS for form in what.values()}
    calls = [(op, aligned, rows, e, cin, cout, looked_up) for op in OPS for aligned in (0, 1)
             for rows in (1, 2, 33, 1000, 70_000, 20_000_000, (1 << 31) - 1) for e in (1, 2, 64, 4096)
             for cin, cout in ((1, 1), (8, 65536), (65536, 8), (77, 133), (256, 256), (1024, 4096), (65535, 65536)) for looked_up in (0, rows)]
    for call, (form, chunk, runs) in zip(calls, forms(*calls)):
        op, aligned, rows, e, cin, cout, looked_up = call
        assert form in built and (op != "wgrad" or not form[0]), call
        assert not form[3] or (aligned and cin % 8 == 0 and cout % 8 == 0), call
        assert form[0] or not form[3] or looked_up * cin < (1 << 31) - 8, call
        assert chunk % 64 == 0 and 256 <= chunk <= 1 << 28 and runs == rows // chunk + e, call
