"""Every way the library does the products grouped by expert, against the fp64 implementation and bounds of
test_gpu_group.py."""
import pytest

from group_forms import FORMS
from test_gpu_group import DT, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("case", FORMS, ids=lambda c: c[0])
def test_form(ts, case, dt):
    _, lens, cin, cout, what = case
    Case(ts, dt, lens, cin, cout).check(what)
    Case(ts, dt, lens, cin, cout, gather=False).check(what)
