"""Which kernel of the microscaled 4-bit product a shape takes (host rule, on
the CPU): the shapes that the GPU tests run reach every one."""
import os

import pytest

from bit_quantized_matmul_q4_amd import build
from tests.mx4_forms import FORMS, form_of


@pytest.fixture(scope="module", autouse=True)
def probe():
    if not os.path.exists(build.PROBE_LIB):
        build.build_probe()


@pytest.mark.parametrize("form", list(FORMS))
def test_shapes_take_their_form(form):
    for M, N, K in FORMS[form]:
        assert form_of(True, M, N, K) == form, (M, N, K)
        packed = form_of(False, M, N, K)  # (the relay loads packed rows beside W, and is faster up to more columns)
        assert packed == form.replace("/q", "") or (form, packed) == ("wide/q", "relay"), (M, N, K)


def test_every_form_is_named():
    """No shape of a coarse grid takes a form that the tests do not list."""
    seen = set()
    for dense in (True, False):
        for M in (1, 2, 3, 4, 5, 16, 17, 32, 33, 64, 65, 128, 200, 333, 700, 1024, 2048, 4096, 8192, 30000, 70000):
            for N in (1, 16, 60, 200, 896, 2048, 3584, 8192, 8200, 18944, 152064):
                for K in (32, 96, 896, 3584, 5120, 10240, 18944, 131072):
                    seen.add(form_of(dense, M, N, K))
    assert seen == set(FORMS)


def test_groups_and_last_steps_are_covered():
    """Every tile kernel meets one group, odd and even numbers of groups, and one to four steps in the last."""
    for form, shapes in FORMS.items():
        if "x" not in form:
            continue
        groups = {-(-K // 512) for _, _, K in shapes}
        assert 1 in groups and {g % 2 for g in groups} == {0, 1}, (form, groups)
        last = {(-(-K // 128) - 1) % 4 + 1 for _, _, K in shapes}
        assert last == {1, 2, 3, 4}, (form, last)


def test_last_steps_after_several_groups_are_covered():
    """And one to four steps in the last group where whole groups come before it, in odd and even numbers."""
    for form, shapes in FORMS.items():
        if "x" not in form:
            continue
        met = {(min(-(-K // 512), 4), (-(-K // 128) - 1) % 4 + 1) for _, _, K in shapes if K > 512}
        assert {last for _, last in met} == {1, 2, 3, 4}, (form, met)
        assert {last for groups, last in met if groups >= 3} == {1, 2, 3, 4}, (form, met)

