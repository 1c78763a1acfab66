"""Which kernel of the 8-bit product a shape takes (host rule, on the CPU): the
shapes that the GPU tests run reach every one."""
import os

import pytest

from bit_quantized_matmul_q4_amd import build
from tests.int8_forms import FORMS, form_of


@pytest.fixture(scope="module", autouse=True)
def probe():
    if not os.path.exists(build.PROBE_LIB):
        build.build_probe()


@pytest.mark.parametrize("form", list(FORMS))
def test_shapes_take_their_form(form):
    for M, N, K in FORMS[form]:
        assert form_of(True, M, N, K)[0] == form, (M, N, K)


def test_every_form_is_named():
    """No shape of a coarse grid takes a form that the tests do not list."""
    seen = set()
    for dense in (True, False):
        for M in (1, 2, 3, 4, 5, 16, 17, 64, 65, 128, 200, 333, 700, 1024, 2048, 4096, 8192, 30000, 70000):
            for N in (1, 16, 60, 200, 896, 2048, 3584, 8192, 8200, 18944, 152064):
                for K in (32, 96, 896, 3584, 5120, 10240, 18944, 131040):
                    seen.add(form_of(dense, M, N, K)[0])
    assert seen == set(FORMS)


def test_both_quantizers_are_reached():
    assert {form_of(True, *s)[1] for shapes in FORMS.values() for s in shapes} == {1, 4}
