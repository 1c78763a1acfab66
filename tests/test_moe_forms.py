"""Which launches the expert layer takes (host rule, on the CPU): the choice
within gate/up where that was measured faster, a launch of its own where not,
and GPU test shapes on both sides."""
import ctypes
import os

import pytest

from bit_quantized_matmul_q4_amd import build
from tests.moe_forms import BY_ROWS, FUSED, SEPARATE


@pytest.fixture(scope="module")
def form():
    if not os.path.exists(build.PROBE_LIB):
        build.build_probe()
    f = ctypes.CDLL(build.PROBE_LIB).q4probe_moe_form
    f.argtypes = [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int)]

    def of(M, E, H):
        r = (ctypes.c_int * 2)()
        f(M, E, H, r)
        return bool(r[0]), bool(r[1])

    return of


def test_choice_where_it_was_measured_faster(form):
    for H in (896, 2048, 3584):
        for M, E in ((1, 8), (1, 64), (1, 128), (2, 64), (4, 16), (16, 8)):
            assert form(M, E, H) == (True, False), (M, E, H)
        for M, E in ((64, 8), (64, 16), (128, 2), (256, 8), (250, 4), (1000, 4), (1000, 2), (16, 32), (8, 128)):
            assert not form(M, E, H)[0], (M, E, H)
    assert not form(4, 64, 3584)[0] and not form(3, 64, 3584)[0]


def test_gpu_shapes_take_their_form(form):
    for M, E, H, I, topk in FUSED:
        assert form(M, E, H) == (True, False), (M, E, H)
    for M, E, H, I, topk in SEPARATE:
        assert form(M, E, H) == (False, False), (M, E, H)
    for M, E, H, I, topk in BY_ROWS:
        assert form(M, E, H) == (False, True), (M, E, H)


def test_logits_where_they_were_measured_faster(form):
    for M, E, H in ((4096, 64, 2048), (2048, 128, 3584), (6000, 64, 3584), (16384, 8, 3584)):
        assert not form(M, E, H)[1], (M, E, H)
    for M, E, H in ((16384, 128, 2048), (2048, 512, 1024), (65536, 8, 3584), (1030, 512, 320), (32760, 3, 288),
                    (2049, 250, 832)):
        assert form(M, E, H)[1], (M, E, H)
