"""q4_block_norm's argument checks on the CPU (before any HIP call), and what
the binding refuses.  No call here reaches a launch."""
import ctypes
import os

import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from bit_quantized_matmul_q4_amd import _lib

FAKE = 1 << 20  # an aligned non-null address, never dereferenced
F16, BF16, F32, I8, MX4 = _lib.Q4_F16, _lib.Q4_BF16, _lib.Q4_F32, _lib.Q4_I8, _lib.Q4_MX4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from bit_quantized_matmul_q4_amd import build
        build.build_library()
    return _lib.load()


def side(weight=FAKE, bias=None, kind=_lib.Q4_NORM_RMS, dtype=BF16, eps=1e-6):
    return _lib.NormSide(weight, bias, kind, dtype, eps)


def norm(lib, y=FAKE, yd=F32, post=None, gate=None, gd=BF16, form=0, scale=1.0, res=FAKE, r=FAKE, rd=BF16, pre=None,
         h=FAKE, hd=BF16, hs=None, M=4, H=64):
    return lib.q4_block_norm(y, yd, post, gate, gd, form, scale, res, r, rd, pre, h, hd, hs, M, H, None)


def test_null(lib):
    assert norm(lib, y=None) == _lib.Q4_ERR_NULL
    assert norm(lib, r=None, h=None) == _lib.Q4_ERR_NULL
    assert norm(lib, hd=MX4, hs=None) == _lib.Q4_ERR_NULL
    for form in (1, 2, 3):
        assert norm(lib, form=form) == _lib.Q4_ERR_NULL


def test_enum(lib):
    for d in (I8, MX4, -1, 9):
        assert norm(lib, yd=d) == _lib.Q4_ERR_ENUM
        assert norm(lib, rd=d) == _lib.Q4_ERR_ENUM
        assert norm(lib, rd=d, res=None) == _lib.Q4_ERR_ENUM
        assert norm(lib, rd=d, r=None) == _lib.Q4_ERR_ENUM
        assert norm(lib, gd=d, gate=FAKE, form=1) == _lib.Q4_ERR_ENUM
        assert norm(lib, pre=side(dtype=d)) == _lib.Q4_ERR_ENUM
        assert norm(lib, post=side(dtype=d)) == _lib.Q4_ERR_ENUM
    for d in (I8, -1, 9):
        assert norm(lib, hd=d) == _lib.Q4_ERR_ENUM
    for form in (-1, 4):
        assert norm(lib, gate=FAKE, form=form) == _lib.Q4_ERR_ENUM
    for kind in (-1, 3):
        assert norm(lib, pre=side(kind=kind)) == _lib.Q4_ERR_ENUM
        assert norm(lib, post=side(kind=kind)) == _lib.Q4_ERR_ENUM


def test_shape(lib):
    for M, H in ((0, 64), (-1, 64), (4, 0), (4, -8), ((1 << 20) + 1, 64), (4, 32769)):
        assert norm(lib, M=M, H=H) == _lib.Q4_ERR_SHAPE, (M, H)
    assert norm(lib, hd=MX4, hs=FAKE, H=40) == _lib.Q4_ERR_SHAPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(lib, pre=side(eps=eps)) == _lib.Q4_ERR_SHAPE
        assert norm(lib, post=side(eps=eps)) == _lib.Q4_ERR_SHAPE


def test_align(lib):
    assert norm(lib, y=FAKE + 2) == _lib.Q4_ERR_ALIGN
    assert norm(lib, yd=BF16, y=FAKE + 1) == _lib.Q4_ERR_ALIGN
    assert norm(lib, res=FAKE + 1) == _lib.Q4_ERR_ALIGN
    assert norm(lib, r=FAKE + 1) == _lib.Q4_ERR_ALIGN
    assert norm(lib, rd=F32, r=FAKE + 2) == _lib.Q4_ERR_ALIGN
    assert norm(lib, h=FAKE + 1) == _lib.Q4_ERR_ALIGN
    assert norm(lib, hd=F32, h=FAKE + 2) == _lib.Q4_ERR_ALIGN
    assert norm(lib, hd=MX4, h=FAKE + 8, hs=FAKE) == _lib.Q4_ERR_ALIGN
    assert norm(lib, hd=MX4, hs=FAKE + 2) == _lib.Q4_ERR_ALIGN
    assert norm(lib, gate=FAKE + 1, form=1) == _lib.Q4_ERR_ALIGN
    assert norm(lib, pre=side(weight=FAKE + 1)) == _lib.Q4_ERR_ALIGN
    assert norm(lib, post=side(bias=FAKE + 2, dtype=F32)) == _lib.Q4_ERR_ALIGN
    assert lib.q4_last_hip_error() == 0


def test_struct_matches_the_header():
    assert ctypes.sizeof(_lib.NormSide) == 32


def test_binding_refuses():
    with pytest.raises(ValueError, match="GPU tensor"):
        q4.block_norm(torch.zeros(4, 64))
    with pytest.raises(TypeError, match="torch.Tensor"):
        q4.block_norm([1.0])
