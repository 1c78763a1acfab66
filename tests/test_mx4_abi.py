"""The microscaled 4-bit form's host logic on the CPU: argument checks (before
any HIP call), packed and workspace sizes, and what the binding refuses.  No
call here reaches a launch."""
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


def linear(lib, x=FAKE, xd=BF16, xs=None, w=FAKE, ws=FAKE, y=FAKE, yd=F32, M=128, N=64, K=64, work=FAKE, wb=1 << 40):
    return lib.q4_mx4_linear(x, xd, xs, w, ws, y, yd, M, N, K, work, wb, None)


def test_linear_argument_checks(lib):
    for bad in ("x", "w", "ws", "y"):
        assert linear(lib, **{bad: None}) == _lib.Q4_ERR_NULL
    assert linear(lib, xd=MX4, xs=None) == _lib.Q4_ERR_NULL
    for d in (F32, I8, 7, -1):
        assert linear(lib, xd=d) == _lib.Q4_ERR_ENUM
    for d in (I8, MX4, -1, 9):
        assert linear(lib, yd=d) == _lib.Q4_ERR_ENUM
    for M, N, K in ((0, 64, 64), (-1, 64, 64), (4, 0, 64), (4, 64, 0), (4, 64, 48), (4, 64, 131104),
                    ((1 << 24) + 1, 1, 64), (1, (1 << 24) + 1, 64), (1 << 20, 1 << 20, 64)):
        assert linear(lib, M=M, N=N, K=K) == _lib.Q4_ERR_SHAPE, (M, N, K)
    assert linear(lib, x=FAKE + 8) == _lib.Q4_ERR_ALIGN
    assert linear(lib, w=FAKE + 8) == _lib.Q4_ERR_ALIGN
    assert linear(lib, ws=FAKE + 2) == _lib.Q4_ERR_ALIGN
    assert linear(lib, y=FAKE + 2) == _lib.Q4_ERR_ALIGN
    assert linear(lib, y=FAKE + 1, yd=BF16) == _lib.Q4_ERR_ALIGN
    assert linear(lib, xd=MX4, xs=FAKE + 2) == _lib.Q4_ERR_ALIGN
    assert linear(lib, work=FAKE + 16) == _lib.Q4_ERR_ALIGN
    assert linear(lib, work=None, wb=64) == _lib.Q4_ERR_WORKSPACE
    need = lib.q4_mx4_workspace_bytes(128, 64, 64, BF16)
    assert need > 0
    assert linear(lib, wb=need - 1) == _lib.Q4_ERR_WORKSPACE
    assert linear(lib, work=None, wb=0) == _lib.Q4_ERR_WORKSPACE
    assert lib.q4_last_hip_error() == 0


def test_quantize_and_pack_argument_checks(lib):
    for f, scale in ((lib.q4_mx4_quantize, 1), (lib.q4_mx4_quantize_pack, 4)):
        assert f(None, F32, FAKE, FAKE, 4, 64, None) == _lib.Q4_ERR_NULL
        assert f(FAKE, F32, None, FAKE, 4, 64, None) == _lib.Q4_ERR_NULL
        assert f(FAKE, F32, FAKE, None, 4, 64, None) == _lib.Q4_ERR_NULL
        assert f(FAKE, MX4, FAKE, FAKE, 4, 64, None) == _lib.Q4_ERR_ENUM
        assert f(FAKE, I8, FAKE, FAKE, 4, 64, None) == _lib.Q4_ERR_ENUM
        assert f(FAKE, F32, FAKE, FAKE, 0, 64, None) == _lib.Q4_ERR_SHAPE
        assert f(FAKE, F32, FAKE, FAKE, 4, 40, None) == _lib.Q4_ERR_SHAPE
        assert f(FAKE + 4, F32, FAKE, FAKE, 4, 64, None) == _lib.Q4_ERR_ALIGN
        assert f(FAKE, F32, FAKE + 8, FAKE, 4, 64, None) == _lib.Q4_ERR_ALIGN
        if scale > 1:
            assert f(FAKE, F32, FAKE, FAKE + 2, 4, 64, None) == _lib.Q4_ERR_ALIGN
    p = lib.q4_mx4_pack
    for i in range(4):
        assert p(*[None if j == i else FAKE for j in range(4)], 4, 64, None) == _lib.Q4_ERR_NULL
    assert p(FAKE, FAKE, FAKE, FAKE, 4, 16, None) == _lib.Q4_ERR_SHAPE
    assert p(FAKE + 8, FAKE, FAKE, FAKE, 4, 64, None) == _lib.Q4_ERR_ALIGN
    assert p(FAKE, FAKE, FAKE + 8, FAKE, 4, 64, None) == _lib.Q4_ERR_ALIGN
    assert p(FAKE, FAKE, FAKE, FAKE + 2, 4, 64, None) == _lib.Q4_ERR_ALIGN
    d = lib.q4_mx4_dequantize
    assert d(None, FAKE, FAKE, F32, 4, 64, None) == _lib.Q4_ERR_NULL
    assert d(FAKE, None, FAKE, F32, 4, 64, None) == _lib.Q4_ERR_NULL
    assert d(FAKE, FAKE, None, F32, 4, 64, None) == _lib.Q4_ERR_NULL
    assert d(FAKE, FAKE, FAKE, MX4, 4, 64, None) == _lib.Q4_ERR_ENUM
    assert d(FAKE, FAKE, FAKE, F32, 4, 33, None) == _lib.Q4_ERR_SHAPE
    assert d(FAKE + 8, FAKE, FAKE, F32, 4, 64, None) == _lib.Q4_ERR_ALIGN
    assert d(FAKE, FAKE + 1, FAKE, F32, 4, 64, None) == _lib.Q4_ERR_ALIGN
    assert d(FAKE, FAKE, FAKE + 4, F32, 4, 64, None) == _lib.Q4_ERR_ALIGN
    assert lib.q4_last_hip_error() == 0


def test_sizes(lib):
    for R, K in ((1, 32), (16, 128), (17, 160), (4863, 896), (3584, 18944), (1 << 24, 1 << 17)):
        assert lib.q4_mx4_code_bytes(R, K) == -(-R // 16) * -(-K // 128) * 1024
        assert lib.q4_mx4_scale_bytes(R, K) == -(-R // 16) * -(-K // 512) * 256
    for R, K in ((0, 64), (4, 48), (4, 131104), ((1 << 24) + 1, 32)):
        assert lib.q4_mx4_code_bytes(R, K) == 0 and lib.q4_mx4_scale_bytes(R, K) == 0
    assert lib.q4_mx4_workspace_bytes(4, 64, 48, BF16) == 0
    assert lib.q4_mx4_workspace_bytes(4, 64, 64, F32) == 0
    for M, N, K in ((1, 64, 64), (20, 512, 3584), (124, 3584, 18944), (333, 4863, 896), (4096, 18944, 3584)):
        dense, packed = (lib.q4_mx4_workspace_bytes(M, N, K, d) for d in (BF16, MX4))
        assert dense == lib.q4_mx4_workspace_bytes(M, N, K, F16)
        assert packed == 0  # packed rows need no room for codes


def test_binding_refuses():
    """Tensors off the GPU and objects of other kinds, before the library is asked."""
    x = torch.zeros(4, 64)
    for f in (q4.quantize_mx4, q4.quantize_pack_mx4):
        with pytest.raises(ValueError, match="GPU tensor"):
            f(x)
    with pytest.raises(ValueError, match="GPU tensor"):
        q4.pack_mx4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(TypeError, match="Mx4Matrix"):
        q4.dequantize_mx4(x)
    with pytest.raises(ValueError, match="GPU tensor"):
        q4.linear_mx4(x.bfloat16(), None)
