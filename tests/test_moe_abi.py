"""The expert layer's host logic on the CPU: argument checks (before any HIP
call) and workspace sizes.  No call here reaches a launch."""
import os

import pytest

from bit_quantized_matmul_q4_amd import _lib

FAKE = 1 << 20  # an aligned non-null address, never dereferenced
F16, BF16, F32, I8 = _lib.Q4_F16, _lib.Q4_BF16, _lib.Q4_F32, _lib.Q4_I8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from bit_quantized_matmul_q4_amd import build
        build.build_library()
    return _lib.load()


def route(lib, x=FAKE, xd=BF16, r=FAKE, rd=BF16, bias=None, ids=FAKE, w=FAKE, M=4, E=8, K=64, k=2, ws=FAKE,
          wb=1 << 30):
    return lib.q4_moe_route(x, xd, r, rd, bias, ids, w, M, E, K, k, 1, ws, wb, None)


def experts(lib, x=FAKE, xd=BF16, ids=FAKE, w=FAKE, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, y=FAKE, M=4, E=8, H=64,
            I=32, k=2, ws=FAKE, wb=1 << 30):
    return lib.q4_moe_experts(x, xd, ids, w, w13, s13, w2, s2, y, M, E, H, I, k, ws, wb, None)


def test_route_argument_checks(lib):
    for bad in ("x", "r", "ids", "w"):
        assert route(lib, **{bad: None}) == _lib.Q4_ERR_NULL
    for d in (F32, I8, 9):
        assert route(lib, xd=d, rd=d) == _lib.Q4_ERR_ENUM
    assert route(lib, xd=BF16, rd=F16) == _lib.Q4_ERR_ENUM
    for kw in ({"M": 0}, {"E": 0}, {"E": 1025}, {"k": 0}, {"k": 9}, {"K": 48}, {"K": 0}, {"K": (1 << 17) + 32},
               {"M": (1 << 20) + 1}):
        assert route(lib, **kw) == _lib.Q4_ERR_SHAPE, kw
    for kw in ({"x": FAKE + 8}, {"r": FAKE + 8}, {"bias": FAKE + 2}, {"ids": FAKE + 2}, {"w": FAKE + 1},
               {"ws": FAKE + 16}):
        assert route(lib, **kw) == _lib.Q4_ERR_ALIGN, kw
    need = lib.q4_moe_route_workspace_bytes(4, 8, 64)
    assert need > 0
    assert route(lib, wb=need - 1) == _lib.Q4_ERR_WORKSPACE
    assert route(lib, ws=None) == _lib.Q4_ERR_WORKSPACE
    assert route(lib, ws=None, wb=0) == _lib.Q4_ERR_WORKSPACE
    assert lib.q4_last_hip_error() == 0


def test_experts_argument_checks(lib):
    for bad in ("x", "ids", "w", "w13", "s13", "w2", "s2", "y"):
        assert experts(lib, **{bad: None}) == _lib.Q4_ERR_NULL
    for d in (F32, I8, 9):
        assert experts(lib, xd=d) == _lib.Q4_ERR_ENUM
    for kw in ({"M": 0}, {"E": 0}, {"E": 1025}, {"k": 0}, {"k": 1025}, {"H": 48}, {"I": 16}, {"H": 0},
               {"I": (1 << 17) + 32}, {"M": (1 << 20) + 1}):
        assert experts(lib, **kw) == _lib.Q4_ERR_SHAPE, kw
    for kw in ({"x": FAKE + 8}, {"ids": FAKE + 2}, {"w": FAKE + 2}, {"w13": FAKE + 8}, {"s13": FAKE + 4},
               {"w2": FAKE + 8}, {"s2": FAKE + 4}, {"y": FAKE + 2}, {"ws": FAKE + 16}):
        assert experts(lib, **kw) == _lib.Q4_ERR_ALIGN, kw
    need = lib.q4_moe_experts_workspace_bytes(4, 64, 32, 2)
    assert need > 0
    assert experts(lib, wb=need - 1) == _lib.Q4_ERR_WORKSPACE
    assert experts(lib, ws=None) == _lib.Q4_ERR_WORKSPACE
    assert lib.q4_last_hip_error() == 0


def test_sizes(lib):
    route, room, layer = (lib.q4_moe_route_workspace_bytes, lib.q4_moe_experts_workspace_bytes,
                          lib.q4_moe_layer_workspace_bytes)
    assert route(0, 8, 64) == 0 and route(3, 1025, 64) == 0 and route(3, 8, 40) == 0
    assert room(3, 64, 48, 2) == 0 and room(3, 48, 64, 2) == 0 and room(3, 64, 64, 0) == 0
    assert layer(3, 4, 64, 64, 5) == 0 and layer(3, 4, 64, 48, 2) == 0
    # past 1024 (row, expert) pairs the products run in pieces: no more room
    assert room(128, 96, 64, 8) == room(5000, 96, 64, 8)
    assert layer(3, 4, 64, 64, 2) >= route(3, 4, 64) + room(3, 64, 64, 2)


def test_layer_argument_checks(lib):
    def layer(x=FAKE, xd=BF16, r=FAKE, rd=BF16, bias=None, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, y=FAKE, M=4, E=8, H=64,
              I=32, k=2, ws=FAKE, wb=1 << 30):
        return lib.q4_moe_layer(x, xd, r, rd, bias, w13, s13, w2, s2, y, M, E, H, I, k, 1, ws, wb, None)

    for bad in ("x", "r", "w13", "s13", "w2", "s2", "y"):
        assert layer(**{bad: None}) == _lib.Q4_ERR_NULL
    assert layer(xd=F32) == _lib.Q4_ERR_ENUM
    assert layer(rd=F16) == _lib.Q4_ERR_ENUM
    for kw in ({"M": 0}, {"E": 0}, {"E": 1025}, {"k": 0}, {"k": 9}, {"H": 48}, {"I": 16}, {"I": (1 << 17) + 32}):
        assert layer(**kw) == _lib.Q4_ERR_SHAPE, kw
    for kw in ({"x": FAKE + 8}, {"r": FAKE + 8}, {"bias": FAKE + 2}, {"w13": FAKE + 8}, {"s13": FAKE + 4},
               {"w2": FAKE + 8}, {"s2": FAKE + 4}, {"y": FAKE + 2}, {"ws": FAKE + 16}):
        assert layer(**kw) == _lib.Q4_ERR_ALIGN, kw
    assert layer(wb=lib.q4_moe_layer_workspace_bytes(4, 8, 64, 32, 2) - 1) == _lib.Q4_ERR_WORKSPACE
    assert layer(ws=None) == _lib.Q4_ERR_WORKSPACE
    assert lib.q4_last_hip_error() == 0
