"""The binding on the CPU: what it says when a call or the library is not what it needs."""
import os
import shutil
import subprocess
import sys

import pytest

from bit_quantized_matmul_q4_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from bit_quantized_matmul_q4_amd import build
        build.build_library()
    return _lib.load()


def test_workspace_status_text(lib):
    """The status of a workspace that is absent, NULL with a size, or too small: its text holds for all three."""
    text = lib.q4_strerror(_lib.Q4_ERR_WORKSPACE).decode()
    assert "NULL" in text and "too small" in text and "needs" in text
