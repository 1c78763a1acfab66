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


def run(code, **kw):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                          text=True, timeout=300, **kw)


def test_import_without_torch_gpu_support(lib):
    """A torch built without GPU support: the import and the host-side calls work."""
    p = run("import torch\n"
            "for name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, name):\n"
            "        delattr(torch._C, name)\n"
            "import bit_quantized_matmul_q4_amd as q4\n"
            "assert q4.packed_sizes(16, 32) == (1024, 128) and q4.segments(3584) == 16\n"
            "try:\n"
            "    q4.quantize_int8(torch.zeros(4, 64))\n"
            "except ValueError as e:\n"
            "    print('refused:', e)\n")
    assert p.returncode == 0 and "refused: w must be a GPU tensor" in p.stdout, p.stdout


def stub(tmp_path, name, body):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, out = tmp_path / (name + ".c"), tmp_path / (name + ".so")
    src.write_text(body)
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", str(out)], check=True)
    return str(out)


def test_other_builds_of_the_library_are_named(tmp_path, monkeypatch):
    """A library without some of the functions, of another ABI version, or of another kind: an ImportError that says so."""
    older = stub(tmp_path, "older", "int q4_abi_version(void) { return %d; } int q4_linear(void) { return 0; }"
                 % _lib.ABI_VERSION)
    other = stub(tmp_path, "other", "int q4_abi_version(void) { return %d; }" % (_lib.ABI_VERSION + 1))
    alien = stub(tmp_path, "alien", "int f(void) { return 0; }")
    for path, text in ((older, "q4_int8_linear"), (other, "ABI %d" % (_lib.ABI_VERSION + 1)), (alien, "q4_abi_version")):
        with pytest.raises(ImportError, match=text):
            _lib.load(path)
        monkeypatch.setattr(_lib, "LIB_PATH", path)
        monkeypatch.setattr(_lib, "_lib", None)
        with pytest.raises(ImportError, match=text):
            _lib.load()


def test_status_texts_hold_for_every_call(lib):
    """Shapes and alignments that only the 8-bit product or the expert layer check are in the texts."""
    shape, align = (lib.q4_strerror(s).decode() for s in (_lib.Q4_ERR_SHAPE, _lib.Q4_ERR_ALIGN))
    assert "topk" in shape and "experts" in shape
    assert "router" in align and "ids" in align and "16-bit y" in align
