"""17 to 32 rows by many columns in the microscaled 4-bit product: which of the
32-row tiles they take (host rule, on the CPU), and that the bits do not change
at the border (GPU)."""
import os

import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from bit_quantized_matmul_q4_amd import build
from tests import gpu_util as gu
from tests.mx4_forms import form_of


@pytest.fixture(scope="module", autouse=True)
def probe():
    if not os.path.exists(build.PROBE_LIB):
        build.build_probe()


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("M", [17, 20, 32])
@pytest.mark.parametrize("K", [32, 896, 3584, 8192])
def test_three_workgroups_a_compute_unit(dense, M, K):
    """32 x 32 while that is at most three workgroups for each of 256 compute units, then 32 x 64."""
    for N in (16416, 18944, 24575, 24576):
        assert form_of(dense, M, N, K) == "32x32", N
    for N in (24577, 25600, 28672, 32736, 32768, 100000):
        assert form_of(dense, M, N, K) == "32x64", N


@pytest.mark.gpu
@pytest.mark.parametrize("N", [24576, 24577, 25600, 28673, 32736])
@pytest.mark.parametrize("M,K", [(17, 96), (32, 1184), (20, 2400), (31, 3584)])
def test_bits_at_the_border(M, N, K):
    gu.require_gpu()
    gu.note("linear_mx4 M=%d N=%d K=%d: %s" % (M, N, K, form_of(True, M, N, K)))
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    x = torch.randn(M, K, device=gu.DEV, generator=g).bfloat16()
    w = q4.quantize_mx4(torch.randn(N, K, device=gu.DEV, generator=g))
    packed = q4.pack_mx4(*w)
    for dtype in (torch.float32, torch.bfloat16):
        y = q4.linear_mx4(x, packed, out_dtype=dtype)
        assert torch.equal(q4.linear_mx4(q4.quantize_pack_mx4(x), packed, out_dtype=dtype), y)
        few = q4.linear_mx4(x[:16].contiguous(), packed, out_dtype=dtype)  # (a kernel for few rows)
        assert torch.equal(few, y[:16])
        last = q4.pack_mx4(*(t[-96:].contiguous() for t in w))  # (a smaller tile)
        assert torch.equal(q4.linear_mx4(x, last, out_dtype=dtype), y[:, -96:].contiguous())
