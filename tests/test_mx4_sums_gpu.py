"""What the sums of the microscaled 4-bit product lose beside values of very
different size, on the GPU, in every kernel.

The matrix instruction's precision is known by measurement.  It adds the blocks
of 32 products of a step one after another: a block's products are added exactly
and the sum is then within 2^-23 of its own size, unless the power of two of every
product in the block is 2^-28 of the sum's or less, where the block is lost: 32
products below 2.25 2^-28 of the sum, 4.5 2^-24 of it.  So a sum over B blocks
is within 4.5 B 2^-24 of the sum of the magnitudes, and what rounding to the output's
type adds.  Values of like size stay exact."""
from fractions import Fraction

import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from tests import gpu_util as gu
from tests import mx4_ref as ref
from tests.mx4_forms import form_of

pytestmark = pytest.mark.gpu

SHAPES = [(1, 40), (5, 33), (16, 40), (16, 20000), (17, 40), (40, 4000), (70, 2100), (100, 4097), (200, 8200), (1000, 4100)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()
    yield
    torch.cuda.empty_cache()


def pack(codes, scales):
    return q4.pack_mx4(ref.nibbles(codes).to(gu.DEV), scales.to(gu.DEV))


def within(y, x, w):
    """y against the 64-bit product of two packed matrices."""
    x, w = (q4.dequantize_mx4(m).double() for m in (x, w))
    want, mag = x @ w.T.contiguous(), x.abs() @ w.abs().T.contiguous()
    bound = 4.5 * (x.shape[1] // 32) * 2.0 ** -24 * mag
    f = torch.finfo(y.dtype)
    off = (y.double() - want).abs() - bound - f.eps / 2 * (want.abs() + bound) - f.smallest_normal * f.eps
    assert (off <= 0).all(), "%g over" % off.max()


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("K", [64, 128, 480, 2080])
@pytest.mark.parametrize("span", [8, 20, 27, 34, 50])
def test_blocks_of_very_different_size(M, N, K, span):
    """Codes of one sign, so that nothing cancels what is lost; scales over `span` powers of two."""
    gu.note("linear_mx4 sums M=%d N=%d K=%d span %d: %s" % (M, N, K, span, form_of(False, M, N, K)))
    g = torch.Generator()
    g.manual_seed(M + N + K + span)
    for lowest in (1, 6):
        x, w = (pack(torch.randint(lowest, 8, (R, K), generator=g, dtype=torch.uint8),
                     torch.randint(127 - span, 128, (R, K // 32), generator=g).to(torch.uint8)) for R in (M, N))
        within(q4.linear_mx4(x, w), x, w)


@pytest.mark.parametrize("M,N", SHAPES)
def test_a_sum_and_the_blocks_far_below_it(M, N):
    """1, then four blocks of 32 equal products each at 2^-k: kept, rounded or lost, the same in every kernel."""
    K = 256
    gu.note("linear_mx4 far blocks M=%d N=%d: %s" % (M, N, form_of(False, M, N, K)))
    for code, value in ((1, 0.5), (2, 1.0), (3, 1.5), (7, 6.0)):
        w = torch.zeros(N, K, dtype=torch.uint8)
        w[:, 0], w[:, 128:] = 2, code
        w = pack(w, torch.full((N, K // 32), 127, dtype=torch.uint8))
        for k in range(16, 36):
            x = torch.zeros(M, K, dtype=torch.uint8)
            x[:, 0], x[:, 128:] = 2, code
            s = torch.full((M, K // 32), 127 - k, dtype=torch.uint8)
            s[:, :4] = 127
            y = q4.linear_mx4(pack(x, s), w)
            assert (y == y[0, 0]).all()
            small = 128 * Fraction(value) ** 2 / 2 ** k
            off = abs(Fraction(y[0, 0].item()) - 1 - small)
            # four blocks join a sum that stands (4.5 each), then nothing else rounds
            assert off <= 4 * Fraction(9, 2) / 2 ** 24 * (1 + small), (code, k, float(off))


def test_values_of_like_size_stay_exact():
    """Products are multiples of a quarter of their scales: sums below 2^22 of that are exact."""
    g = torch.Generator()
    g.manual_seed(3)
    for M, N, K in ((1, 40, 2048), (40, 300, 2048), (300, 5000, 1024)):
        x, w = (pack(torch.randint(0, 16, (R, K), generator=g, dtype=torch.uint8),
                     torch.full((R, K // 32), 127, dtype=torch.uint8)) for R in (M, N))
        want = q4.dequantize_mx4(x).double() @ q4.dequantize_mx4(w).double().T.contiguous()
        assert torch.equal(q4.linear_mx4(x, w).double(), want)
