"""The norms around a block where their statistics leave the ordinary range, on
the GPU: rows of equal and of nearly equal values, and an eps next to the
largest number.

A layer norm of equal values is exactly 0 (then weight and bias): every
difference from the mean is 0, and so is their square's mean, whatever the row's
size.  With eps 0 it is 0 / 0.  Of nearly equal values the bounds of
test_norm_gpu.py hold, with the 64-bit formula on the differences from the row's
first value (which are exact, and have the same norm)."""
import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from tests import gpu_util as gu
from tests.test_norm_gpu import check, dev, gen, norm64, norm_error, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()


# 3622 and 31145: a binary32 sum of so many equal values, divided by their
# number, is one and three units off for the second and third of FACTORS.
WIDTHS = [1, 40, 64, 896, 3584, 3622, 4096, 4863, 9000, 31145, 32768]
FACTORS = (1.0, 1.4600450992584229, 1.8647782802581787)


def equal_rows(H, exponents):
    """Rows of one value each: FACTORS times a power of two, of either sign."""
    v = torch.tensor([s * f * 2.0 ** e for e in exponents for f in FACTORS for s in (1, -1)], dtype=torch.float64)
    return v.float()[:, None].expand(-1, H).contiguous()


def layer(eps, weight=None, bias=None):
    return {"kind": "layer", "weight": weight, "bias": bias, "eps": eps}


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("eps", [1e-5, 1e-6, 1e-30, 1e-40])
def test_equal_values(H, eps):
    """0 as h, and nothing onto the residual as post, from the smallest values to the largest."""
    gu.note("equal values H=%d eps %g" % (H, eps))
    y = equal_rows(H, (-149, -140, -126, -100, -60, -41, -20, 0, 20, 30, 40, 63, 64, 80, 100, 113, 119, 120, 127))
    g = gen(H)
    bias = torch.randn(H, generator=g)
    h = run(y, None, None, None, 1.0, layer(eps), out_dtype=torch.float32)[1].cpu()
    assert (h == 0).all(), (h != 0).any(1).nonzero().view(-1).tolist()
    h = run(y, None, None, None, 1.0, layer(eps, torch.full((H,), 3.0), bias), out_dtype=torch.float32)[1].cpu()
    assert torch.equal(h, bias.expand_as(h))
    res = torch.randn(y.shape, generator=g).bfloat16()
    r, h = run(y, res, layer(eps), None, 2.0, None)
    assert torch.equal(r.cpu(), res) and torch.equal(h.cpu(), res)


@pytest.mark.parametrize("dtype,exponents", [("bf16", (-130, -20, 0, 64, 100, 120, 127)), ("f16", (-24, -14, 0, 15))])
@pytest.mark.parametrize("H", [1, 64, 3584, 4863])
def test_equal_values_of_16_bits(dtype, exponents, H):
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    y = equal_rows(H, exponents).to(t)
    assert torch.isfinite(y).all()
    for eps in (1e-5, 1e-6, 1e-30):
        gu.note("equal values %s H=%d eps %g" % (dtype, H, eps))
        h = run(y, None, None, None, 1.0, layer(eps), out_dtype=t)[1]
        assert (h == 0).all()


@pytest.mark.parametrize("H", [64, 896, 3584, 9024, 32768])
def test_equal_values_in_packed_rows(H):
    """Codes of zeros, no block that is not a number, and so products of 0."""
    gu.note("equal values packed H=%d" % H)
    y = equal_rows(H, (0, 60, 100, 119, 127))
    w = q4.quantize_pack_mx4(torch.randn(40, H, generator=gen(H)).to(gu.DEV))
    for eps in (1e-6, 1e-30):
        h = run(y, None, None, None, 1.0, layer(eps), out_dtype="mx4")[1]
        assert (h.scales == 0).all()
        assert (q4.dequantize_mx4(h) == 0).all()
        assert (q4.linear_mx4(h, w) == 0).all()


@pytest.mark.parametrize("H", [1, 40, 3584, 3622, 31145])
def test_equal_values_without_eps(H):
    """0 / 0, in both kinds of norm of zeros too; a rms norm of equal values is 1."""
    y = torch.cat([equal_rows(H, (-100, 0, 60, 120)), torch.zeros(1, H)])
    h = run(y, None, None, None, 1.0, layer(0.0), out_dtype=torch.float32)[1]
    assert torch.isnan(h).all()
    h = run(y, None, None, None, 1.0, {**layer(0.0), "kind": "rms"}, out_dtype=torch.float32)[1].cpu()
    assert torch.isnan(h[-1]).all()
    check(h[:-1], torch.sign(y[:-1].double()), (54 / 2 + 6) * 2.0 ** -24 * torch.ones(1, H).double(), H)


@pytest.mark.parametrize("H", [40, 896, 3584, 3622, 4863, 31145, 32768])
@pytest.mark.parametrize("exponent", [-100, 0, 30, 60, 120])
def test_nearly_equal_values(H, exponent):
    """Rows in which one value, half of them or all of them are some units off the others."""
    g = gen(H + exponent)
    rows = []
    for f in FACTORS:
        unit = 2.0 ** -23
        one, half = torch.zeros(H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
        one[H // 3] = unit
        half[::2] = 2 * unit
        rows += [f + one, f + half, f + unit * torch.randint(0, 4, (H,), generator=g).double()]
    y = torch.stack(rows) * 2.0 ** exponent
    assert torch.equal(y, y.float().double())
    for eps in (0.0, 1e-30, 1e-6):
        gu.note("nearly equal values H=%d 2^%d eps %g" % (H, exponent, eps))
        n = layer(eps)
        h = run(y.float(), None, None, None, 1.0, n, out_dtype=torch.float32)[1]
        d = y - y[:, :1]
        # Where eps keeps the row as it is (over 2^-40), what is left about the mean may be subnormal: it rounds to a
        # multiple of 2^-149, so that every difference is off by 2^-150 at most (a subtraction there is exact).
        e = torch.full_like(d, 2.0 ** -150 if eps > 2.0 ** -40 else 0.0)
        check(h, norm64(d, n), norm_error(d, e, n), (H, exponent, eps))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [1, 2, 3, 8, 40, 896, 3584])
def test_large_eps(kind, H):
    """An eps up to the largest number, beside squares that reach the rest of the range or none of it."""
    g = gen(H)
    base = torch.randn(12, H, generator=g)
    base = base / base.abs().max(1, keepdim=True).values
    size = torch.tensor([0.0, 1e-30, 1.0, 1e10, 1e17, 1e18, 5e18, 1e19, 1.8e19, 2.5e19, 1e25, 3e38], dtype=torch.float64)
    y = (base.double() * size[:, None]).float()
    for eps in (1.0, 1e30, 1e37, 1.7e38, 3.3e38, torch.finfo(torch.float32).max):
        gu.note("%s H=%d eps %g" % (kind, H, eps))
        n = {"kind": kind, "weight": None, "bias": None, "eps": eps}
        h = run(y, None, None, None, 1.0, n, out_dtype=torch.float32)[1]
        n["eps"] = torch.tensor(eps, dtype=torch.float32).double().item()
        check(h, norm64(y.double(), n), norm_error(y.double(), torch.zeros_like(y).double(), n), (kind, H, eps))
