"""Every kernel of the microscaled 4-bit product on the GPU, at shapes named by
the kernel they take (tests/mx4_forms.py; the rule itself is checked on the
CPU), with the bounds of test_mx4_gpu.py; and the form at the largest rows,
columns and lengths that the library takes."""
import random

import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from bit_quantized_matmul_q4_amd import _lib
from tests import gpu_util as gu
from tests import mx4_ref as ref
from tests.mx4_forms import FORMS, form_of
from tests.test_mx4_gpu import DTYPES, bound, matrix, rows

pytestmark = pytest.mark.gpu

CASES = [(form, shape) for form, shapes in FORMS.items() for shape in shapes]
IDS = ["%s-%dx%dx%d" % (form, *shape) for form, shape in CASES]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()
    yield
    torch.cuda.empty_cache()


def cuda_gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def check_on_gpu(y, x, w, dtype, what):
    """check() of test_mx4_gpu.py, with the 64-bit products on the GPU (both values and magnitudes)."""
    x, w = x.to(gu.DEV), w.to(gu.DEV)
    want, mag = x @ w.T.contiguous(), x.abs() @ w.abs().T.contiguous()
    off = (y.double() - want).abs() - bound(x.shape[1], want, mag, dtype)
    assert (off <= 0).all(), "%s: %g over" % (what, off.max())


@pytest.mark.parametrize("form,shape", CASES, ids=IDS)
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_form(form, shape, xt, yt):
    """Against the sums in 64 bits; packed x gives the same bits; nothing past the outputs is written."""
    M, N, K = shape
    assert form_of(True, M, N, K) == form
    gu.note("linear_mx4 %s M=%d N=%d K=%d %s -> %s" % (form, M, N, K, xt, yt))
    x = rows(M * 3 + N, M, K, xt, wide=K < 20000)
    xc = ref.quantize(x)
    g = cuda_gen(N + K)
    size = torch.exp2(torch.randint(-12, 4, (N, K // 32, 1), generator=g, device=gu.DEV).float())
    w = q4.quantize_pack_mx4((torch.randn(N, K // 32, 32, generator=g, device=gu.DEV) * size).view(N, K) / K ** 0.5)
    buf = torch.full((M * N + 64,), 7.0, dtype=DTYPES[yt], device=gu.DEV)
    y = buf[32:32 + M * N].view(M, N)
    q4.linear_mx4(x.to(gu.DEV), w, out=y)
    shared = q4.linear_mx4(q4.quantize_pack_mx4(x.to(gu.DEV)), w, out_dtype=DTYPES[yt])
    torch.cuda.synchronize()
    assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()
    assert torch.equal(y, shared)
    check_on_gpu(y, ref.values(*xc), q4.dequantize_mx4(w).double(), yt, (form, M, N, K))


@pytest.mark.parametrize("form,shape", [c for c in CASES if c[1][0] > 32], ids=[i for i, c in zip(IDS, CASES) if c[1][0] > 32])
def test_rows_have_the_bits_of_the_smaller_forms(form, shape):
    """Rows of a large batch against the same rows through the kernels for fewer."""
    M, N, K = shape
    g = cuda_gen(M + K)
    x = torch.randn(M, K, device=gu.DEV, generator=g).bfloat16()
    w = q4.quantize_pack_mx4(torch.randn(N, K, device=gu.DEV, generator=g))
    whole = q4.linear_mx4(x, w)
    for n in (1, 5, 16, 17, 33, 65, 100):
        if n >= M:
            continue
        for at in (0, M // 2, M - n):
            gu.note("linear_mx4 %s rows %d at %d of M=%d N=%d K=%d: %s" % (form, n, at, M, N, K,
                                                                          form_of(True, n, N, K)))
            part = q4.linear_mx4(x[at:at + n].contiguous(), w)
            torch.cuda.synchronize()
            assert torch.equal(part.view(torch.int32), whole[at:at + n].view(torch.int32)), (n, at)


@pytest.mark.parametrize("form,shape", [(f, s[0]) for f, s in FORMS.items()], ids=list(FORMS))
def test_not_a_number_stays_in_its_row_and_column(form, shape):
    M, N, K = shape
    gu.note("linear_mx4 NaN %s M=%d N=%d K=%d" % (form, M, N, K))
    x = rows(1, M, K, "bf16")
    x[M - 1, K - 1] = float("inf")
    codes, scales = ref.quantize(rows(2, min(N, 64), K, "f32"))
    scales[0, 0] = 255
    reps = -(-N // 64)
    w = matrix(codes.repeat(reps, 1)[:N].contiguous(), scales.repeat(reps, 1)[:N].contiguous())
    y = torch.isnan(q4.linear_mx4(x.to(gu.DEV), w)).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M - 1] = True
    want[:, 0::64] = True
    assert torch.equal(y, want)


@pytest.mark.parametrize("form,shape", [(f, s[-1]) for f, s in FORMS.items()], ids=list(FORMS))
def test_captured_beside_another_stream(form, shape):
    """Replays of a captured call on new inputs, while another stream runs the same shape; each against an eager call."""
    M, N, K = shape
    gu.note("linear_mx4 captured, two streams, %s M=%d N=%d K=%d" % (form, M, N, K))
    w = q4.quantize_pack_mx4(torch.randn(N, K, device=gu.DEV, generator=cuda_gen(1)) / K ** 0.5)
    xs = [torch.randn(M, K, device=gu.DEV, generator=cuda_gen(2 + i)).bfloat16() for i in range(4)]
    want = [q4.linear_mx4(x, w) for x in xs]
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = q4.linear_mx4(x, w)
    other = torch.cuda.Stream()
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            beside = [q4.linear_mx4(xs[j], w) for j in (i - 1, i)]
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(beside[0], want[i - 1]) and torch.equal(beside[1], want[i])


def at_random(seed):
    """A shape over the whole range (the logarithm of each size spread evenly), products of 8e10 at most."""
    rng = random.Random(seed)
    while True:
        M, N, K = (int(round(2 ** rng.uniform(0, top))) for top in (12, 15.5, 9.6))
        if 1 << 20 <= M * N * 32 * K <= 8e10:
            return M, N, 32 * K


@pytest.mark.parametrize("seed", range(96))
def test_shapes_at_random(seed):
    """Against the sums in 64 bits; the same bits from packed rows, from a row alone and from a second call."""
    M, N, K = at_random(seed)
    yt = ("f32", "bf16", "f16")[seed % 3]
    gu.note("linear_mx4 M=%d N=%d K=%d -> %s: %s" % (M, N, K, yt, form_of(True, M, N, K)))
    x = torch.randn(M, K, device=gu.DEV, generator=cuda_gen(seed)).to(DTYPES["f16" if seed & 1 else "bf16"])
    xq = q4.quantize_pack_mx4(x)
    w = q4.quantize_pack_mx4(torch.randn(N, K, device=gu.DEV, generator=cuda_gen(seed + 1000)) / K ** 0.5)
    y = q4.linear_mx4(x, w, out_dtype=DTYPES[yt])
    m = seed % M
    for what, other, of in (("again", q4.linear_mx4(x, w, out_dtype=DTYPES[yt]), y),
                            ("packed", q4.linear_mx4(xq, w, out_dtype=DTYPES[yt]), y),
                            ("a row", q4.linear_mx4(x[m:m + 1].contiguous(), w, out_dtype=DTYPES[yt]), y[m:m + 1])):
        assert torch.equal(other, of), what
    check_on_gpu(y, q4.dequantize_mx4(xq).double(), q4.dequantize_mx4(w).double(), yt, (M, N, K))


# ---------------------------------------------------------------- the limits
@pytest.mark.parametrize("M,N", [(1 << 24, 17), ((1 << 24) - 3, 65)])
def test_most_rows(M, N):
    gu.note("linear_mx4 M=%d N=%d" % (M, N))
    K = 32
    x = torch.randn(M, K, device="cuda", generator=cuda_gen(1), dtype=torch.bfloat16)
    w = q4.quantize_pack_mx4(torch.randn(N, K, device="cuda", generator=cuda_gen(2)))
    y = q4.linear_mx4(x, w)
    for at in (0, M // 2 - 7, M - 40):
        part = q4.linear_mx4(x[at:at + 40].contiguous(), w)
        torch.cuda.synchronize()
        assert torch.equal(part, y[at:at + 40]), at
    m = q4.quantize_pack_mx4(x)
    back = q4.dequantize_mx4(m, torch.bfloat16)
    part = q4.dequantize_mx4(q4.quantize_pack_mx4(x[M - 40:].contiguous()), torch.bfloat16)
    assert torch.equal(back[M - 40:], part)
    codes, scales = q4.quantize_mx4(x)
    again = q4.pack_mx4(codes, scales)
    assert torch.equal(again.codes, m.codes) and torch.equal(again.scales, m.scales)


@pytest.mark.parametrize("M", [1, 16, 20, 40, 100, 200])
def test_most_columns(M):
    N, K = 1 << 24, 32
    gu.note("linear_mx4 M=%d N=%d" % (M, N))
    x = torch.randn(M, K, device="cuda", generator=cuda_gen(3), dtype=torch.bfloat16)
    codes, scales = q4.quantize_mx4(torch.randn(N, K, device="cuda", generator=cuda_gen(4)))
    y = q4.linear_mx4(x, q4.pack_mx4(codes, scales), out_dtype=torch.bfloat16)
    for at in (0, N // 2 - 32, N - 64):
        part = q4.linear_mx4(x, q4.pack_mx4(codes[at:at + 64].contiguous(), scales[at:at + 64].contiguous()),
                             out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        assert torch.equal(part, y[:, at:at + 64].contiguous()), at


@pytest.mark.parametrize("M", [1, 17, 70, 700])
def test_longest_rows(M):
    N, K = 161, 1 << 17
    gu.note("linear_mx4 M=%d K=%d" % (M, K))
    x = torch.randn(M, K, device="cuda", generator=cuda_gen(5)).half()
    w = q4.quantize_pack_mx4(torch.randn(N, K, device="cuda", generator=cuda_gen(6)))
    y = q4.linear_mx4(x, w)
    check_on_gpu(y, q4.dequantize_mx4(q4.quantize_pack_mx4(x)).double(), q4.dequantize_mx4(w).double(), "f32", M)


def test_most_units():
    """More pieces of 16 rows by 512 k than the quantizer's, packer's and reader's grids."""
    R, K = (1 << 16) + 5, 1 << 17
    gu.note("quantize %dx%d" % (R, K))
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    x = torch.randn(R, K, device="cuda", generator=cuda_gen(7), dtype=torch.bfloat16)
    m = q4.quantize_pack_mx4(x)
    part = q4.quantize_pack_mx4(x[R - 21:].contiguous())  # (starts on a tile)
    assert torch.equal(m.codes[-part.codes.numel():], part.codes)
    assert torch.equal(m.scales[-part.scales.numel():], part.scales)
    back = q4.dequantize_mx4(m, torch.bfloat16)
    assert torch.equal(back[R - 21:], q4.dequantize_mx4(part, torch.bfloat16))


@pytest.mark.parametrize("M,H,mx4", [(1 << 20, 8, False), ((1 << 20) - 7, 32, True), (3, 32768, True)])
def test_norm_limits(M, H, mx4):
    gu.note("block_norm %dx%d" % (M, H))
    y = torch.randn(M, H, device="cuda", generator=cuda_gen(8))
    res = torch.randn(M, H, device="cuda", generator=cuda_gen(9)).bfloat16()
    n = q4.Norm(torch.ones(H, device="cuda"))
    r, h = q4.block_norm(y, res, pre=n)
    k = min(M, 50)
    pr, ph = q4.block_norm(y[M - k:].contiguous(), res[M - k:].contiguous(), pre=n)
    assert torch.equal(r[M - k:], pr) and torch.equal(h[M - k:], ph)
    if mx4:
        _, packed = q4.block_norm(y, res, pre=n, out_dtype="mx4")
        _, part = q4.block_norm(y[M - k:].contiguous(), res[M - k:].contiguous(), pre=n, out_dtype="mx4")
        assert torch.equal(q4.dequantize_mx4(packed)[M - k:], q4.dequantize_mx4(part))
