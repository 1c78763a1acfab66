"""The microscaled 4-bit form and its product on the GPU against plain 64-bit
computations.

Codes, scales and packed bytes are integer decisions: equal, bit for bit, and
so are the values that they stand for.  The product is a chain of ceil(K / 128)
steps; each adds its 128 products to the sum with an error of at most 2^-23 of
the magnitudes that it adds, which are at most the sum of |x w| over the row:
an output is off by at most ceil(K / 128) 2^-23 of that sum, then by its type's
own rounding: finfo(type).eps / 2 of the value, and half its smallest number."""
import ctypes

import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from bit_quantized_matmul_q4_amd import _lib
from tests import gpu_util as gu
from tests import mx4_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rows(seed, R, K, dtype, wide=False):
    g = gen(seed)
    x = torch.randn(R, K, generator=g)
    if wide:  # blocks of very different size
        x = x * torch.exp2(torch.randint(-12, 4, (R, K // 32, 1), generator=g).float()).expand(R, K // 32, 32).reshape(R, K)
    return x.to(DTYPES[dtype])


def matrix(codes, scales):
    return q4.pack_mx4(ref.nibbles(codes).to(gu.DEV), scales.to(gu.DEV))


def bound(K, y, mag, dtype):
    t = DTYPES[dtype]
    f = torch.finfo(t)
    return -(-K // 128) * 2.0 ** -23 * mag + f.eps / 2 * (y.abs() + mag * 2.0 ** -20) + f.smallest_normal * f.eps


def check(y, x, w, dtype, what):
    want, mag = ref.product(x, w)
    got = y.cpu().double()
    off = (got - want).abs() - bound(x.shape[1], want, mag, dtype)
    assert (off <= 0).all(), "%s: %g over at %s" % (what, off.max(), divmod(int(off.argmax()), want.shape[1]))


# ------------------------------------------------------------- quantization
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("R,K", [(1, 32), (1, 3584), (2, 64), (15, 96), (16, 128), (17, 160), (33, 512), (5, 544),
                                 (64, 896), (3, 18944), (130, 1056)])
def test_quantize(R, K, dtype):
    gu.note("quantize %dx%d %s" % (R, K, dtype))
    x = rows(R * 7 + K, R, K, dtype, wide=True)
    x[0, :32] = 0
    codes, scales = ref.quantize(x)
    c, s = q4.quantize_mx4(x.to(gu.DEV))
    assert torch.equal(s.cpu(), scales)
    assert torch.equal(c.cpu(), ref.nibbles(codes))
    want_c, want_s = ref.packed(codes, scales)
    for m in (q4.quantize_pack_mx4(x.to(gu.DEV)), q4.pack_mx4(c, s)):
        assert (m.rows, m.K) == (R, K)
        assert torch.equal(m.codes.cpu(), want_c) and torch.equal(m.scales.cpu(), want_s)
    v = ref.values(codes, scales)
    for d in DTYPES.values():
        assert torch.equal(q4.dequantize_mx4(m, d).cpu(), v.to(d))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_quantize_borders(dtype):
    """Values on and next to every border between codes, at scales from the smallest to the largest."""
    t = DTYPES[dtype]
    f = torch.finfo(t)
    marks = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.5, 2.0], dtype=torch.float64)
    near = torch.cat([marks, marks * (1 + f.eps), marks * (1 - f.eps / 2)])[:31]
    if dtype == "f16":
        exps = list(range(-22, 14))
    else:
        exps = list(range(-127, 126)) if dtype == "f32" else list(range(-133, 126))
    x = torch.zeros(len(exps), 64, dtype=torch.float64)
    for i, e in enumerate(exps):
        x[i, :31] = torch.ldexp(near, torch.tensor(e))
        x[i, 31] = 2.0 ** (e + 2)
        x[i, 32:] = -x[i, :32]
    x = x.to(t)
    assert torch.isfinite(x).all()
    codes, scales = ref.quantize(x)
    c, s = q4.quantize_mx4(x.to(gu.DEV))
    assert torch.equal(s.cpu(), scales) and torch.equal(c.cpu(), ref.nibbles(codes))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_every_value(dtype):
    """Every finite 16-bit value, in blocks whose largest value is 1, 2 or 4 times its power of two."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DTYPES[dtype])
    v = bits[torch.isfinite(bits)]
    v = v[torch.argsort(v.double().abs(), stable=True)]
    for lift in (1, 31):  # a value beside 31 neighbours, and beside 31 that are larger
        n = v.numel() // 32 * 32
        x = v[:n].reshape(-1, 32) if lift == 1 else v[:n].reshape(32, -1).T.contiguous()
        x = x[:x.shape[0] // 2 * 2].reshape(-1, 64)
        codes, scales = ref.quantize(x)
        c, s = q4.quantize_mx4(x.to(gu.DEV))
        assert torch.equal(s.cpu(), scales) and torch.equal(c.cpu(), ref.nibbles(codes))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_quantize_not_finite(dtype):
    x = rows(5, 20, 256, dtype)
    x[3, 40] = float("inf")
    x[4, 31] = float("nan")
    x[5, 32] = float("-inf")
    x[19, 255] = float("nan")
    x[7] = 0
    x[8, :] = -0.0
    codes, scales = ref.quantize(x)
    c, s = q4.quantize_mx4(x.to(gu.DEV))
    assert torch.equal(s.cpu(), scales) and torch.equal(c.cpu(), ref.nibbles(codes))
    m = q4.quantize_pack_mx4(x.to(gu.DEV))
    v = q4.dequantize_mx4(m).cpu()
    assert torch.equal(torch.isnan(v), torch.isnan(ref.values(codes, scales)))
    w = rows(6, 40, 256, "f32")
    wc, wsc = ref.quantize(w)
    y = q4.linear_mx4(m, matrix(wc, wsc)).cpu()
    bad = torch.zeros(20, dtype=torch.bool)
    bad[[3, 4, 5, 19]] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
    assert (y[7] == 0).all() and (y[8] == 0).all()
    wsc[11, 2] = 255
    y = q4.linear_mx4(m, matrix(wc, wsc)).cpu()
    assert torch.isnan(y[:, 11]).all() and torch.isfinite(y[~bad][:, :11]).all() and torch.isfinite(y[~bad][:, 12:]).all()


def test_dequantize_every_code_and_scale():
    """Every code times every scale byte, in every type: rounded once, an infinity past the type's largest."""
    codes = torch.arange(16, dtype=torch.uint8).repeat(256, 2)
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None]
    m = matrix(codes, scales)
    v = ref.values(codes, scales)
    for t in DTYPES.values():
        got = q4.dequantize_mx4(m, t).cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(v))
        # (a value rounds to binary32 first: exact below 2^128 but for the type's own rounding)
        assert torch.equal(got.nan_to_num(nan=0.0, posinf=float("inf"), neginf=float("-inf")),
                           v.to(torch.float32).to(t).nan_to_num(nan=0.0, posinf=float("inf"), neginf=float("-inf")))


# ------------------------------------------------------------------ product
SHAPES = [(1, 1, 32), (1, 16, 128), (1, 40, 18944), (2, 17, 64), (3, 33, 160), (4, 100, 512), (5, 40, 544),
          (8, 64, 3584), (9, 31, 96), (15, 48, 1056), (16, 16, 896), (17, 300, 384), (31, 65, 640), (33, 70, 9984),
          (48, 129, 32), (63, 20, 2080), (64, 64, 512), (65, 130, 160), (70, 33, 20512), (100, 257, 896),
          (124, 301, 18944), (128, 128, 1024), (129, 200, 672), (200, 97, 4864), (257, 513, 288), (300, 60, 131072)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("x_dtype,y_dtype", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_linear(M, N, K, x_dtype, y_dtype):
    gu.note("linear %dx%dx%d %s %s" % (M, N, K, x_dtype, y_dtype))
    x = rows(M + N + K, M, K, x_dtype)
    wc, wsc = ref.quantize(rows(M * N, N, K, "f32", wide=True) / K ** 0.5)
    w = matrix(wc, wsc)
    y = q4.linear_mx4(x.to(gu.DEV), w, out_dtype=DTYPES[y_dtype])
    assert y.dtype == DTYPES[y_dtype] and tuple(y.shape) == (M, N)
    check(y, ref.values(*ref.quantize(x)), ref.values(wc, wsc), y_dtype, (M, N, K))
    packed = q4.quantize_pack_mx4(x.to(gu.DEV))
    again = q4.linear_mx4(packed, w, out_dtype=DTYPES[y_dtype])
    assert torch.equal(again, y)


@pytest.mark.parametrize("K", [128, 256, 3584])
def test_linear_wide_scales(K):
    """Random codes with scales over 50 powers of two: a step's error is at most 2^-23 of the magnitudes it adds."""
    g = gen(K)
    M, N = 37, 90
    xc = torch.randint(0, 16, (M, K), generator=g).to(torch.uint8)
    wc = torch.randint(0, 16, (N, K), generator=g).to(torch.uint8)
    xs = torch.randint(100, 150, (M, K // 32), generator=g).to(torch.uint8)
    ws = torch.randint(100, 150, (N, K // 32), generator=g).to(torch.uint8)
    check(q4.linear_mx4(matrix(xc, xs), matrix(wc, ws)), ref.values(xc, xs), ref.values(wc, ws), "f32", K)


def test_linear_scales_at_the_ends():
    """The smallest and largest scales against each other, results below and past binary32's range."""
    K, v = 128, torch.full((1, 128), 2, dtype=torch.uint8)  # ones
    for ex in (0, 1, 120, 127, 200, 253, 254):
        for ew in (0, 1, 127, 130, 254):
            want = 128 * 2.0 ** (ex + ew - 254)
            x = matrix(v, torch.full((1, K // 32), ex, dtype=torch.uint8))
            w = matrix(v, torch.full((1, K // 32), ew, dtype=torch.uint8))
            y = q4.linear_mx4(x, w).cpu()
            assert y.item() == torch.tensor(want, dtype=torch.float64).to(torch.float32).item(), (ex, ew)


# rows of one batch against the same rows in others: (N, K)
@pytest.mark.parametrize("N,K", [(40, 18944), (300, 3584), (2000, 160), (97, 9984)])
@pytest.mark.parametrize("x_dtype", ["bf16", "f16"])
def test_rows_do_not_depend_on_the_batch(N, K, x_dtype):
    x = rows(N, 600, K, x_dtype, wide=True).to(gu.DEV)
    w = q4.quantize_pack_mx4((rows(K, N, K, "f32", wide=True) / K ** 0.5).to(gu.DEV))
    full = q4.linear_mx4(x, w)
    for M in (1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 511):
        for first in (0, 600 - M):
            gu.note("rows %d from %d of N=%d K=%d" % (M, first, N, K))
            part = x[first:first + M].contiguous()
            assert torch.equal(q4.linear_mx4(part, w), full[first:first + M])
            assert torch.equal(q4.linear_mx4(q4.quantize_pack_mx4(part), w), full[first:first + M])


def test_columns_do_not_depend_on_the_others():
    x = rows(1, 70, 1056, "bf16").to(gu.DEV)
    wd = (rows(2, 700, 1056, "f32") / 30).to(gu.DEV)
    full = q4.linear_mx4(x, q4.quantize_pack_mx4(wd))
    for N in (1, 15, 64, 333):
        assert torch.equal(q4.linear_mx4(x, q4.quantize_pack_mx4(wd[:N].contiguous())), full[:, :N])


# ------------------------------------------------------- calls and refusals
def test_out_workspace_and_unaligned_outputs():
    x = rows(3, 20, 512, "bf16").to(gu.DEV)
    w = q4.quantize_pack_mx4(rows(4, 36, 512, "f32").to(gu.DEV))
    y = q4.linear_mx4(x, w)
    need = _lib.load().q4_mx4_workspace_bytes(20, 36, 512, _lib.Q4_BF16)
    work = torch.empty(max(need, 256), dtype=torch.uint8, device=gu.DEV)
    for t in DTYPES.values():
        buf = torch.full((20 * 36 + 9,), 7.0, dtype=t, device=gu.DEV)
        for off in (0, 1, 3):
            out = buf[off:off + 720].view(20, 36)
            assert q4.linear_mx4(x, w, out=out, workspace=work) is out
            assert torch.equal(out, y.to(t))
            buf[off:off + 720] = 7.0
            assert (buf == 7.0).all()  # nothing outside
    with pytest.raises(q4.Q4Error):
        q4.linear_mx4(rows(3, 300, 512, "bf16").to(gu.DEV), w, workspace=None)


def test_nothing_outside_is_written():
    """Codes, scales and values between guard bytes."""
    lib = _lib.load()
    R, K = 19, 672
    x = rows(8, R, K, "bf16").to(gu.DEV)
    nc, ns = lib.q4_mx4_code_bytes(R, K), lib.q4_mx4_scale_bytes(R, K)
    stream = torch.cuda.current_stream().cuda_stream
    buf = torch.full((nc + ns + 768,), 0xA5, dtype=torch.uint8, device=gu.DEV)
    c, s = buf[256:256 + nc], buf[512 + nc:512 + nc + ns]
    _lib.check(lib.q4_mx4_quantize_pack(x.data_ptr(), _lib.Q4_BF16, c.data_ptr(), s.data_ptr(), R, K, stream), "pack")
    want = q4.quantize_pack_mx4(x)
    assert torch.equal(c, want.codes) and torch.equal(s, want.scales)
    for a, b in ((0, 256), (256 + nc, 512 + nc), (512 + nc + ns, 768 + nc + ns)):
        assert (buf[a:b] == 0xA5).all()
    out = torch.full((R * K + 128,), 3.0, dtype=torch.bfloat16, device=gu.DEV)
    q4.dequantize_mx4(want, out=out[64:64 + R * K].view(R, K))
    assert (out[:64] == 3).all() and (out[64 + R * K:] == 3).all()


def test_binding_refuses():
    x = rows(3, 4, 64, "bf16").to(gu.DEV)
    m = q4.quantize_pack_mx4(rows(4, 40, 64, "f32").to(gu.DEV))
    with pytest.raises(TypeError, match="dtype"):
        q4.linear_mx4(x.float(), m)
    with pytest.raises(ValueError, match="K=96"):
        q4.linear_mx4(rows(3, 4, 96, "bf16").to(gu.DEV), m)
    with pytest.raises(TypeError, match="Mx4Matrix"):
        q4.linear_mx4(x, x)
    with pytest.raises(TypeError, match="out_dtype"):
        q4.linear_mx4(x, m, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="out must be"):
        q4.linear_mx4(x, m, out=torch.empty(4, 41, device=gu.DEV))
    with pytest.raises(ValueError, match="does not hold"):
        q4.linear_mx4(x, q4.Mx4Matrix(m.codes, m.scales, 400, 64))
    with pytest.raises(ValueError, match="contiguous"):
        q4.quantize_mx4(rows(3, 64, 64, "f32").to(gu.DEV).T)
    with pytest.raises(ValueError, match="bad shape"):
        q4.quantize_pack_mx4(rows(3, 4, 64, "f32")[:, :48].contiguous().to(gu.DEV))
    with pytest.raises(ValueError, match="scales must be"):
        q4.pack_mx4(torch.zeros(4, 32, dtype=torch.uint8, device=gu.DEV),
                    torch.zeros(4, 3, dtype=torch.uint8, device=gu.DEV))
    with pytest.raises(ValueError, match="bad shape"):
        q4.quantize_pack_mx4(torch.empty(0, 64, device=gu.DEV))


def test_another_stream():
    x = rows(3, 300, 3584, "bf16").to(gu.DEV)
    w = q4.quantize_pack_mx4(rows(4, 700, 3584, "f32").to(gu.DEV))
    want = q4.linear_mx4(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [q4.linear_mx4(x, w) for _ in range(3)]
    here = [q4.linear_mx4(x, w) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got + here)


@pytest.mark.parametrize("M", [1, 4, 12, 40, 300])
def test_captured(M):
    """A captured call replayed over changing inputs, eager calls between."""
    w = q4.quantize_pack_mx4(rows(4, 300, 1056, "f32").to(gu.DEV))
    x = torch.empty(M, 1056, dtype=torch.bfloat16, device=gu.DEV)
    x.copy_(rows(1, M, 1056, "bf16"))
    q4.linear_mx4(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = q4.linear_mx4(x, w)
    for seed in range(4):
        x.copy_(rows(seed, M, 1056, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, q4.linear_mx4(x, w))
