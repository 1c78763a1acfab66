"""The 8-bit product on the GPU against plain 64-bit computations.

Codes and scales are integer decisions and one rounding: equal, bit for bit.
The product's sum is an exact integer, so an output is
fl(fl(fl32(sum) sx) sw), three roundings of at most 2^-24 of the value each
(plus half the smallest float32 where it underflows), then the output type's
own: finfo(type).eps / 2 of the value, and half its smallest number."""
import ctypes

import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from bit_quantized_matmul_q4_amd import _lib
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def codes_of(x):
    """The quantizer's rule in 64 bits (x on the CPU)."""
    d = x.double()
    bad = ~torch.isfinite(d).all(1)
    s = (torch.where(bad[:, None], torch.zeros_like(d), d).abs().amax(1) / 127).float()
    div = torch.where(s > 0, s, torch.ones_like(s)).double()[:, None]
    q = torch.round(d / div).clamp(-127, 127)
    q[(s == 0) | bad] = 0
    s[bad] = float("nan")
    return q, s


def tiles_of(codes):
    R, K = codes.shape
    T, Q = -(-R // 16), 2 * -(-K // 128)
    p = torch.zeros((T * 16, Q * 64), dtype=torch.int8)
    p[:R, :K] = codes
    return p.view(T, 16, Q, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1)


def check_y(y, qx, sx, qw, sw, what):
    """y against the exact product, output by output."""
    ref = (qx.double() @ qw.double().T) * sx.double()[:, None] * sw.double()[None, :]
    y = y.cpu()
    fi = torch.finfo(y.dtype)
    tol = ref.abs() * (3.01 * 2.0**-24)
    tol = tol + 2.0**-148
    if y.dtype != torch.float32:
        tol = tol * (1 + fi.eps) + ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
    got = y.double()
    over = ref.abs() > fi.max  # rounds to infinity, or just below it
    ok = ((got - ref).abs() <= tol) | (torch.isnan(ref) & torch.isnan(got)) | (over & (got.abs() >= fi.max))
    assert ok.all(), "%s: %d of %d outputs off, worst at %s" % (
        what, int((~ok).sum()), ok.numel(), torch.nonzero(~ok)[:3].tolist())


def tricky_rows(g, R, K, dtype):
    """Rows of different size, with values on and next to the borders between codes."""
    x = torch.randn(R, K, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))
    for r in range(0, R, 3):
        s = float((torch.rand(1, generator=g) + 0.5) * 2.0 ** (r % 19 - 9))
        k = torch.randint(-127, 127, (K,), generator=g)
        x[r] = (k + 0.5) * s
        x[r, K // 2:] = torch.nextafter(x[r, K // 2:], torch.tensor(float("inf")))
        x[r, 0] = 127 * s
    return x.to(dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (16, 96), (17, 160), (33, 896), (124, 3584), (5, 18944),
                                 (1030, 224), (4100, 288)])
def test_quantize_is_exact(R, K, dtype):
    gu.note("quantize_int8 %dx%d %s" % (R, K, dtype))
    x = tricky_rows(gen(R + K), R, K, DTYPES[dtype])
    q, s = codes_of(x)
    codes, scales = q4.quantize_int8(x.cuda())
    torch.cuda.synchronize()
    assert torch.equal(scales.cpu().view(torch.int32), s.view(torch.int32))
    assert torch.equal(codes.cpu().double(), q)
    packed = q4.quantize_pack_int8(x.cuda())
    again = q4.pack_int8(codes, scales)
    torch.cuda.synchronize()
    want = tiles_of(codes.cpu())
    assert torch.equal(packed.codes.cpu(), want) and torch.equal(again.codes.cpu(), want)
    assert torch.equal(packed.scales.cpu().view(torch.int32), s.view(torch.int32))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_quantize_edges(dtype):
    """Zero rows, the smallest numbers, one value, the largest, infinities and NaN: each only in its own row."""
    t = DTYPES[dtype]
    fi = torch.finfo(t)
    x = torch.randn(12, 64, generator=gen(3)).to(t)
    x[0] = 0
    x[1] = -0.0
    x[2] = fi.smallest_normal * fi.eps  # the smallest subnormal
    x[3, :] = 0
    x[3, 5] = -1.5
    x[4] = fi.max
    x[4, ::2] = -fi.max
    x[5, 3] = float("inf")
    x[6, 63] = float("-inf")
    x[7, 0] = float("nan")
    x[8] = x[8] * fi.smallest_normal
    x[9] = x[9].sign() * fi.smallest_normal * fi.eps * torch.arange(1, 65)
    gu.note("quantize_int8 edges %s" % dtype)
    q, s = codes_of(x)
    codes, scales = q4.quantize_int8(x.cuda())
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(scales.cpu()), torch.isnan(s))
    assert torch.equal(torch.nan_to_num(scales.cpu()), torch.nan_to_num(s))
    assert torch.equal(codes.cpu().double(), q)
    # the rows' products: NaN where the scale is, exact elsewhere
    w = q4.quantize_pack_int8(torch.randn(40, 64, generator=gen(4)).cuda())
    qw, sw = q4.quantize_int8(torch.randn(40, 64, generator=gen(4)).cuda())
    if t != torch.float32:
        y = q4.linear_int8(x.cuda(), w)
        torch.cuda.synchronize()
        check_y(y, q, s, qw.cpu(), sw.cpu(), "edges")


SHAPES = [(1, 1, 32), (1, 17, 64), (2, 16, 160), (7, 100, 896), (16, 33, 128), (17, 257, 320), (40, 130, 96),
          (48, 512, 3584), (64, 31, 2080), (65, 129, 608), (124, 300, 8224), (129, 64, 32), (200, 1000, 1056),
          (333, 4863, 896), (513, 770, 352)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_linear(M, N, K, xt, yt):
    gu.note("linear_int8 M=%d N=%d K=%d %s -> %s" % (M, N, K, xt, yt))
    g = gen(M * 7 + N)
    x = tricky_rows(g, M, K, DTYPES[xt])
    qw = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8)
    sw = (torch.rand(N, generator=g) + 0.1) / 1024
    w = q4.pack_int8(qw.cuda(), sw.cuda())
    y = q4.linear_int8(x.cuda(), w, out_dtype=DTYPES[yt])
    shared = q4.linear_int8(q4.quantize_pack_int8(x.cuda()), w, out_dtype=DTYPES[yt])
    torch.cuda.synchronize()
    q, s = codes_of(x)
    check_y(y, q, s, qw, sw, "M=%d N=%d K=%d" % (M, N, K))
    assert torch.equal(y.view(torch.uint8), shared.view(torch.uint8))


@pytest.mark.parametrize("K", [131040])
def test_largest_sum(K):
    """Codes of -128 against -128 over the longest K: the 32-bit sum does not wrap."""
    gu.note("linear_int8 largest sum")
    M, N = 70, 40
    qx = torch.full((M, K), -128, dtype=torch.int8)
    qw = torch.full((N, K), -128, dtype=torch.int8)
    qx[1::2] = 127
    one = torch.ones(M).cuda()
    w = q4.pack_int8(qw.cuda(), one[:N].contiguous())
    for rows in (M, 3):
        y = q4.linear_int8(q4.pack_int8(qx[:rows].cuda(), one[:rows].contiguous()), w)
        torch.cuda.synchronize()
        check_y(y, qx[:rows], one[:rows].cpu(), qw, one[:N].cpu(), "largest sum")


@pytest.mark.parametrize("N,K", [(272, 3584), (3584, 896), (2048, 2048)])
def test_rows_do_not_depend_on_the_batch(N, K):
    """A row's bits are the same alone, in any batch, tile and split."""
    g = gen(11)
    x = tricky_rows(g, 700, K, torch.bfloat16).cuda()
    w = q4.quantize_pack_int8(torch.randn(N, K, generator=g).cuda())
    whole = q4.linear_int8(x, w)
    for M in (1, 5, 16, 17, 33, 64, 65, 124, 128, 300):
        gu.note("linear_int8 rows N=%d K=%d M=%d" % (N, K, M))
        part = q4.linear_int8(x[700 - M:].contiguous(), w)
        torch.cuda.synchronize()
        assert torch.equal(part.view(torch.int32), whole[700 - M:].view(torch.int32)), M


@pytest.mark.parametrize("M", [1, 40, 124, 300])
def test_unaligned_output_and_guards(M):
    """Outputs that start at an odd element, and what lies around them stays."""
    gu.note("linear_int8 guards M=%d" % M)
    g = gen(5)
    N, K = 132, 416
    x = torch.randn(M, K, generator=g).half().cuda()
    w = q4.quantize_pack_int8(torch.randn(N, K, generator=g).cuda())
    for dtype in DTYPES.values():
        ref = q4.linear_int8(x, w, out_dtype=dtype)
        room = torch.full((M * N + 64,), 7.0, dtype=dtype, device="cuda")
        out = room[31:31 + M * N].view(M, N)
        q4.linear_int8(x, w, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        assert (room[:31] == 7).all() and (room[31 + M * N:] == 7).all()


@pytest.mark.parametrize("M", [2, 100])
def test_workspace_rules(M):
    gu.note("linear_int8 workspace M=%d" % M)
    g = gen(6)
    N, K = 64, 2048
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    w = q4.quantize_pack_int8(torch.randn(N, K, generator=g).cuda())
    need = int(_lib.load().q4_int8_workspace_bytes(M, N, K, _lib.Q4_BF16))
    ref = q4.linear_int8(x, w)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    got = q4.linear_int8(x, w, workspace=ws[:need] if need else None)
    torch.cuda.synchronize()
    assert torch.equal(ref, got)
    assert (ws[need:] == 255).all()
    if need:
        with pytest.raises(q4.Q4Error):
            q4.linear_int8(x, w, workspace=ws[:need - 1])
        with pytest.raises(q4.Q4Error):
            q4.linear_int8(x, w, workspace=None)


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = q4.quantize_pack_int8(torch.zeros(8, 64, device="cuda"))
    with pytest.raises(TypeError):
        q4.linear_int8(x.float(), w)
    with pytest.raises(TypeError):
        q4.linear_int8(x, torch.zeros(8, 64, device="cuda"))
    with pytest.raises(ValueError):
        q4.linear_int8(x[:, :32].contiguous(), w)
    with pytest.raises(ValueError):
        q4.linear_int8(x[:, ::2], w)
    with pytest.raises(ValueError):
        q4.linear_int8(x.cpu(), w)
    with pytest.raises(ValueError):
        q4.linear_int8(x, w, out=torch.empty(4, 9, device="cuda"))
    with pytest.raises(TypeError):
        q4.linear_int8(x, w, out_dtype=torch.float64)
    with pytest.raises(q4.Q4Error):
        q4.linear_int8(x[:0], w)
    with pytest.raises(q4.Q4Error):  # two bytes off
        q4.linear_int8(torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 64), w)
    with pytest.raises(ValueError):
        q4.linear_int8(x, q4.Int8Matrix(w.codes[:1024], w.scales, 8, 64))
    with pytest.raises(ValueError):
        q4.pack_int8(torch.zeros(4, 48, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        q4.pack_int8(torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        q4.quantize_int8(torch.zeros(4, 64, dtype=torch.int8, device="cuda"))
    with pytest.raises(q4.Q4Error):
        q4.quantize_int8(torch.zeros(4, 48, device="cuda"))


@pytest.mark.parametrize("M", [1, 8, 124, 333])
def test_graph_replay_and_streams(M):
    """Captured once and replayed with new inputs, eager work between; and the
    same call on another stream."""
    gu.note("linear_int8 graph M=%d" % M)
    g = gen(9)
    N, K = 520, 1056
    w = q4.quantize_pack_int8(torch.randn(N, K, generator=g).cuda())
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    out = torch.empty(M, N, device="cuda")
    need = int(_lib.load().q4_int8_workspace_bytes(M, N, K, _lib.Q4_BF16))
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q4.linear_int8(x, w, out=out, workspace=ws if need else None)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, q4.linear_int8(x, w))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.linear_int8(x, w, out=out, workspace=ws if need else None)
    for i in range(4):
        x.copy_(torch.randn(M, K, generator=g).bfloat16())
        ref = q4.linear_int8(x, w)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), i
