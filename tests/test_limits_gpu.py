"""The 8-bit product, the router and the expert layer at the largest rows,
columns and lengths that the library takes: rows against the same rows in a
small call (bit for bit), and long sums against 64 bits."""
import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from tests import gpu_util as gu
from tests.test_int8_gpu import check_y, codes_of
from tests.test_moe_gpu import Layer, check_experts, check_route, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()
    yield
    torch.cuda.empty_cache()


def cuda_gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def same(a, b):
    return torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("M,N", [(1 << 24, 17), ((1 << 24) - 3, 65)])
def test_most_rows(M, N):
    gu.note("linear_int8 M=%d N=%d" % (M, N))
    K = 32
    x = torch.randn(M, K, device="cuda", generator=cuda_gen(1), dtype=torch.bfloat16)
    w = q4.quantize_pack_int8(torch.randn(N, K, device="cuda", generator=cuda_gen(2)))
    y = q4.linear_int8(x, w)
    for at in (0, M // 2 - 7, M - 40):
        part = q4.linear_int8(x[at:at + 40].contiguous(), w)
        torch.cuda.synchronize()
        assert same(part, y[at:at + 40]), at
    del x, y


@pytest.mark.parametrize("M", [1, 16, 40, 100, 200])
def test_most_columns(M):
    N, K = 1 << 24, 32
    gu.note("linear_int8 M=%d N=%d" % (M, N))
    x = torch.randn(M, K, device="cuda", generator=cuda_gen(3), dtype=torch.bfloat16)
    codes, scales = q4.quantize_int8(torch.randn(N, K, device="cuda", generator=cuda_gen(4)))
    y = q4.linear_int8(x, q4.pack_int8(codes, scales))
    for at in (0, N // 2 - 32, N - 64):
        part = q4.linear_int8(x, q4.pack_int8(codes[at:at + 64].contiguous(), scales[at:at + 64].contiguous()))
        torch.cuda.synchronize()
        assert same(part, y[:, at:at + 64].contiguous()), at
    del codes, y


@pytest.mark.parametrize("M", [1, 17, 70])
def test_longest_int8_rows(M):
    gu.note("linear_int8 M=%d K=131040" % M)
    N, K = 33, 131040
    g = gen(5)
    x = torch.randn(M, K, generator=g).half()
    qw = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8)
    sw = torch.rand(N, generator=g) + 0.5
    y = q4.linear_int8(x.cuda(), q4.pack_int8(qw.cuda(), sw.cuda()))
    torch.cuda.synchronize()
    check_y(y, *codes_of(x), qw, sw, "K=131040")


@pytest.mark.parametrize("M,E,K", [(1 << 20, 3, 64), ((1 << 20) - 5, 2, 288), (3, 5, 1 << 17), (40, 1024, 96)])
def test_route_limits(M, E, K):
    gu.note("moe_route M=%d E=%d K=%d" % (M, E, K))
    g = gen(6)
    x = torch.randn(M, K, generator=g).bfloat16()
    r = (torch.randn(E, K, generator=g) / K**0.5).bfloat16()
    check_route(x, r, torch.randn(E, generator=g) * 0.1, 2, True, "limits")


@pytest.mark.parametrize("H,I", [(1 << 17, 32), (32, 1 << 17)])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16])
def test_longest_expert_rows(H, I, xt):
    gu.note("moe_experts H=%d I=%d" % (H, I))
    layer = Layer(2, H, I, 7)
    g = gen(7)
    M = 6
    ids = torch.tensor([[0, 1], [1, -1], [1, 0], [0, 0], [-1, -1], [1, 2]]).int()
    check_experts(layer, torch.randn(M, H, generator=g).to(xt), ids, torch.rand(M, 2, generator=g), "longest")


def test_most_pairs_of_the_longest_h():
    """1024 (row, expert) pairs of the longest h: offsets up to 2^28 bytes."""
    gu.note("moe_experts 1024 pairs, I=131072")
    layer = Layer(1, 32, 1 << 17, 8)
    x = torch.randn(1024, 32, generator=gen(8)).bfloat16().cuda()
    ids, w = torch.zeros(1024, 1, dtype=torch.int32, device="cuda"), torch.ones(1024, 1, device="cuda")
    y = q4.moe_experts(x, ids, w, layer.w13, layer.w2)
    part = q4.moe_experts(x[1020:].contiguous(), ids[1020:], w[1020:], layer.w13, layer.w2)
    torch.cuda.synchronize()
    assert same(y[1020:], part)


def test_most_expert_rows():
    """As many rows as a call takes, in pieces: the last ones' bits, in the experts and the layer."""
    gu.note("moe M=2^20")
    M, H = 1 << 20, 32
    layer = Layer(3, H, 32, 9)
    x = torch.randn(M, H, device="cuda", generator=cuda_gen(9), dtype=torch.bfloat16)
    r = torch.randn(3, H, device="cuda", generator=cuda_gen(10), dtype=torch.bfloat16)
    y = q4.moe(x, r, layer.w13, layer.w2, 2)
    ids, w = q4.moe_route(x, r, 2)
    z = q4.moe_experts(x, ids, w, layer.w13, layer.w2)
    part = q4.moe(x[M - 50:].contiguous(), r, layer.w13, layer.w2, 2)
    torch.cuda.synchronize()
    assert same(y, z) and same(y[M - 50:], part)
