"""Where the expert layer's operands are held in fewer bits than binary32,
against plain 64-bit computations and the bounds of test_moe_gpu.py.

bfloat16 x is held as binary16 times powers of two: exact down to 2^-19 of the
largest of its block of 32, and off by at most 2^-27 of it below that, so such a
value moves a gate or up sum by at most |w| 2^-27 of its block's largest.  h
keeps 22 bits of the largest of its block of 32 down to the smallest normal
binary32 number."""
import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from bit_quantized_matmul_q4_amd import _lib
from tests import gpu_util as gu
from tests.test_moe_gpu import U, blocks_of, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()


class Codes:
    """Experts from given codes and scales: dense values in 64 bits, packed on demand."""

    def __init__(self, E, H, I, seed):
        g = gen(seed)
        self.E, self.H, self.I = E, H, I
        self.c13 = torch.randint(0, 16, (E * 2 * I, H), generator=g, dtype=torch.uint8)
        self.c2 = torch.randint(0, 16, (E * H, I), generator=g, dtype=torch.uint8)
        self.s13 = ((torch.rand(E * 2 * I, H // 32, generator=g) + 0.5) / (4.6 * H**0.5)).half()
        self.s2 = ((torch.rand(E * H, I // 32, generator=g) + 0.5) / (4.6 * I**0.5)).half()

    def done(self):
        E, H, I = self.E, self.H, self.I
        self.w13, self.w2 = q4.pack(self.c13.cuda(), self.s13.cuda()), q4.pack(self.c2.cuda(), self.s2.cuda())
        self.d13 = ((self.c13.double() - 8) * self.s13.double().repeat_interleave(32, 1)).view(E, 2 * I, H)
        self.d2 = ((self.c2.double() - 8) * self.s2.double().repeat_interleave(32, 1)).view(E, H, I)
        return self


def check(layer, x, e, what):
    """One expert a row, weight 1, with the bounds of test_moe_gpu.py and x's own."""
    M, I = x.shape[0], layer.I
    ids = torch.full((M, 1), e, dtype=torch.int32).cuda()
    y = q4.moe_experts(x.cuda(), ids, torch.ones(M, 1).cuda(), layer.w13, layer.w2)
    torch.cuda.synchronize()
    xd = x.double()
    held = torch.zeros_like(xd)
    if x.dtype == torch.bfloat16:
        top = xd.abs().view(M, -1, 32).amax(2).repeat_interleave(32, 1)
        held = torch.where(xd.abs() < 2.0**-19 * top, 2.0**-27 * top, held)
    w13, w2 = layer.d13[e], layer.d2[e]
    gu_ = xd @ w13.T
    d = (blocks_of(layer.H) * U) * (xd.abs() @ w13.abs().T) + held @ w13.abs().T
    g, u, dg, du = gu_[:, :I], gu_[:, I:], d[:, :I], d[:, I:]
    act = g * torch.sigmoid(g)
    h = act * u
    # silu's slope is at most 1.1, and at -10 and below at most (1 - g) exp(g)
    slope = torch.where(g + dg < -10, (1 - g + dg) * torch.exp(g + dg), torch.full_like(g, 1.1))
    dh = slope * dg * (u.abs() + du) + act.abs() * du + 8 * U * h.abs()
    dh = dh + 2.0**-22 * h.abs().view(M, -1, 32).amax(2).repeat_interleave(32, 1)
    ref = h @ w2.T
    tol = (dh @ w2.abs().T) * (1 + 1e-4) + (blocks_of(I) * U) * (h.abs() @ w2.abs().T) + 2 * U * ref.abs()
    tol = tol * (1 + 1e-3) + 2.0**-148 * I  # (a product below the smallest normal number: half its step each)
    off = (y.cpu().double() - ref).abs()
    assert torch.isfinite(ref).all()
    assert (off <= tol).all(), "%s: off by %.3g times the bound, %.3g of the largest output, rows %s" % (
        what, float((off / tol).max()), float(off.max() / ref.abs().max()),
        torch.nonzero((off > tol).any(1)).flatten().tolist()[:8])


OUTLIERS = [10, 12, 13, 14, 16, 20, 25, 31, 33, 38, 45, 60, 90, 120]


@pytest.mark.parametrize("how", ["code 8", "zero scale"])
@pytest.mark.parametrize("M", [1, 7, 9])
@pytest.mark.parametrize("H", [64, 288, 2080])
def test_outlier_without_weight(H, M, how):
    """A value far above the others of its row whose weight is zero: the sums are the other values'."""
    layer = Codes(2, H, 64, H)
    at = 37
    if how == "code 8":
        layer.c13[:, at] = 8
    else:
        layer.s13[:, at // 32] = 0
    layer.done()
    for up in OUTLIERS:
        gu.note("moe_experts H=%d M=%d outlier 2^%d, %s" % (H, M, up, how))
        x = torch.randn(M, H, generator=gen(up))
        x[:, at] = 2.0**up
        check(layer, x.bfloat16(), 1, "2^%d" % up)


@pytest.mark.parametrize("M", [1, 6, 16, 20])
def test_blocks_of_very_different_size(M):
    """Blocks of 32 values from 2^-60 to 2^60 in one row, the largest ones without weight."""
    gu.note("moe_experts blocks M=%d" % M)
    H = 1056
    layer = Codes(2, H, 96, M)
    size = torch.randint(-60, 61, (H // 32,), generator=gen(M)).float()
    layer.s13[:, size > 0] = 0
    layer.done()
    x = torch.randn(M, H, generator=gen(M + 1)) * (2.0**size).repeat_interleave(32)
    check(layer, x.bfloat16(), 0, "blocks")


@pytest.mark.parametrize("M,E,topk", [(5, 3, 2), (40, 2, 1), (64, 2, 2), (70, 40, 3)])
def test_wide_rows_do_not_change_the_others(M, E, topk):
    """Rows keep their bits beside rows that need powers of two for their blocks, in calls of the parts and the layer."""
    H, I = 416, 96
    layer = Codes(E, H, I, M)
    layer.s13[:, 3] = 0
    layer.done()
    g = gen(M)
    x = torch.randn(M, H, generator=g)
    r = (torch.randn(E, H, generator=g) / H**0.5).bfloat16().cuda()
    r[:, 96:128] = 0
    good = x.bfloat16().cuda()
    wide = x.clone()
    wide[::7, 100] = 2.0**50
    wide = wide.bfloat16().cuda()
    rest = [m for m in range(M) if m % 7]
    gu.note("moe wide rows M=%d E=%d" % (M, E))
    ids, w = q4.moe_route(good, r, topk)
    a = q4.moe_experts(good, ids, w, layer.w13, layer.w2)
    b = q4.moe_experts(wide, ids, w, layer.w13, layer.w2)
    c = q4.moe(good, r, layer.w13, layer.w2, topk)
    d = q4.moe(wide, r, layer.w13, layer.w2, topk)
    torch.cuda.synchronize()
    assert torch.equal(a[rest].view(torch.int32), b[rest].view(torch.int32))
    assert torch.equal(a.view(torch.int32), c.view(torch.int32)) and torch.equal(b.view(torch.int32), d.view(torch.int32))
    for m in range(0, M, 7):  # alone
        one = q4.moe(wide[m:m + 1].contiguous(), r, layer.w13, layer.w2, topk)
        torch.cuda.synchronize()
        assert torch.equal(one.view(torch.int32), b[m:m + 1].view(torch.int32)), m
    # the outlier meets no weight, so the outputs are those without it, but for 2^-27 of a block's largest a value:
    # a sum of 416 of them moves by about 2^-22 of its size
    assert ((b - a).abs() <= 2.0**-18 * a.abs().amax()).all()
@pytest.mark.parametrize("M", [1, 5, 12])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16])
def test_small_h(M, xt):
    """h down to the smallest normal numbers: outputs that are normal keep their bits."""
    layer = Codes(1, 96, 64, M)
    layer.s2[:] = ((torch.rand(96, 2, generator=gen(M + 7)) + 0.5) / 64).half()
    layer.s2[::3] *= 2.0**-6
    layer.s2[1::3] *= 2.0**10
    if xt == torch.float16:  # gate and up by the scales, down to 2^-24 each, and x to 2^-14: about 2^-70 at the least
        layer.s13[:] = 2.0**-22
    layer.done()
    for low in ((-10, -40, -52, -55, -57, -58, -60) if xt == torch.bfloat16 else (0, -7, -14)):
        gu.note("moe_experts small h M=%d 2^%d" % (M, low))
        x = torch.randn(M, 96, generator=gen(M)).sign() * 2.0**low
        check(layer, x.to(xt), 0, "x of 2^%d" % low)


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16])
def test_far_negative_gate(xt):
    """silu where exp(-gate) passes the largest binary32 number: gate exp(gate), still normal at -89, times a large up."""
    H, I = 64, 64
    layer = Codes(1, H, I, 5)
    layer.c13[:I, :32], layer.c13[:I, 32:] = 9, 8  # gate: the sum of the first 32 values
    layer.c13[I:, :32], layer.c13[I:, 32:] = 8, 9  # up: of the others
    layer.s13[:] = 1
    layer.done()
    gates = torch.tensor([-60.0, -79, -81, -86, -88, -89, -90, -91, -95, -100, -103, -120, -1000])
    for big in (1.0, 1000.0):
        gu.note("moe_experts far negative gates, up %g" % big)
        x = torch.full((len(gates), H), big)
        x[:, :32] = 0
        x[:, 3] = gates
        check(layer, x.to(xt), 0, "gates")




@pytest.mark.parametrize("M", [1, 6, 70])
def test_wide_rows_in_a_replayed_graph(M):
    """One captured layer over inputs with and without wide rows, in a workspace that starts as NaN, eager work between."""
    H, I, E, topk = 288, 64, 6, 3
    layer = Codes(E, H, I, M).done()
    g = gen(M)
    r = (torch.randn(E, H, generator=g) / H**0.5).bfloat16().cuda()
    x = torch.randn(M, H, generator=g).bfloat16().cuda()
    need = int(_lib.load().q4_moe_layer_workspace_bytes(M, E, H, I, topk))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty(M, H, device="cuda")
    gu.note("moe wide rows in a graph M=%d" % M)
    q4.moe(x, r, layer.w13, layer.w2, topk, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.moe(x, r, layer.w13, layer.w2, topk, out=out, workspace=ws)
    for i in range(6):
        new = torch.randn(M, H, generator=g)
        if i % 2:
            new[:: 1 + i % 3, 40 + i] = 2.0**(36 + i)
        x.copy_(new.bfloat16())
        eager = q4.moe(x, r, layer.w13, layer.w2, topk)
        torch.cuda.synchronize()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, eager), i


def same(a, b):
    return torch.equal(a.view(torch.int32), b.view(torch.int32))
