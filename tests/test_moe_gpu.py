"""The router and the expert layer on the GPU against plain 64-bit
computations.

Router: the choice is exact (64-bit logits); a weight is
exp(fl(l - top)) / sum, with u = 2^-24: the difference's rounding moves the
exponent by |l - top| u, the exponential and the division give 4 u together,
the sum as many as its terms and 6 joins, each term with its own.

Experts, by the order of the sums: a block's dot of 32 exact products is within
33 u of the sum of their magnitudes, a segment adds one rounding a block, the
tree log2 S <= 4, the block scale's product one: a product of length K is
within c(K) u A, A its sum of magnitudes.  That error goes through silu (slope
at most 1.1) into h, whose own arithmetic gives 8 u and whose storage 2^-22 of
its block's largest; the down product carries it and adds its own; the sum over
the experts adds one rounding for each."""
import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from bit_quantized_matmul_q4_amd import _lib
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

U = 2.0**-24
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------- router
def ref_route(x, router, bias, topk, renormalize):
    l = x.double() @ router.double().T
    if bias is not None:
        l = l + bias.double()
    key = torch.where(torch.isnan(l), torch.full_like(l, float("inf")), l)
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :topk]
    chosen = torch.gather(l, 1, ids)
    top = chosen[:, :1]
    over = chosen if renormalize else l
    e = torch.where(over == -float("inf"), torch.zeros_like(over), torch.exp(over - top))
    total = e.sum(1, keepdim=True)
    w = torch.where(chosen == -float("inf"), torch.zeros_like(chosen), torch.exp(chosen - top) / total)
    d = torch.where(over == -float("inf"), torch.zeros_like(over), top - over)
    spread = (torch.nan_to_num(d * e)).sum(1, keepdim=True) / total
    tol = w * U * ((top - chosen).nan_to_num(0, 0, 0) + spread + over.shape[1] / 64 + 6 + 2 * 4 + 2)
    ids = torch.where(chosen == -float("inf"), torch.full_like(ids, -1), ids)
    return ids, w, torch.nan_to_num(tol)  # (no expert left: 0 / 0, and a weight of exactly 0)


def check_route(x, router, bias, topk, renormalize, what):
    ids, w = q4.moe_route(x.cuda(), router.cuda(), topk, None if bias is None else bias.cuda(), renormalize)
    torch.cuda.synchronize()
    rid, rw, tol = ref_route(x, router, bias, topk, renormalize)
    assert torch.equal(ids.cpu().long(), rid), what
    w = w.cpu().double()
    ok = ((w - rw).abs() <= tol + 2.0**-149) | (torch.isnan(w) & torch.isnan(rw))
    assert ok.all(), "%s: weights %s against %s" % (what, w[~ok][:4], rw[~ok][:4])


@pytest.mark.parametrize("M,E,K,topk", [(1, 1, 32, 1), (1, 8, 64, 2), (2, 17, 96, 17), (3, 60, 896, 4),
                                        (16, 64, 2048, 8), (17, 127, 416, 6), (33, 128, 3584, 8), (5, 1024, 160, 32),
                                        (300, 40, 224, 3), (530, 512, 320, 4)])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32")])
def test_route(M, E, K, topk, xt, rt):
    gu.note("moe_route M=%d E=%d K=%d topk=%d %s %s" % (M, E, K, topk, xt, rt))
    g = gen(M + E)
    x = torch.randn(M, K, generator=g).to(DTYPES[xt])
    r = (torch.randn(E, K, generator=g) / K**0.5).to(DTYPES[rt])
    bias = torch.randn(E, generator=g) * 0.1
    check_route(x, r, None, topk, True, "no bias")
    check_route(x, r, bias, topk, False, "bias, softmax weights")


def test_route_ties_go_to_the_lowest_index():
    """Whole-number logits (exact in any order) with many equal ones."""
    gu.note("moe_route ties")
    g = gen(2)
    x = torch.randint(-2, 3, (40, 64), generator=g).bfloat16()
    r = torch.randint(-1, 2, (48, 64), generator=g).bfloat16()
    r[24:] = r[:24]
    r[5] = 0
    r[6] = 0
    for topk in (1, 7, 48):
        check_route(x, r, None, topk, True, "ties %d" % topk)
    check_route(torch.zeros(3, 64).bfloat16(), r, None, 9, True, "all equal")


def test_route_neighbours():
    """Logits that differ in the last places of 64 bits only: 32-bit sums would call them equal."""
    gu.note("moe_route neighbours")
    x = torch.zeros(1, 64)
    x[0, 0], x[0, 1] = 1.0, 2.0**-40
    r = torch.zeros(20, 64)
    r[:, 0] = 1024.0
    r[:, 1] = torch.arange(20) % 7
    check_route(x.bfloat16(), r, None, 6, True, "neighbours")


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_masked_and_not_finite(renormalize):
    gu.note("moe_route masks")
    g = gen(3)
    E, K = 20, 64
    x = torch.randn(6, K, generator=g).bfloat16()
    r = torch.randn(E, K, generator=g).bfloat16()
    inf = float("inf")
    bias = torch.zeros(E)
    bias[3:] = -inf  # three experts left
    check_route(x, r, bias, 5, renormalize, "three left")
    check_route(x, r, torch.full((E,), -inf), 4, renormalize, "none left")
    low = torch.zeros(E)
    low[2:] = torch.finfo(torch.float32).min  # lowest values are no mask: still chosen in order
    check_route(x, r, low, 4, renormalize, "lowest values")
    bad = r.clone()
    bad[7, 0] = float("nan")
    ids, w = q4.moe_route(x.cuda(), bad.cuda(), 3, None, renormalize)
    torch.cuda.synchronize()
    assert (ids[:, 0] == 7).all() and torch.isnan(w).all()
    one = x.clone()
    one[2, 5] = float("nan")  # a row's own: the others keep their bits
    ids, w = q4.moe_route(one.cuda(), r.cuda(), 3, None, renormalize)
    good, gw = q4.moe_route(x.cuda(), r.cuda(), 3, None, renormalize)
    torch.cuda.synchronize()
    rest = [0, 1, 3, 4, 5]
    assert torch.equal(ids[rest], good[rest]) and torch.equal(w[rest], gw[rest])
    assert torch.isnan(w[2]).all() and ((ids[2] >= 0) & (ids[2] < E)).all()


def test_route_rows_do_not_depend_on_the_form():
    """Enough tiles for the form that keeps a row's whole sum in a wave: the bits of the one that splits it."""
    gu.note("moe_route forms")
    g = gen(14)
    for t in (torch.bfloat16, torch.float32):
        x = torch.randn(530, 832, generator=g).bfloat16().cuda()
        r = (torch.randn(512, 832, generator=g) / 29).to(t).cuda()
        ids, w = q4.moe_route(x, r, 5, None, False)
        i, v = q4.moe_route(x[500:].contiguous(), r, 5, None, False)
        torch.cuda.synchronize()
        assert torch.equal(i, ids[500:]) and torch.equal(v.view(torch.int32), w[500:].view(torch.int32))


def test_route_rows_do_not_depend_on_the_batch():
    gu.note("moe_route rows")
    g = gen(4)
    x = torch.randn(90, 3584, generator=g).bfloat16().cuda()
    r = (torch.randn(72, 3584, generator=g) / 60).bfloat16().cuda()
    ids, w = q4.moe_route(x, r, 6)
    for M in (1, 2, 7, 16, 17, 64):
        i, v = q4.moe_route(x[90 - M:].contiguous(), r, 6)
        torch.cuda.synchronize()
        assert torch.equal(i, ids[90 - M:]) and torch.equal(v.view(torch.int32), w[90 - M:].view(torch.int32)), M


# --------------------------------------------------------------- experts
class Layer:
    """Random 4-bit experts: dense values in 64 bits and the packed weights."""

    def __init__(self, E, H, I, seed):
        g = gen(seed)
        self.E, self.H, self.I = E, H, I
        c13 = torch.randint(0, 16, (E * 2 * I, H), generator=g, dtype=torch.uint8)
        c2 = torch.randint(0, 16, (E * H, I), generator=g, dtype=torch.uint8)
        s13 = ((torch.rand(E * 2 * I, H // 32, generator=g) + 0.5) / (4.6 * H**0.5)).half()
        s2 = ((torch.rand(E * H, I // 32, generator=g) + 0.5) / (4.6 * I**0.5)).half()
        s13[::5, 0] = 0
        s2[::7, 0] = 6e-8  # subnormal
        self.w13, self.w2 = q4.pack(c13.cuda(), s13.cuda()), q4.pack(c2.cuda(), s2.cuda())
        self.d13 = ((c13.double() - 8) * s13.double().repeat_interleave(32, 1)).view(E, 2 * I, H)
        self.d2 = ((c2.double() - 8) * s2.double().repeat_interleave(32, 1)).view(E, H, I)


def blocks_of(K):
    """c(K): 33 for a block's dot and its scale, the longest segment's blocks, the tree."""
    G = -(-(K // 32) // 4)
    S = 1
    while 2 * S <= G and S < 16:
        S *= 2
    return 33 + 1 + 4 * -(-G // S) + 4


def ref_experts(layer, x, ids, weights):
    """y and the bound on its error, in 64 bits."""
    M, topk = ids.shape
    H, I = layer.H, layer.I
    y, tol = torch.zeros(M, H, dtype=torch.float64), torch.zeros(M, H, dtype=torch.float64)
    xd, wd = x.double(), weights.double()
    cu, cd = blocks_of(H) * U, blocks_of(I) * U
    for m in range(M):
        for j in range(topk):
            e = int(ids[m, j])
            if not 0 <= e < layer.E:
                continue
            gu_, au = layer.d13[e] @ xd[m], layer.d13[e].abs() @ xd[m].abs()
            g, u = gu_[:I], gu_[I:]
            act = g * torch.sigmoid(g)
            h = act * u
            dh = 1.1 * cu * au[:I] * (u.abs() + cu * au[I:]) + act.abs() * cu * au[I:] + 8 * U * h.abs()
            dh = dh + 2.0**-22 * h.abs().view(-1, 32).amax(1).repeat_interleave(32)
            t, at = layer.d2[e] @ h, layer.d2[e].abs() @ h.abs()
            dt = layer.d2[e].abs() @ dh * (1 + 1e-4) + cd * at
            y[m] += wd[m, j] * t
            tol[m] += wd[m, j].abs() * (dt + (topk + 1) * U * t.abs())
    return y, tol * (1 + 1e-3) + 1e-38


def check_experts(layer, x, ids, weights, what):
    y = q4.moe_experts(x.cuda(), ids.cuda(), weights.cuda(), layer.w13, layer.w2)
    torch.cuda.synchronize()
    ref, tol = ref_experts(layer, x, ids, weights)
    d = (y.cpu().double() - ref).abs()
    assert (d <= tol).all(), "%s: off by %.3g times the bound at %s" % (
        what, float((d / tol).max()), torch.nonzero(d > tol)[:3].tolist())
    return y


def choose(g, M, E, topk):
    return torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(M)]).int()


SHAPES = [(1, 1, 32, 32, 1), (1, 4, 64, 96, 2), (2, 3, 160, 32, 3), (3, 8, 896, 160, 4), (5, 6, 128, 1376, 2),
          (8, 16, 224, 544, 8), (9, 40, 512, 64, 3), (17, 7, 288, 96, 5), (30, 3, 96, 128, 2), (64, 12, 544, 288, 4),
          (4, 2, 3584, 2592, 2), (1, 2, 4256, 64, 1), (12, 2, 64, 4128, 1), (40, 1024, 32, 32, 20), (60, 70, 64, 32, 17),
          (33, 2, 2080, 160, 1), (100, 2, 96, 160, 2), (64, 3, 544, 96, 3), (70, 1, 160, 64, 1)]


@pytest.mark.parametrize("M,E,H,I,topk", SHAPES)
@pytest.mark.parametrize("xt", ["bf16", "f16"])
def test_experts(M, E, H, I, topk, xt):
    gu.note("moe_experts M=%d E=%d H=%d I=%d topk=%d %s" % (M, E, H, I, topk, xt))
    layer = Layer(E, H, I, M + H)
    g = gen(M)
    x = (torch.randn(M, H, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(DTYPES[xt])
    ids, w = choose(g, M, E, topk), torch.rand(M, topk, generator=g)
    check_experts(layer, x, ids, w, "M=%d" % M)


def test_experts_few_and_none():
    """Rows without an expert, ids outside the range, one expert twice, one expert for all rows."""
    gu.note("moe_experts ids")
    layer = Layer(6, 192, 96, 1)
    g = gen(1)
    M, topk = 20, 4
    x = torch.randn(M, 192, generator=g).bfloat16()
    w = torch.randn(M, topk, generator=g)
    ids = choose(g, M, 6, topk)
    ids[3] = -1
    ids[4] = torch.tensor([6, 1000000, -7, -(2**31)])
    ids[5] = torch.tensor([2, 2, 2, 2])
    ids[6] = torch.tensor([-1, 4, 9, 4])
    y = check_experts(layer, x, ids, w, "ids")
    assert (y[3] == 0).all() and (y[4] == 0).all()
    check_experts(layer, x, torch.full((M, topk), 5, dtype=torch.int32), w, "one expert")
    y = check_experts(layer, x, torch.full((M, topk), -1, dtype=torch.int32), w, "none")
    assert (y == 0).all()
    # more choices in a row than experts
    ids = torch.randint(-1, 7, (3, 50), generator=g).int()
    check_experts(layer, x[:3], ids, torch.randn(3, 50, generator=g), "fifty choices")


def test_experts_in_pieces():
    """More (row, expert) pairs than one launch takes, the last piece short."""
    gu.note("moe_experts pieces")
    layer = Layer(5, 64, 64, 2)
    g = gen(2)
    for M, topk in ((300, 4), (3, 900), (1025, 1)):
        x = torch.randn(M, 64, generator=g).half()
        ids = torch.randint(0, 5, (M, topk), generator=g).int()
        check_experts(layer, x, ids, torch.rand(M, topk, generator=g) / topk, "M=%d" % M)


@pytest.mark.parametrize("xt", ["bf16", "f16"])
def test_experts_range(xt):
    """Rows of very different size and values that span the type, each row with its own bound."""
    gu.note("moe_experts range %s" % xt)
    layer = Layer(3, 256, 128, 3)
    g = gen(3)
    M = 10
    x = torch.randn(M, 256, generator=g)
    if xt == "bf16":
        x = x * 2.0 ** (torch.arange(M, dtype=torch.float32)[:, None] * 4 - 24)
        x[2] = x[2] * 2.0 ** (-torch.randint(0, 60, (256,), generator=g).float())
        x[4, 17] = 1e6
    else:
        x = x * 2.0 ** (torch.arange(M, dtype=torch.float32)[:, None] - 14)
    x[5] = 0
    x = x.to(DTYPES[xt])
    check_experts(layer, x, choose(g, M, 3, 2), torch.rand(M, 2, generator=g), "range")


def test_experts_not_finite_stays_in_its_row():
    gu.note("moe_experts inf and nan")
    layer = Layer(4, 160, 64, 4)
    g = gen(4)
    for t in (torch.bfloat16, torch.float16):
        x = torch.randn(9, 160, generator=g).to(t)
        ids, w = choose(g, 9, 4, 2), torch.rand(9, 2, generator=g)
        good = q4.moe_experts(x.cuda(), ids.cuda(), w.cuda(), layer.w13, layer.w2)
        x[1, 3], x[4, 100], x[6, 0] = float("nan"), float("inf"), float("-inf")
        y = q4.moe_experts(x.cuda(), ids.cuda(), w.cuda(), layer.w13, layer.w2)
        torch.cuda.synchronize()
        rest = [0, 2, 3, 5, 7, 8]
        assert torch.equal(y[rest].view(torch.int32), good[rest].view(torch.int32))
        assert torch.isnan(y[1]).all()
        assert not torch.isfinite(y[4]).any() and not torch.isfinite(y[6]).any()


@pytest.mark.parametrize("H,I", [(2048, 768), (896, 1376)])
def test_rows_do_not_depend_on_the_batch(H, I):
    """The whole layer: a row's bits alone, and in batches of other rows that share or not its experts."""
    layer = Layer(8, H, I, 5)
    g = gen(5)
    x = torch.randn(70, H, generator=g).bfloat16().cuda()
    r = (torch.randn(8, H, generator=g) / H**0.5).bfloat16().cuda()
    whole = q4.moe(x, r, layer.w13, layer.w2, 3)
    for M in (1, 2, 4, 5, 8, 9, 16, 33, 64):
        gu.note("moe rows H=%d I=%d M=%d" % (H, I, M))
        part = q4.moe(x[70 - M:].contiguous(), r, layer.w13, layer.w2, 3)
        torch.cuda.synchronize()
        assert torch.equal(part.view(torch.int32), whole[70 - M:].view(torch.int32)), M


@pytest.mark.parametrize("M,E,H,I,topk,xt", [(1, 8, 96, 64, 2, "bf16"), (4, 128, 288, 32, 8, "f16"),
                                              (16, 64, 512, 96, 5, "bf16"), (17, 64, 512, 96, 5, "bf16"),
                                              (9, 120, 160, 32, 3, "bf16"), (3, 5, 4256, 32, 2, "bf16"),
                                              (300, 12, 64, 32, 6, "bf16"), (300, 12, 64, 32, 6, "f16"),
                                              (1024, 1, 64, 32, 1, "bf16"), (1000, 4, 64, 32, 1, "f16"),
                                              (1024, 256, 288, 32, 1, "bf16")])
@pytest.mark.parametrize("renormalize", [True, False])
def test_layer_is_route_and_experts(M, E, H, I, topk, xt, renormalize):
    """The whole layer in one call, in each of its forms: the bits of its two parts."""
    gu.note("moe M=%d E=%d H=%d I=%d topk=%d %s" % (M, E, H, I, topk, xt))
    layer = Layer(E, H, I, M + E)
    g = gen(M + E)
    x = torch.randn(M, H, generator=g).to(DTYPES[xt]).cuda()
    r = (torch.randn(E, H, generator=g) / H**0.5).cuda()
    bias = torch.randn(E, generator=g).cuda()
    bias[E // 2] = -float("inf")
    ids, w = q4.moe_route(x, r, topk, bias, renormalize)
    ref = q4.moe_experts(x, ids, w, layer.w13, layer.w2)
    y = q4.moe(x, r, layer.w13, layer.w2, topk, bias, renormalize)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int32), ref.view(torch.int32))
    none = q4.moe(x, r, layer.w13, layer.w2, topk, torch.full_like(bias, -float("inf")), renormalize)
    torch.cuda.synchronize()
    assert (none == 0).all()


def test_weights_from_concat():
    """The stacked weights by concat_n of separately packed experts: the same bits."""
    gu.note("moe concat_n")
    E, H, I = 3, 160, 96
    g = gen(6)
    parts13, parts2 = [], []
    for _ in range(E):
        parts13 += [q4.quantize_pack(torch.randn(I, H, generator=g).cuda()) for _ in range(2)]
        parts2.append(q4.quantize_pack(torch.randn(H, I, generator=g).cuda()))
    x = torch.randn(4, H, generator=g).half().cuda()
    ids = torch.tensor([[0, 1], [2, 0], [1, 2], [1, -1]]).int().cuda()
    w = torch.rand(4, 2, generator=g).cuda()
    y = q4.moe_experts(x, ids, w, q4.concat_n(parts13), q4.concat_n(parts2))
    # one expert by the 4-bit product itself (h in 64 bits between): near, by the products' own errors
    ref = torch.zeros(4, H, dtype=torch.float64)
    for m in range(4):
        for j in range(2):
            e = int(ids[m, j])
            if e >= 0:
                gg = q4.linear(x[m:m + 1], parts13[2 * e]).double()
                uu = q4.linear(x[m:m + 1], parts13[2 * e + 1]).double()
                h = (gg * torch.sigmoid(gg) * uu).half()
                scale = h.abs().max().double() * 2.0**-11 * I**0.5
                t = q4.linear(h, parts2[e]).double().cpu()[0]
                ref[m] += w[m, j].double().cpu() * t
                assert scale > 0
    torch.cuda.synchronize()
    rel = (y.cpu().double() - ref).norm() / ref.norm()
    assert rel < 2.0**-11  # h rounded to binary16 in the comparison: half a step of each value


def test_layer_together_graph_and_streams():
    """A decode step as a server runs it: an 8-bit projection of the attention's
    output, the router and experts on it, an 8-bit projection of the result --
    eager on another stream, then captured and replayed with new inputs and
    eager work between the replays."""
    E, H, I, topk = 16, 320, 224, 4
    layer = Layer(E, H, I, 7)
    g = gen(7)
    r = (torch.randn(E, H, generator=g) / H**0.5).bfloat16().cuda()
    wo = q4.quantize_pack_int8((torch.randn(H, 256, generator=g) / 16).cuda())
    wn = q4.quantize_pack_int8((torch.randn(500, H, generator=g) / 18).cuda())

    def step(a):
        x = q4.linear_int8(a, wo, out_dtype=torch.bfloat16)
        y = q4.moe(x, r, layer.w13, layer.w2, topk)
        return x, y, q4.linear_int8((x.float() + y).bfloat16(), wn)

    for M in (1, 6, 20):
        gu.note("decode step M=%d" % M)
        a = torch.randn(M, 256, generator=g).bfloat16().cuda()
        x, y, z = step(a)
        ids, w = q4.moe_route(x, r, topk)
        ref, tol = ref_experts(layer, x.cpu(), ids.cpu(), w.cpu())
        assert ((y.cpu().double() - ref).abs() <= tol).all()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step(a)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(other, (x, y, z)))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(a)
        for i in range(4):
            a.copy_(torch.randn(M, 256, generator=g).bfloat16())
            eager = [t.clone() for t in step(a)]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, eager)), i


def test_two_streams_at_once():
    """Two streams with calls of their own in flight together, and a third of both operators' inputs shared."""
    gu.note("two streams")
    E, H, I, topk = 24, 512, 160, 4
    layer = Layer(E, H, I, 10)
    g = gen(10)
    r = (torch.randn(E, H, generator=g) / H**0.5).bfloat16().cuda()
    w = q4.quantize_pack_int8((torch.randn(2000, H, generator=g) / 22).cuda())
    xs = [torch.randn(M, H, generator=g).bfloat16().cuda() for M in (3, 70)]
    ref = [(q4.moe(x, r, layer.w13, layer.w2, topk), q4.linear_int8(x, w)) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (s, x) in enumerate(zip(streams, xs)):
            with torch.cuda.stream(s):
                got[i].append((q4.moe(x, r, layer.w13, layer.w2, topk), q4.linear_int8(x, w)))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in got[i]:
            assert torch.equal(a, ref[i][0]) and torch.equal(b, ref[i][1])


def test_workspace_and_output_guards():
    gu.note("moe guards")
    layer = Layer(4, 96, 64, 8)
    g = gen(8)
    M, topk = 7, 2
    x = torch.randn(M, 96, generator=g).bfloat16().cuda()
    ids, w = choose(g, M, 4, topk).cuda(), torch.rand(M, topk, generator=g).cuda()
    ref = q4.moe_experts(x, ids, w, layer.w13, layer.w2)
    need = int(_lib.load().q4_moe_experts_workspace_bytes(M, 96, 64, topk))
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN in every unwritten place
    room = torch.full((M * 96 + 50,), 7.0, device="cuda")
    out = room[25:25 + M * 96].view(M, 96)
    q4.moe_experts(x, ids, w, layer.w13, layer.w2, out=out, workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    assert (ws[need:] == 255).all() and (room[:25] == 7).all() and (room[25 + M * 96:] == 7).all()
    with pytest.raises(q4.Q4Error):
        q4.moe_experts(x, ids, w, layer.w13, layer.w2, workspace=ws[:need - 1])
    with pytest.raises(q4.Q4Error):
        q4.moe_experts(x, ids, w, layer.w13, layer.w2, workspace=None)


def test_refusals():
    layer = Layer(4, 96, 64, 9)
    x = torch.zeros(3, 96, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros(4, 96, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(3, 2, device="cuda")
    with pytest.raises(TypeError):
        q4.moe_route(x.float(), r, 2)
    with pytest.raises(TypeError):
        q4.moe_route(x, r.half(), 2)
    with pytest.raises(ValueError):
        q4.moe_route(x, r[:, :64].contiguous(), 2)
    for topk in (0, 5):
        with pytest.raises(ValueError):
            q4.moe_route(x, r, topk)
    with pytest.raises(ValueError):
        q4.moe_route(x, r, 2, bias=torch.zeros(5, device="cuda"))
    with pytest.raises(ValueError):
        q4.moe_route(x, r.cpu(), 2)
    with pytest.raises(q4.Q4Error):
        q4.moe_route(x[:0], r, 2)
    off = torch.zeros(3 * 96 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, 96)  # two bytes off
    with pytest.raises(q4.Q4Error):
        q4.moe_route(off, r, 2)
    with pytest.raises(q4.Q4Error):
        q4.moe(off, r, layer.w13, layer.w2, 2)
    with pytest.raises(TypeError):
        q4.moe_experts(x, ids.long(), w, layer.w13, layer.w2)
    with pytest.raises(ValueError):
        q4.moe_experts(x, ids[:2], w, layer.w13, layer.w2)
    with pytest.raises(ValueError):
        q4.moe_experts(x, ids, w[:, :1].contiguous(), layer.w13, layer.w2)
    with pytest.raises(ValueError):
        q4.moe_experts(x, ids, w, layer.w2, layer.w13)
    with pytest.raises(TypeError):
        q4.moe_experts(x, ids, w, layer.d13, layer.w2)
    with pytest.raises(ValueError):
        q4.moe(x, r[:3], layer.w13, layer.w2, 2)
    with pytest.raises(ValueError):
        q4.moe(x, r, layer.w13, layer.w2, 5)
    with pytest.raises(ValueError):
        q4.moe_experts(x[:, :64].contiguous(), ids, w, layer.w13, layer.w2)
    with pytest.raises(q4.Q4Error):
        q4.moe_experts(x[:0], ids[:0], w[:0], layer.w13, layer.w2)
