"""The whole expert layer in each of its forms, named by the launches they take
(tests/moe_forms.py; the rule itself is checked on the CPU): the bits of the
router and the experts called one after the other."""
import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from tests import gpu_util as gu
from tests.moe_forms import BY_ROWS, FUSED, SEPARATE
from tests.test_moe_gpu import DTYPES, Layer, check_route, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()


@pytest.mark.parametrize("M,E,H,I,topk", FUSED + SEPARATE + BY_ROWS)
@pytest.mark.parametrize("xt", ["bf16", "f16"])
def test_layer_is_route_and_experts(M, E, H, I, topk, xt):
    layer = Layer(E, H, I, M + E)
    g = gen(M + E)
    x = torch.randn(M, H, generator=g).to(DTYPES[xt]).cuda()
    r = (torch.randn(E, H, generator=g) / H**0.5).to(DTYPES[xt]).cuda()
    bias = torch.randn(E, generator=g).cuda()
    for renormalize in (True, False):
        gu.note("moe M=%d E=%d H=%d I=%d topk=%d %s %s" % (M, E, H, I, topk, xt, renormalize))
        ids, w = q4.moe_route(x, r, topk, bias, renormalize)
        ref = q4.moe_experts(x, ids, w, layer.w13, layer.w2)
        y = q4.moe(x, r, layer.w13, layer.w2, topk, bias, renormalize)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int32), ref.view(torch.int32))


@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("M,E,K", [(1030, 512, 320), (32760, 3, 288), (2049, 250, 832)])
def test_route_by_rows(M, E, K, xt, rt):
    """Against 64 bits, and a part of the rows by the form that splits the sums: the same bits."""
    gu.note("moe_route by rows M=%d E=%d K=%d %s %s" % (M, E, K, xt, rt))
    g = gen(M)
    x = torch.randn(M, K, generator=g).to(DTYPES[xt])
    r = (torch.randn(E, K, generator=g) / K**0.5).to(DTYPES[rt])
    bias = torch.randn(E, generator=g) * 0.1
    check_route(x, r, bias, 3, False, "by rows")
    ids, w = q4.moe_route(x.cuda(), r.cuda(), 3, bias.cuda())
    i, v = q4.moe_route(x[-77:].contiguous().cuda(), r.cuda(), 3, bias.cuda())
    torch.cuda.synchronize()
    assert torch.equal(i, ids[-77:]) and torch.equal(v.view(torch.int32), w[-77:].view(torch.int32))
