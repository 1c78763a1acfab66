"""Every kernel of the 8-bit product on the GPU, at shapes named by the kernel
they take (tests/int8_forms.py; the rule itself is checked on the CPU), with the
bounds of test_int8_gpu.py."""
import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from tests import gpu_util as gu
from tests.int8_forms import FORMS, form_of
from tests.test_int8_gpu import DTYPES, check_y, codes_of, gen, tiles_of, tricky_rows

pytestmark = pytest.mark.gpu

CASES = [(form, shape) for form, shapes in FORMS.items() for shape in shapes]
IDS = ["%s-%dx%dx%d" % (form, *shape) for form, shape in CASES]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()


@pytest.mark.parametrize("form,shape", CASES, ids=IDS)
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
def test_form(form, shape, xt, yt):
    """Against the exact product; packed x gives the same bits."""
    M, N, K = shape
    assert form_of(True, M, N, K)[0] == form
    gu.note("linear_int8 %s M=%d N=%d K=%d %s -> %s" % (form, M, N, K, xt, yt))
    g = gen(M * 3 + N)
    x = tricky_rows(g, M, K, DTYPES[xt])
    qw = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8)
    sw = (torch.rand(N, generator=g) + 0.1) / 1024
    w = q4.pack_int8(qw.cuda(), sw.cuda())
    y = q4.linear_int8(x.cuda(), w, out_dtype=DTYPES[yt])
    shared = q4.linear_int8(q4.quantize_pack_int8(x.cuda()), w, out_dtype=DTYPES[yt])
    torch.cuda.synchronize()
    q, s = codes_of(x)
    check_y(y, q, s, qw, sw, "%s M=%d N=%d K=%d" % (form, M, N, K))
    assert torch.equal(y.view(torch.uint8), shared.view(torch.uint8))


@pytest.mark.parametrize("form,shape", [c for c in CASES if c[1][0] > 64], ids=[i for i, c in zip(IDS, CASES) if c[1][0] > 64])
def test_rows_have_the_bits_of_the_smaller_forms(form, shape):
    """Rows of a large batch against the same rows through the few-row kernels and the smallest tiles."""
    M, N, K = shape
    g = gen(M + K)
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    w = q4.quantize_pack_int8(torch.randn(N, K, generator=g).cuda())
    whole = q4.linear_int8(x, w)
    for rows in (1, 5, 64, 65, 100):
        if rows >= M:
            continue
        for at in (0, M // 2, M - rows):
            gu.note("linear_int8 %s rows %d at %d of M=%d N=%d K=%d: %s" % (form, rows, at, M, N, K,
                                                                           form_of(True, rows, N, K)[0]))
            part = q4.linear_int8(x[at:at + rows].contiguous(), w)
            torch.cuda.synchronize()
            assert torch.equal(part.view(torch.int32), whole[at:at + rows].view(torch.int32)), (rows, at)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("R,K", [(2050, 8480), (2051, 4128), (3, 33024), (1, 131040)])
def test_quantizers_reload_what_they_do_not_hold(R, K, dtype):
    """Rows longer than the pieces that a lane keeps in registers, in both quantizers."""
    gu.note("quantize_int8 %dx%d %s" % (R, K, dtype))
    x = tricky_rows(gen(R + K), R, K, DTYPES[dtype])
    q, s = codes_of(x)
    codes, scales = q4.quantize_int8(x.cuda())
    packed = q4.quantize_pack_int8(x.cuda())
    torch.cuda.synchronize()
    assert torch.equal(scales.cpu().view(torch.int32), s.view(torch.int32))
    assert torch.equal(codes.cpu(), q.to(torch.int8))
    assert torch.equal(packed.codes.cpu(), tiles_of(codes.cpu()))
    assert torch.equal(packed.scales.cpu().view(torch.int32), s.view(torch.int32))
