"""The norms around a block on the GPU against the formulas in 64 bits.

Tolerances count roundings of u = 2^-24.  A sum over a row passes through at
most 32 values in a thread, 6 levels of a wave and 16 waves: D = 54 additions,
so it is off by D u of its magnitudes.  A norm's root then carries D / 2 + 6
roundings (mean, eps, root, quotient, and the squares' own), a layer norm's
difference d from the mean is off by D u mean|d| + 3 u |d|, and weight and bias
add two more of the value: ``norm_error`` passes an error of its input on
through that.  An output rounds once more to its type: finfo(type).eps / 2 of
the value, and half its smallest number."""
import pytest
import torch

import bit_quantized_matmul_q4_amd as q4
from tests import gpu_util as gu
from tests import mx4_ref

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
D = 54


@pytest.fixture(scope="module", autouse=True)
def gpu():
    gu.require_gpu()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def norm64(v, n):
    if n is None:
        return v
    if n["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + n["eps"])
    if n["weight"] is not None:
        v = v * n["weight"].double()
    return v if n["bias"] is None else v + n["bias"].double()


def norm_error(v, e, n):
    """What norm64(v) may be off by where v is off by e."""
    if n is None:
        return e
    d = v
    if n["kind"] == "layer":
        d = v - v.mean(1, keepdim=True)
        e = e + e.mean(1, keepdim=True) + D * U * d.abs().mean(1, keepdim=True) + 3 * U * d.abs()
    root = torch.sqrt((d * d).mean(1, keepdim=True) + n["eps"])
    slip = torch.sqrt((e * e).mean(1, keepdim=True)) / root + (D / 2 + 6) * U
    out = (e + d.abs() * slip) / root
    if n["weight"] is not None:
        out = out * n["weight"].double().abs()
    return out + 2 * U * norm64(v, n).abs() + 2 * U * (d.abs() / root * (1 if n["weight"] is None else n["weight"].double().abs()))


def expected(y, res, post, gate, scale, pre):
    """(r, its error, h, its error) in 64 bits."""
    v = y.double()
    e = norm_error(v, torch.zeros_like(v), post)
    v = norm64(v, post)
    g = torch.tensor(scale, dtype=torch.float32).double() * (1 if gate is None else gate.double())
    r = g * v
    er = abs(g) * e + 2 * U * r.abs()
    if res is not None:
        r = r + res.double()
    er = er + U * r.abs()
    return r, er, norm64(r, pre), norm_error(r, er, pre)


def check(got, want, error, what):
    f = torch.finfo(got.dtype)
    got = got.cpu().double()
    bound = error * 1.01 + f.eps / 2 * (want.abs() + error) + f.smallest_normal * f.eps
    off = (got - want).abs() - bound
    assert (off <= 0).all(), "%s: %g over at %s" % (what, off.max(), divmod(int(off.argmax()), want.shape[1]))


def to_norm(n):
    if n is None:
        return None
    return q4.Norm(*(None if n[k] is None else n[k].to(gu.DEV) for k in ("weight", "bias")), n["kind"], n["eps"])


def dev(t):
    return None if t is None else t.to(gu.DEV)


def side(g, kind, H, dtype="bf16", weight=True, bias=False, eps=1e-6):
    if kind == "none":
        return None
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(DTYPES[dtype]) if weight else None
    b = (0.2 * torch.randn(H, generator=g)).to(DTYPES[dtype]) if bias else None
    return {"kind": kind, "weight": w, "bias": b, "eps": eps}


def gate_of(g, form, M, H, dtype="bf16"):
    shape = {"none": None, "channel": (H,), "row": (M, 1), "value": (M, H)}[form]
    return None if shape is None else torch.randn(*shape, generator=g).to(DTYPES[dtype])


def run(y, res, post, gate, scale, pre, **kw):
    return q4.block_norm(dev(y), dev(res), to_norm(post), dev(gate), scale, to_norm(pre), **kw)


def check_all(y, res, post, gate, scale, pre, h_dtype, what):
    gu.note(str(what))
    r, h = run(y, res, post, gate, scale, pre, out_dtype=DTYPES[h_dtype])
    want_r, er, want_h, eh = expected(y, res, post, gate, scale, pre)
    assert r.dtype == (y if res is None else res).dtype and h.dtype == DTYPES[h_dtype]
    check(r, want_r, er, ("r", what))
    check(h, want_h, eh, ("h", what))
    return r, h


WIDTHS = [1, 2, 3, 7, 8, 9, 31, 32, 63, 64, 65, 127, 255, 511, 512, 513, 520, 896, 1023, 1024, 1025, 1032, 2047, 2048,
          2049, 3583, 3584, 4095, 4096, 4097, 4863, 8191, 8192, 8193, 11008, 16383, 16384, 16385, 18944, 32767, 32768]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_widths(H, kind):
    g = gen(H)
    y = torch.randn(3, H, generator=g)
    res = 2 * torch.randn(3, H, generator=g).bfloat16()
    eps = 1e-6 if H > 1 else 0.1  # (a layer norm of one value divides by sqrt(eps))
    post = side(g, kind, H, bias=kind == "layer", eps=eps)
    check_all(y, res, post, None, 1.0, side(g, kind, H, "f32", eps=eps), "bf16", (H, kind))


@pytest.mark.parametrize("y_dtype", list(DTYPES))
@pytest.mark.parametrize("r_dtype", list(DTYPES))
@pytest.mark.parametrize("h_dtype", list(DTYPES))
@pytest.mark.parametrize("H", [200, 203, 3584])
def test_types(y_dtype, r_dtype, h_dtype, H):
    g = gen(H)
    y = torch.randn(5, H, generator=g).to(DTYPES[y_dtype])
    res = torch.randn(5, H, generator=g).to(DTYPES[r_dtype])
    check_all(y, res, side(g, "rms", H, y_dtype), gate_of(g, "channel", 5, H, h_dtype), 0.5,
              side(g, "layer", H, r_dtype, bias=True), h_dtype, (y_dtype, r_dtype, h_dtype))


@pytest.mark.parametrize("gate", ["none", "channel", "row", "value"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("H", [96, 4863, 9000])
def test_forms(gate, post, pre, H):
    g = gen(H + len(gate))
    M = 6
    y = torch.randn(M, H, generator=g)
    res = torch.randn(M, H, generator=g).bfloat16()
    for dtype in ("bf16", "f32"):
        check_all(y, res, side(g, post, H, bias=True), gate_of(g, gate, M, H, dtype), -0.22,
                  side(g, pre, H, weight=False, bias=True), "bf16", (gate, post, pre, H))
    check_all(y, None, side(g, post, H, weight=False), gate_of(g, gate, M, H, "f16"), 3.0, side(g, pre, H), "f32",
              ("no residual", gate, post, pre, H))


@pytest.mark.parametrize("H", [64, 896, 3584, 18944])
def test_rows_do_not_depend_on_the_batch(H):
    g = gen(H)
    y, res = torch.randn(300, H, generator=g), torch.randn(300, H, generator=g).bfloat16()
    post, pre = side(g, "layer", H, bias=True), side(g, "rms", H)
    gate = gate_of(g, "row", 300, H)
    r, h = run(y, res, post, gate, 1.0, pre)
    rm, hm = run(y, res, post, gate, 1.0, pre, out_dtype="mx4")
    assert torch.equal(rm, r)
    full = q4.dequantize_mx4(hm)
    for M, first in ((1, 0), (1, 299), (7, 100), (16, 284), (64, 31), (129, 0)):
        cut = slice(first, first + M)
        a, b = run(y[cut], res[cut], post, gate[cut], 1.0, pre)
        assert torch.equal(a, r[cut]) and torch.equal(b, h[cut])
        a, b = run(y[cut], res[cut], post, gate[cut], 1.0, pre, out_dtype="mx4")
        assert torch.equal(a, r[cut]) and torch.equal(q4.dequantize_mx4(b), full[cut])


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 40, 300])
@pytest.mark.parametrize("H", [32, 64, 96, 544, 896, 3584, 4096, 8224, 16416, 32768])
def test_packed_rows(M, H):
    """h in the packed form: the bytes of quantize_pack_mx4 on the float32 h, padding included."""
    gu.note("packed %dx%d" % (M, H))
    g = gen(M + H)
    y, res = torch.randn(M, H, generator=g), torch.randn(M, H, generator=g)
    pre = side(g, "rms", H)
    r, h = run(y, res, None, None, 1.0, pre, out_dtype=torch.float32)
    buf = q4.quantize_pack_mx4(torch.randn(M, H, generator=g).to(gu.DEV))  # (other bytes in place)
    buf.codes.fill_(0xA5)
    buf.scales.fill_(0xA5)
    r2, m = run(y, res, None, None, 1.0, pre, out=buf)
    assert m is buf and torch.equal(r2, r)
    codes, scales = mx4_ref.packed(*mx4_ref.quantize(h.cpu()))
    assert torch.equal(m.codes.cpu(), codes) and torch.equal(m.scales.cpu(), scales)


def test_packed_rows_not_finite():
    g = gen(1)
    y = torch.randn(20, 1056, generator=g)
    y[3, 7], y[4, 1055], y[6] = float("nan"), float("inf"), 0.0
    pre = side(g, "layer", 1056)
    r, h = run(y, None, None, None, 1.0, pre, out_dtype=torch.float32)
    _, m = run(y, None, None, None, 1.0, pre, out_dtype="mx4")
    codes, scales = mx4_ref.packed(*mx4_ref.quantize(h.cpu()))
    assert torch.equal(m.codes.cpu(), codes) and torch.equal(m.scales.cpu(), scales)
    bad = torch.isnan(q4.dequantize_mx4(m)).all(1).cpu()
    assert bad.nonzero().view(-1).tolist() == [3, 4]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [40, 1000, 3584])
def test_large_and_small_rows(kind, H):
    """Rows whose squares leave binary32, from the largest values to the smallest."""
    g = gen(H)
    base = torch.randn(12, H, generator=g)
    base = base / base.abs().max()
    size = torch.tensor([2.0 ** e for e in (127, 120, 100, 64, 40, 0, -20, -40, -60, -80, -100, -120)])
    y = (base.double() * size.double()[:, None] * 1.9).float()
    for eps in (0.0, 1e-30, 1e-6):
        n = side(g, kind, H, "f32", eps=eps)
        gu.note("%s %d eps %g" % (kind, H, eps))
        h = run(y, None, n, None, 1.0, None, out_dtype=torch.float32, r_out=False)[1]
        r, er, want, e = expected(y, None, n, None, 1.0, None)
        check(h, want, e, (kind, H, eps))


@pytest.mark.parametrize("H", [40, 1000])
def test_rows_far_from_zero(H):
    """A layer norm of values that differ little: the mean's own rounding does not reach the result."""
    g = gen(H)
    y = (1000 + torch.randn(8, H, generator=g)).float()
    check_all(y, None, None, None, 1.0, side(g, "layer", H, "f32"), "f32", H)
    y = torch.full((2, H), 3.25)
    h = run(y, None, None, None, 1.0, {"kind": "layer", "weight": None, "bias": None, "eps": 1e-6},
            out_dtype=torch.float32)[1]
    assert (h == 0).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [100, 3584])
def test_not_finite(kind, H):
    """Each row's infinities and NaN are its own, and what the formulas give."""
    g = gen(H)
    y = torch.randn(9, H, generator=g)
    y[1, 5], y[3, H - 1], y[5, 0] = float("nan"), float("inf"), float("-inf")
    y[7] = 0
    n = {"kind": kind, "weight": None, "bias": None, "eps": 0.0}
    h = run(y, None, None, None, 1.0, n, out_dtype=torch.float32)[1].cpu()
    want = norm64(y.double(), n)
    assert torch.equal(torch.isnan(h), torch.isnan(want))
    ok = [0, 2, 4, 6, 8]
    assert torch.isfinite(h[ok]).all()
    assert (h.nan_to_num() - want.float().nan_to_num()).abs().max() < 1e-4
    res = torch.zeros(9, H)
    res[2, 3] = float("inf")
    r = run(y, res, None, None, 1.0, None, out=False)[0].cpu()
    assert torch.equal(torch.isinf(r), torch.isinf(y + res)) and torch.equal(torch.isnan(r), torch.isnan(y))


def test_in_place_and_parts():
    g = gen(4)
    for H in (896, 4863, 18944):
        y, res = torch.randn(33, H, generator=g), torch.randn(33, H, generator=g).bfloat16()
        pre = side(g, "rms", H)
        r, h = run(y, res, None, None, 0.5, pre)
        stream = dev(res)
        r2, h2 = q4.block_norm(dev(y), stream, None, None, 0.5, to_norm(pre), r_out=stream)
        assert r2 is stream and torch.equal(r2, r) and torch.equal(h2, h)
        none, h3 = run(y, res, None, None, 0.5, pre, r_out=False)
        assert none is None and torch.equal(h3, h)
        r4, none = run(y, res, None, None, 0.5, pre, out=False)
        assert none is None and torch.equal(r4, r)


def test_unaligned_and_nothing_outside():
    g = gen(6)
    M, H = 7, 331
    y, res = torch.randn(M, H, generator=g).half(), torch.randn(M, H, generator=g).bfloat16()
    n = side(g, "rms", H, "bf16", bias=True)
    gate = gate_of(g, "value", M, H, "f16")
    want = run(y, res, n, gate, 1.0, n)
    size = M * H
    for off in (0, 1, 2, 5):
        def place(t, k):
            buf = torch.full((t.numel() + 16,), 3.0, dtype=t.dtype, device=gu.DEV)
            buf[off:off + t.numel()] = dev(t).reshape(-1)
            return buf, buf[off:off + t.numel()].view(t.shape)
        rb, r_out = place(torch.zeros(M, H, dtype=torch.bfloat16), off)
        hb, h_out = place(torch.zeros(M, H, dtype=torch.bfloat16), off)
        w = q4.Norm(place(n["weight"], off)[1], place(n["bias"], off)[1], "rms", 1e-6)
        r, h = q4.block_norm(place(y, off)[1], place(res, off)[1], w, place(gate, off)[1], 1.0, w, r_out=r_out,
                             out=h_out)
        assert torch.equal(r, want[0]) and torch.equal(h, want[1])
        for b in (rb, hb):
            assert (b[:off] == 3).all() and (b[off + size:] == 3).all()


def test_binding_refuses():
    y = torch.zeros(4, 64, device=gu.DEV)
    n = q4.Norm(torch.ones(64, device=gu.DEV))
    cases = [
        (ValueError, "residual must be", dict(residual=torch.zeros(4, 32, device=gu.DEV))),
        (ValueError, "residual is on|GPU tensor", dict(residual=torch.zeros(4, 64))),
        (TypeError, "dtype", dict(residual=torch.zeros(4, 64, device=gu.DEV, dtype=torch.float64))),
        (ValueError, "gate must be", dict(gate=torch.zeros(4, device=gu.DEV))),
        (ValueError, "gate must be", dict(gate=torch.zeros(1, 64, device=gu.DEV))),
        (TypeError, "gate must be", dict(gate=0.5)),
        (TypeError, "Norm", dict(pre=torch.ones(64, device=gu.DEV))),
        (ValueError, "weight must be", dict(pre=q4.Norm(torch.ones(63, device=gu.DEV)))),
        (TypeError, "one dtype", dict(pre=q4.Norm(n.weight, n.weight.half()))),
        (ValueError, "kind", dict(post=q4.Norm(n.weight, kind="batch"))),
        (TypeError, "out_dtype", dict(out_dtype=torch.float64)),
        (TypeError, "out_dtype", dict(out_dtype="int8")),
        (ValueError, "out must be", dict(out=torch.zeros(4, 65, device=gu.DEV))),
        (ValueError, "r_out must be", dict(r_out=torch.zeros(5, 64, device=gu.DEV))),
        (TypeError, "r_out has dtype", dict(residual=y, r_out=torch.zeros(4, 64, device=gu.DEV).half())),
        (ValueError, "stores", dict(r_out=False, out=False)),
        (q4.Q4Error, "shape", dict(pre=q4.Norm(n.weight, eps=-1.0))),
    ]
    for kind, text, kw in cases:
        with pytest.raises(kind, match=text):
            q4.block_norm(y, **kw)
    with pytest.raises(ValueError, match="bad shape"):
        q4.block_norm(torch.zeros(4, 40, device=gu.DEV), out_dtype="mx4")
    with pytest.raises(ValueError, match="contiguous"):
        q4.block_norm(torch.zeros(64, 4, device=gu.DEV).T)


def test_captured_and_another_stream():
    g = gen(9)
    H, M = 3584, 5
    pre = to_norm(side(g, "rms", H))
    w = q4.quantize_pack_mx4(torch.randn(300, H, generator=g).to(gu.DEV))
    y, res = torch.empty(M, H, device=gu.DEV), torch.zeros(M, H, device=gu.DEV, dtype=torch.bfloat16)
    y.copy_(torch.randn(M, H, generator=g))

    def step():
        r, h = q4.block_norm(y, res, None, None, 1.0, pre, out_dtype="mx4")
        return r, q4.linear_mx4(h, w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, z = step()
    for _ in range(4):
        y.copy_(torch.randn(M, H, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want_r, want_z = step()
        assert torch.equal(r, want_r) and torch.equal(z, want_z)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want_r) and torch.equal(got[1], want_z)


def test_a_block_of_a_model():
    """Norm, gate|up product, down product and the next norm in a row, as a decode step runs them, against the
    formulas on the same 4-bit weights: every rounding of an operand to 4 bits is the library's own (its packed rows
    are read back), so that each product is held to its own bound."""
    g = gen(12)
    M, H, I = 9, 896, 1376
    res = torch.randn(M, H, generator=g).bfloat16()
    n1, n2, post = side(g, "rms", H), side(g, "rms", H), side(g, "rms", H)
    wgu = q4.quantize_pack_mx4((torch.randn(2 * I, H, generator=g) / H ** 0.5).to(gu.DEV))
    wd = q4.quantize_pack_mx4((torch.randn(H, I, generator=g) / I ** 0.5).to(gu.DEV))
    zero = torch.zeros(M, H, device=gu.DEV)
    r0, x = q4.block_norm(zero, dev(res), None, None, 1.0, to_norm(n1), out_dtype="mx4")
    assert torch.equal(r0, dev(res))
    gu_ = q4.linear_mx4(x, wgu)
    a, b = (q4.dequantize_mx4(t).cpu().double() for t in (x, wgu))
    want, mag = mx4_ref.product(a, b)
    assert ((gu_.cpu().double() - want).abs() <= (7 * 2.0 ** -23 + 2.0 ** -24) * mag).all()
    h = (torch.nn.functional.silu(gu_[:, :I]) * gu_[:, I:]).bfloat16()
    y = q4.linear_mx4(h, wd)
    a, b = (q4.dequantize_mx4(t).cpu().double() for t in (q4.quantize_pack_mx4(h), wd))
    want, mag = mx4_ref.product(a, b)
    assert ((y.cpu().double() - want).abs() <= (11 * 2.0 ** -23 + 2.0 ** -24) * mag).all()
    stream = r0.clone()
    r, nxt = q4.block_norm(y, stream, to_norm(post), None, 0.5, to_norm(n2), r_out=stream)
    want_r, er, want_h, eh = expected(y.cpu(), res, post, None, 0.5, n2)
    check(r, want_r, er, "r")
    check(nxt, want_h, eh, "h")
    assert r is stream
