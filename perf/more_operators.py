"""The cases by which the microscaled 4-bit quantizer and product and the norms
around a block are measured: ``listed`` and ``draw`` give cases, ``prepare``
makes what a program has in hand, ``run`` is one call (``own``: the library's
kernels; otherwise the plain form in elementary torch operations), ``exact``
the definition in 64 bits.

Operators:
  quant   rows in blocks of 32 to 4-bit floating point (1 sign, 2 exponent, 1
          mantissa bit; one power of two a block) in the packed form, and from
          there back to the values they stand for
  linear  y = x . w^T with x taken to that form in the call and w held in it
  norm    r = residual + scale gate post(y), h = pre(r): the norm after a
          block, its gate and residual scale, and the norm before the next one
  block   norm with h in the packed form, and the product of h with a weight
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # The hidden state of one decode row, quantized for several products: latency counts.
        {"name": "quant 1x3584", "op": "quant", "M": 1, "K": 3584, "x": "bf16"},
        # The widest weight of the 7B-shaped set, from its float32 master copy.
        {"name": "quant 18944x3584", "op": "quant", "M": 18944, "K": 3584, "x": "f32"},
        # One decode row through the square projection of the 7B-shaped set: latency counts.
        {"name": "linear 1x3584x3584", "op": "linear", "M": 1, "N": 3584, "K": 3584, "x": "bf16", "y": "f32"},
        # A full decode batch through the widest projection of that set: the weights' bytes.
        {"name": "linear 8x18944x3584", "op": "linear", "M": 8, "N": 18944, "K": 3584, "x": "bf16", "y": "bf16"},
        # The mixed batch of 120 prompt rows and 4 verify rows, long K.
        {"name": "linear 124x3584x18944", "op": "linear", "M": 124, "N": 3584, "K": 18944, "x": "bf16", "y": "f32"},
        # A ragged prompt chunk of the 0.5B-shaped set in fp16, odd sizes.
        {"name": "linear 333x4863x896", "op": "linear", "M": 333, "N": 4863, "K": 896, "x": "f16", "y": "f16"},
        # A long prompt through the widest projection: the matrix cores.
        {"name": "linear 4096x18944x3584", "op": "linear", "M": 4096, "N": 18944, "K": 3584, "x": "bf16", "y": "bf16"},
        # One decode row between two blocks of the 7B-shaped set, a norm on both sides: latency counts.
        {"name": "norm 1x3584", "op": "norm", "M": 1, "H": 3584, "y": "f32", "r": "bf16", "h": "bf16", "post": "rms",
         "pre": "rms", "gate": "none", "scale": 1.0},
        # A verify batch of the 0.5B-shaped set: layer norm, a learned gate for each channel, a residual scale.
        {"name": "norm 17x896", "op": "norm", "M": 17, "H": 896, "y": "f16", "r": "f32", "h": "f16", "post": "none",
         "pre": "layer", "gate": "channel", "scale": 0.22},
        # Rows of an odd width, a gate for each row (a shared expert's).
        {"name": "norm 333x4863", "op": "norm", "M": 333, "H": 4863, "y": "bf16", "r": "bf16", "h": "bf16",
         "post": "layer", "pre": "rms", "gate": "row", "scale": 0.5},
        # A long prompt with a gate for each value (computed from a condition): memory.
        {"name": "norm 4096x3584", "op": "norm", "M": 4096, "H": 3584, "y": "f32", "r": "bf16", "h": "bf16",
         "post": "rms", "pre": "rms", "gate": "full", "scale": 1.0},
        # The mixed batch from one block into the widest projection of the next.
        {"name": "block 124x18944x3584", "op": "block", "M": 124, "N": 18944, "H": 3584, "y": "f32", "r": "bf16",
         "post": "none", "pre": "rms", "gate": "none", "scale": 1.0},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "linear", "norm", "norm", "block"])
    any16, any32 = ["bf16", "f16"], ["bf16", "f16", "f32"]
    if op == "quant":
        K = 32 * _spread(rng, 8, 592)
        return {"op": op, "M": _spread(rng, 1, 18944 * 3584 // K), "K": K, "x": rng.choice(any32)}
    if op == "linear":
        N, K = _spread(rng, 200, 18944), 32 * _spread(rng, 8, 592)
        most = min(8192, 4096 * 18944 * 3584 // (N * K), 600_000_000 // (4 * N))
        return {"op": op, "M": _spread(rng, 1, max(1, most)), "N": N, "K": K, "x": rng.choice(any16),
                "y": rng.choice(any32)}
    norms, gates = ["none", "rms", "layer"], ["none", "channel", "row", "full"]
    case = {"op": op, "y": rng.choice(any32), "r": rng.choice(any32), "post": rng.choice(norms),
            "pre": rng.choice(norms[1:]), "gate": rng.choice(gates), "scale": rng.choice([1.0, 0.22])}
    if op == "norm":
        H = _spread(rng, 64, 8192)
        return {**case, "M": _spread(rng, 1, min(8192, 4096 * 3584 // H)), "H": H, "h": rng.choice(any16)}
    N, H = _spread(rng, 200, 18944), 32 * _spread(rng, 8, 256)
    return {**case, "M": _spread(rng, 1, 512), "N": N, "H": H}


# ------------------------------------------------------------------ inputs
def _device():
    return torch.device("cuda:0" if torch.cuda.is_available() else "cpu")


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device)


def _x(gen, M, K, dtype):
    """Hidden states: rows of different size, a few channels far larger than the others."""
    x = _rand(gen, M, K) * torch.exp(0.5 * _rand(gen, M, 1))
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=gen, device=gen.device)] *= 8
    return x.to(DTYPES[dtype])


def _code_tiles(codes):
    """4-bit codes [R, K] (one a byte) -> the packed tiles of 16 rows by 128 k: 16 bytes for each block of 32,
    blocks of the same k together, even k in the low half of a byte; zero past R and K."""
    R, K = codes.shape
    T, Q = -(-R // 16), -(-K // 128)
    p = torch.zeros((T * 16, Q * 128), dtype=torch.uint8, device=codes.device)
    p[:R, :K] = codes
    c = p.view(T, 16, Q, 4, 16, 2).permute(0, 2, 3, 1, 4, 5)
    return (c[..., 0] | (c[..., 1] << 4)).reshape(-1).contiguous()


def _scale_tiles(scales):
    """Scale bytes [R, K / 32] -> the packed tiles of 16 rows by 16 blocks: for a row and each of four
    neighbouring blocks, the bytes of that block in four steps of 128 k; zero past R and K."""
    R, B = scales.shape
    T, Q = -(-R // 16), -(-B // 16)
    p = torch.zeros((T * 16, Q * 16), dtype=torch.uint8, device=scales.device)
    p[:R, :B] = scales
    return p.view(T, 16, Q, 4, 4).permute(0, 2, 4, 1, 3).reshape(-1).contiguous()


def _weight(gen, N, K):
    """A weight in 4-bit blocks: codes [N, K] (one a byte), scale bytes [N, K / 32], and both packed."""
    values, e = _blocks(_rand(gen, N, K) / math.sqrt(K))
    a = values.abs()
    codes = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    codes = (codes + 8 * (values < 0)).to(torch.uint8).view(N, K)
    scales = (e + 127).to(torch.uint8).view(N, K // 32)
    return {"codes": codes, "bytes": scales, "packed": _code_tiles(codes), "tiles": _scale_tiles(scales)}


def _norm(gen, kind, H, dtype):
    if kind == "none":
        return None
    weight = (1 + 0.1 * _rand(gen, H)).to(dtype)
    return {"kind": kind, "weight": weight, "bias": (0.1 * _rand(gen, H)).to(dtype) if kind == "layer" else None}


def prepare(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    s = {"case": case}
    M = case["M"]
    if case["op"] in ("quant", "linear"):
        s["x"] = _x(gen, M, case["K"], case["x"])
        if case["op"] == "linear":
            s["w"] = _weight(gen, case["N"], case["K"])
        return s
    H = case["H"]
    # a projection's output, the residual stream it goes to, weights as a checkpoint holds them
    s["y"] = (_rand(gen, M, H) * torch.exp(0.5 * _rand(gen, M, 1))).to(DTYPES[case["y"]])
    s["residual"] = _x(gen, M, H, case["r"])
    s["post"] = _norm(gen, case["post"], H, torch.bfloat16)
    s["pre"] = _norm(gen, case["pre"], H, torch.bfloat16)
    shape = {"none": None, "channel": (H,), "row": (M, 1), "full": (M, H)}[case["gate"]]
    s["gate"] = None if shape is None else torch.sigmoid(_rand(gen, *shape)).to(torch.bfloat16)
    if case["op"] == "block":
        s["w"] = _weight(gen, case["N"], H)
    return s


# --------------------------------------------------------- the plain forms
def _blocks(x):
    """x [R, K] -> the 4-bit values (before the scale) and the exponents of its blocks of 32, [R, K / 32, 32]
    and [R, K / 32, 1]: the block's largest value lies in 4 .. 8 of its scale (what is over 6 becomes 6), values
    round half to even (in 64 bits: values next to a border)."""
    x = x.double().view(x.shape[0], -1, 32)
    e = torch.frexp(x.abs().amax(2, keepdim=True))[1] - 3
    e = torch.clamp(e, min=-127)
    x = torch.ldexp(x, -e)
    a = x.abs()
    a = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    return torch.copysign(torch.clamp(a, max=6), x), e


def _values(x):
    """x [R, K] -> what its 4-bit form stands for, in 64 bits."""
    v, e = _blocks(x)
    return torch.ldexp(v, e).view(x.shape)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _dense(w):
    codes, scales = w["codes"], w["bytes"]
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    v = table[codes.long()].view(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.to(torch.int32)[:, :, None] - 127).view(codes.shape)


def _plain_norm(v, n):
    if n is None:
        return v
    if n["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * n["weight"].float()
    return v if n["bias"] is None else v + n["bias"].float()


def _plain_block(s):
    """(r, h) in 32 bits"""
    t = s["case"]["scale"] * _plain_norm(s["y"].float(), s["post"])
    if s["gate"] is not None:
        t = s["gate"].float() * t
    r = s["residual"].float() + t
    return r, _plain_norm(r, s["pre"])


def _plain(state):
    case = state["case"]
    if case["op"] == "quant":
        return _values(state["x"]).to(DTYPES[case["x"]])
    if case["op"] == "linear":
        return (_values(state["x"]).float() @ _dense(state["w"]).T).to(DTYPES[case["y"]])
    r, h = _plain_block(state)
    out = {"r": r.to(DTYPES[case["r"]])}
    if case["op"] == "norm":
        return {**out, "h": h.to(DTYPES[case["h"]])}
    return {**out, "y": (_values(h).float() @ _dense(state["w"]).T).to(torch.bfloat16)}


def run(state):
    if not own:
        return _plain(state)
    import bit_quantized_matmul_q4_amd as q4

    case = state["case"]
    op = case["op"]
    if op == "quant":
        return q4.dequantize_mx4(q4.quantize_pack_mx4(state["x"]), DTYPES[case["x"]])
    if op in ("linear", "block"):
        w = q4.Mx4Matrix(state["w"]["packed"], state["w"]["tiles"], case["N"], case["K" if op == "linear" else "H"])
    if op == "linear":
        return q4.linear_mx4(state["x"], w, out_dtype=DTYPES[case["y"]])

    def norm(n):
        return None if n is None else q4.Norm(n["weight"], n["bias"], n["kind"], 1e-6)

    r, h = q4.block_norm(state["y"], state["residual"], post=norm(state["post"]), gate=state["gate"],
                         scale=case["scale"], pre=norm(state["pre"]),
                         out_dtype="mx4" if op == "block" else DTYPES[case["h"]])
    if op == "norm":
        return {"r": r, "h": h}
    return {"r": r, "y": q4.linear_mx4(h, w, out_dtype=torch.bfloat16)}


# ------------------------------------------------------------ what it needs
def work(case):
    M = case["M"]
    if case["op"] == "quant":
        return {"bytes": 2 * SIZE[case["x"]] * M * case["K"], "flops": 0}
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K * 17 / 32 + SIZE[case["y"]] * M * N, "flops": 2 * M * N * K}
    H = case["H"]
    n = (SIZE[case["y"]] + 2 * SIZE[case["r"]]) * M * H
    n += {"none": 0, "channel": 2 * H, "row": 2 * M, "full": 2 * M * H}[case["gate"]]
    n += sum({"none": 0, "rms": 2 * H, "layer": 4 * H}[case[k]] for k in ("post", "pre"))
    if case["op"] == "norm":
        return {"bytes": n + SIZE[case["h"]] * M * H, "flops": 12 * M * H}
    return {"bytes": n + case["N"] * H * 17 / 32 + 2 * M * case["N"], "flops": 2 * M * case["N"] * H}


# -------------------------------------------------- the definition, 64 bits
def _exact_values(x):
    """The 4-bit form's values by comparison with the borders between neighbours: a value on a border goes to the
    neighbour with an even code."""
    R, K = x.shape
    x = x.to(torch.float64).reshape(-1, 32)
    top = x.abs().max(dim=1).values
    scale = torch.ones_like(top)
    at = top > 0
    power = torch.floor(torch.log2(top[at]))
    power = torch.where(torch.exp2(power) > top[at], power - 1, power)  # (log2 next to a power of two)
    power = torch.where(torch.exp2(power + 1) <= top[at], power + 1, power)
    scale[at] = torch.exp2(torch.clamp(power - 2, min=-127.0))
    size = x.abs() / scale[:, None]
    value = torch.zeros_like(size)
    for low, high, up in ((0.0, 0.5, 0), (0.5, 1.0, 1), (1.0, 1.5, 0), (1.5, 2.0, 1), (2.0, 3.0, 0), (3.0, 4.0, 1),
                          (4.0, 6.0, 0)):
        border = (low + high) / 2
        value += (high - low) * ((size >= border) if up else (size > border))
    return (value * torch.sign(x) * scale[:, None]).reshape(R, K)


def _exact_product(x, w, N):
    """x [M, K] in 64 bits by the weight, some columns at a time."""
    out = torch.empty((x.shape[0], N), dtype=torch.float64, device=x.device)
    for n in range(0, N, 4096):
        c = w["codes"][n:n + 4096].to(torch.int64)
        size, sign = c & 7, 1.0 - 2.0 * (c >> 3).to(torch.float64)
        m = torch.where(size < 2, 0.5 * size, (1 + 0.5 * (size & 1)) * torch.exp2((size >> 1).to(torch.float64) - 1))
        power = torch.exp2(w["bytes"][n:n + 4096].to(torch.float64) - 127).repeat_interleave(32, dim=1)
        out[:, n:n + 4096] = torch.mm(x, (sign * m * power).t())
    return out


def _exact_norm(v, n):
    if n is None:
        return v
    if n["kind"] == "layer":
        variance, mean = torch.var_mean(v, dim=1, correction=0, keepdim=True)
        v = (v - mean) * torch.rsqrt(variance + 1e-6)
    else:
        v = v * torch.rsqrt(torch.mean(torch.square(v), dim=1, keepdim=True) + 1e-6)
    v = v * n["weight"].to(torch.float64)
    return v + n["bias"].to(torch.float64) if n["bias"] is not None else v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_values(s["x"])
    if case["op"] == "linear":
        return _exact_product(_exact_values(s["x"]), s["w"], case["N"])
    t = _exact_norm(s["y"].to(torch.float64), s["post"]) * case["scale"]
    if s["gate"] is not None:
        t = t * s["gate"].to(torch.float64)
    r = s["residual"].to(torch.float64) + t
    h = _exact_norm(r, s["pre"])
    if case["op"] == "norm":
        return {"r": r, "h": h}
    return {"r": r, "y": _exact_product(_exact_values(h), s["w"], case["N"])}
