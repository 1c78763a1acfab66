"""The cases by which the 8-bit product, the router and the expert layer are
measured: ``listed`` and ``draw`` give cases, ``prepare`` makes what a program
has in hand, ``run`` is one call (``own``: the library's kernels; otherwise
the plain form in elementary torch operations), ``exact`` the definition in
64 bits.

Operators:
  linear  y[m, n] = (sum_k qx[m, k] qw[n, k]) sx[m] sw[n] with qx, sx made
          from x in the call (a scale for each row), int8 codes
  route   the topk largest of softmax(x . router^T + bias), renormalised
  moe     the whole expert layer: the router, then for each chosen expert
          silu(gate) * up and the down product on 4-bit weights in blocks of
          32, summed with the router's weights
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
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
        # The router of one decode row, and of a mixed batch (a bias on the logits, odd number of experts).
        {"name": "route 1x64x2048", "op": "route", "M": 1, "E": 64, "H": 2048, "k": 8, "x": "bf16", "r": "bf16",
         "bias": False},
        {"name": "route 201x127x3584", "op": "route", "M": 201, "E": 127, "H": 3584, "k": 6, "x": "bf16", "r": "f32",
         "bias": True},
        # One decode row over few large experts.
        {"name": "moe 1 8x3584x2560", "op": "moe", "M": 1, "E": 8, "H": 3584, "I": 2560, "k": 2, "x": "bf16"},
        # One decode row over many small experts: the smallest layer call.
        {"name": "moe 1 64x2048x1024", "op": "moe", "M": 1, "E": 64, "H": 2048, "I": 1024, "k": 8, "x": "bf16"},
        # A decode batch: most experts see a row or none.
        {"name": "moe 8 128x2048x768", "op": "moe", "M": 8, "E": 128, "H": 2048, "I": 768, "k": 8, "x": "bf16"},
        # Odd sizes in fp16 (0.5B-shaped rows, quads that end short).
        {"name": "moe 17 60x896x1376", "op": "moe", "M": 17, "E": 60, "H": 896, "I": 1376, "k": 4, "x": "f16"},
        # A full batch: every expert is read, several rows each.
        {"name": "moe 64 64x3584x1792", "op": "moe", "M": 64, "E": 64, "H": 3584, "I": 1792, "k": 6, "x": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "route", "moe", "moe", "moe"])
    if op == "linear":
        N, K = _spread(rng, 200, 18944), 32 * _spread(rng, 8, 592)
        most = min(8192, 4096 * 18944 * 3584 // (N * K), 600_000_000 // (4 * N))
        return {"op": op, "M": _spread(rng, 1, max(1, most)), "N": N, "K": K, "x": rng.choice(["bf16", "f16"]),
                "y": rng.choice(["f32", "bf16", "f16"])}
    if op == "route":
        return {"op": op, "M": _spread(rng, 1, 256), "E": rng.randint(8, 128), "H": 32 * _spread(rng, 8, 112),
                "k": rng.randint(1, 8), "x": rng.choice(["bf16", "f16"]), "r": rng.choice(["x", "f32"]),
                "bias": rng.random() < 0.5}
    E, H = _spread(rng, 8, 128), 32 * _spread(rng, 16, 112)
    most = min(80, 64 * 3584 * 1792 // (32 * E * H))
    return {"op": op, "M": _spread(rng, 1, 64), "E": E, "H": H, "I": 32 * _spread(rng, 8, max(8, most)),
            "k": rng.randint(1, 8), "x": rng.choice(["bf16", "f16"])}


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


def _int8_tiles(codes):
    """int8 codes [R, K] -> the packed tiles of 16 rows by 64 k in lane order, K padded to 128."""
    R, K = codes.shape
    T, Q = -(-R // 16), 2 * -(-K // 128)
    p = torch.zeros((T * 16, Q * 64), dtype=torch.int8, device=codes.device)
    p[:R, :K] = codes
    return p.view(T, 16, Q, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1).contiguous()


def _q4_tiles(codes, scales):
    """4-bit codes [N, K] (one a byte) and fp16 scales [N, K / 32] -> the packed tiles of 16 rows by 128 k
    (N a multiple of 16; a short last tile is zero past K)."""
    N, K = codes.shape
    T, Q = N // 16, -(-K // 128)
    if K % 128:
        more = Q * 128 - K
        codes = torch.nn.functional.pad(codes, (0, more))
        scales = torch.nn.functional.pad(scales, (0, more // 32))
    c = codes.view(T, 16, Q, 4, 4, 8).permute(0, 2, 4, 1, 3, 5)  # tile, quad, k group, row, block, k
    b = torch.stack([c[..., lo] | (c[..., lo + 2] << 4) for lo in (0, 4, 1, 5)], dim=-1)
    return b.reshape(-1).contiguous(), scales.view(T, 16, Q, 4).permute(0, 2, 1, 3).reshape(-1).contiguous()


def _q4_weight(gen, N, K):
    """A random weight in 4-bit blocks: codes [N, K], scales [N, K / 32], and both packed."""
    codes = torch.randint(0, 16, (N, K), generator=gen, device=gen.device, dtype=torch.uint8)
    scales = ((0.5 + torch.rand(N, K // 32, generator=gen, device=gen.device)) / (4.6 * math.sqrt(K))).half()
    return codes, scales, *_q4_tiles(codes, scales)


def prepare(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        w = torch.clamp(torch.round(_rand(gen, N, K) * 32), -127, 127).to(torch.int8)
        scales = (0.5 + torch.rand(N, generator=gen, device=gen.device)) / (32 * math.sqrt(K))
        return {"case": case, "x": _x(gen, M, K, case["x"]), "w": w, "scales": scales, "packed": _int8_tiles(w)}
    M, E, H = case["M"], case["E"], case["H"]
    s = {"case": case, "x": _x(gen, M, H, case["x"]), "bias": None}
    router = _rand(gen, E, H) / math.sqrt(H)
    if case["op"] == "route":
        s["router"] = router.to(DTYPES[case["x"] if case["r"] == "x" else case["r"]])
        if case["bias"]:
            s["bias"] = 0.1 * _rand(gen, E)
        return s
    s["router"] = router.to(DTYPES[case["x"]])
    s["w13"] = _q4_weight(gen, E * 2 * case["I"], H)  # each expert's gate rows, then its up rows
    s["w2"] = _q4_weight(gen, E * H, case["I"])
    return s


# --------------------------------------------------------- the plain forms
def _row_codes(x):
    """x [M, K] -> whole numbers -127..127 and the scale of each row: s = max|x| / 127 rounded to 32
    bits, the codes rounded half to even on the quotient (in 64 bits: values next to a border)."""
    s = (x.double().abs().amax(1, keepdim=True) / 127).float()
    return torch.round(x.double() / s.double()).clamp(-127, 127).float(), s


def _linear(s):
    case = s["case"]
    q, sx = _row_codes(s["x"])
    y = (q @ s["w"].float().T) * sx * s["scales"]
    return y.to(DTYPES[case["y"]])


def _route(x, router, bias, k):
    # 64 bits: the choice compares neighbouring values
    logits = x.double() @ router.double().T
    if bias is not None:
        logits = logits + bias.double()
    p, ids = torch.sort(torch.softmax(logits, dim=1), dim=1, descending=True, stable=True)
    p = p[:, :k]
    return ids[:, :k].to(torch.int32), (p / p.sum(1, keepdim=True)).float()


def _dense(w):
    codes, scales = w[0], w[1]
    N, K = codes.shape
    return ((codes.float() - 8).view(N, K // 32, 32) * scales.float()[:, :, None]).view(N, K)


def _moe(s):
    case = s["case"]
    M, E, H, I, k = case["M"], case["E"], case["H"], case["I"], case["k"]
    ids, weights = _route(s["x"], s["router"], None, k)
    gu = (_dense(s["w13"]) @ s["x"].float().T).view(E, 2, I, M)
    h = gu[:, 0] / (1 + torch.exp(-gu[:, 0])) * gu[:, 1]
    t = torch.bmm(_dense(s["w2"]).view(E, H, I), h)  # every expert on every row: [E, H, M]
    chosen = t.permute(2, 0, 1)[torch.arange(M, device=t.device)[:, None], ids.long()]
    return (chosen * weights[:, :, None]).sum(1)


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "linear":
            return _linear(state)
        if op == "route":
            ids, weights = _route(state["x"], state["router"], state["bias"], case["k"])
            return {"ids": ids, "weights": weights}
        return _moe(state)
    import bit_quantized_matmul_q4_amd as q4

    if op == "linear":
        w = q4.Int8Matrix(state["packed"], state["scales"], case["N"], case["K"])
        return q4.linear_int8(state["x"], w, out_dtype=DTYPES[case["y"]])
    if op == "route":
        ids, weights = q4.moe_route(state["x"], state["router"], case["k"], bias=state["bias"])
        return {"ids": ids, "weights": weights}
    E, H, I = case["E"], case["H"], case["I"]
    w13 = q4.Q4Weight(state["w13"][2], state["w13"][3], E * 2 * I, H)
    w2 = q4.Q4Weight(state["w2"][2], state["w2"][3], E * H, I)
    return q4.moe(state["x"], state["router"], w13, w2, case["k"])


# ------------------------------------------------------------ what it needs
def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    M = case["M"]
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * N + size[case["y"]] * M * N, "flops": 2 * M * N * K}
    E, H, k = case["E"], case["H"], case["k"]
    if case["op"] == "route":
        r = size[case["x"] if case["r"] == "x" else case["r"]]
        return {"bytes": 2 * M * H + r * E * H + 8 * M * min(k, E), "flops": 2 * M * E * H}
    read = E * (1 - (1 - min(k, E) / E) ** M)  # the experts that M rows with k random choices each are expected to read
    weights = 3 * H * case["I"]
    return {"bytes": read * weights * 0.5625 + 2 * E * H + 2 * M * H + 4 * M * H,
            "flops": 2 * M * k * weights + 2 * M * E * H}


# -------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].to(torch.float64)
    if case["op"] == "linear":
        top = x.abs().max(dim=1).values / 127
        sx = top.to(torch.float32).to(torch.float64)
        codes = torch.round(x / sx[:, None])
        codes = torch.minimum(torch.maximum(codes, codes.new_tensor(-127.0)), codes.new_tensor(127.0))
        total = torch.mm(codes, s["w"].to(torch.float64).t())
        return total * (sx[:, None] * s["scales"].to(torch.float64)[None, :])
    logits = torch.mm(x, s["router"].to(torch.float64).t())
    if s["bias"] is not None:
        logits += s["bias"].to(torch.float64)
    e = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    prob = e / e.sum(dim=1, keepdim=True)
    M, k = case["M"], case["k"]
    ids = torch.empty((M, k), dtype=torch.int64, device=x.device)
    weights = torch.empty((M, k), dtype=torch.float64, device=x.device)
    left = prob.clone()
    for j in range(k):  # the largest left, the lowest index among equals
        best = left.max(dim=1, keepdim=True).values
        at = torch.argmax((left == best).to(torch.int8), dim=1, keepdim=True)
        ids[:, j:j + 1], weights[:, j:j + 1] = at, best
        left.scatter_(1, at, -1.0)
    weights /= weights.sum(dim=1, keepdim=True)
    if case["op"] == "route":
        return {"ids": ids, "weights": weights}
    E, H, I = case["E"], case["H"], case["I"]
    y = torch.zeros((M, H), dtype=torch.float64, device=x.device)

    def dense(w, expert, rows):
        c, d = w[0][expert * rows:(expert + 1) * rows], w[1][expert * rows:(expert + 1) * rows]
        return (c.to(torch.float64) - 8) * d.to(torch.float64).repeat_interleave(32, dim=1)

    for expert in ids.unique().tolist():
        row, slot = (ids == expert).nonzero(as_tuple=True)
        gu = torch.mm(x[row], dense(s["w13"], expert, 2 * I).t())
        g, u = gu[:, :I], gu[:, I:]
        out = torch.mm(g * torch.sigmoid(g) * u, dense(s["w2"], expert, H).t())
        y.index_add_(0, row, weights[row, slot][:, None] * out)
    return y
