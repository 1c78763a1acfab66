"""MI355X-native 4-bit block-quantized linear layer.

    w = pack(codes, scales)           # canonical -> the library's packed form
    y = linear(x, w)                  # y[M, N] = x[M, K] . dequant(W[N, K])^T

A thin binding over libq4.so (include/q4.h): every step runs in the HIP
kernels; this module only checks tensors and passes device pointers and the
current HIP stream.  PyTorch supplies device memory and streams.

Format: blocks of 32 weights along K with one fp16 scale d each, 4-bit codes
q in 0..15, weight (q - 8) * d.  ``quantize`` makes codes and scales from
dense weights (absmax / 7 scaling, include/q4.h).  Canonical inputs: ``codes`` uint8 [N, K]
(one code per byte), ``scales`` float16 [N, K/32].  ``pack`` turns them into
the packed (tiled) form held by a ``Q4Weight``; ``x`` is bfloat16 or float16
[M, K], ``y`` is float32 [M, N].
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import KERNELS, Q4Error

__all__ = ["Q4Weight", "linear", "linear_noalloc", "linear_grouped", "pack", "pack_nibbles", "quantize", "quantize_pack", "concat_n", "split_n", "packed_sizes", "workspace_bytes", "get_crossover",
           "set_crossover", "segments", "Q4Error", "library_path",
           "Int8Matrix", "quantize_int8", "pack_int8", "quantize_pack_int8", "linear_int8",
           "moe_route", "moe_experts", "moe"]


def library_path() -> str:
    return _lib.LIB_PATH


@dataclass
class Q4Weight:
    """A packed N x K weight: ``codes`` uint8 [q4_packed_code_bytes],
    ``scales`` float16 [q4_packed_scale_bytes / 2], both on one GPU."""
    codes: torch.Tensor
    scales: torch.Tensor
    N: int
    K: int

    @property
    def device(self) -> torch.device:
        return self.codes.device


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t: torch.Tensor, name: str, dtypes, ndim: int, device=None):
    if (type(t) is torch.Tensor and t.is_cuda and t.dtype in dtypes and t.dim() == ndim and t.is_contiguous()
            and (device is None or t.device == device)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be a GPU tensor (got %s)" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must be %d-D, got shape %s" % (name, ndim, tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


# The current device and a device's current stream, as a number, without the
# objects around them (a decode step's calls are short).  A torch without GPU
# support has neither, and no GPU tensor that a call would accept.
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(dev: torch.device, name: str, f, *args) -> None:
    """f(*args, stream) with dev current; raises on a status."""
    i = dev.index
    if _get_device() == i:
        st = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _raw_stream(i))
    if st:
        _lib.check(st, name)


def packed_sizes(N: int, K: int):
    """(packed code bytes, packed scale bytes) of an N x K matrix."""
    lib = _lib.load()
    cb, sb = int(lib.q4_packed_code_bytes(N, K)), int(lib.q4_packed_scale_bytes(N, K))
    if cb == 0:
        raise ValueError("bad shape N=%d K=%d (K must be a positive multiple of 32)" % (N, K))
    return cb, sb


def pack(codes: torch.Tensor, scales: torch.Tensor) -> Q4Weight:
    """codes uint8 [N, K] (low 4 bits used), scales float16 [N, K/32] -> Q4Weight."""
    lib = _lib.load()
    _need(codes, "codes", (torch.uint8,), 2)
    dev = codes.device
    _need(scales, "scales", (torch.float16,), 2, dev)
    N, K = codes.shape
    if tuple(scales.shape) != (N, K // 32):
        raise ValueError("scales must be [%d, %d]" % (N, K // 32))
    cb, sb = packed_sizes(N, K)
    wq = torch.empty(cb, dtype=torch.uint8, device=dev)
    ws = torch.empty(sb // 2, dtype=torch.float16, device=dev)
    with torch.cuda.device(dev):
        st = lib.q4_pack(codes.data_ptr(), scales.data_ptr(), wq.data_ptr(), ws.data_ptr(), N, K, _stream(dev))
    _lib.check(st, "q4_pack")
    return Q4Weight(wq, ws, N, K)


def pack_nibbles(rows: torch.Tensor, scales: torch.Tensor) -> Q4Weight:
    """Nibble rows uint8 [N, K/2] (byte j: k = 2j low nibble, 2j + 1 high),
    scales float16 [N, K/32] -> Q4Weight (q4_pack_nibbles)."""
    lib = _lib.load()
    _need(rows, "rows", (torch.uint8,), 2)
    dev = rows.device
    _need(scales, "scales", (torch.float16,), 2, dev)
    N, K = rows.shape[0], rows.shape[1] * 2
    if tuple(scales.shape) != (N, K // 32):
        raise ValueError("scales must be [%d, %d]" % (N, K // 32))
    cb, sb = packed_sizes(N, K)
    wq = torch.empty(cb, dtype=torch.uint8, device=dev)
    ws = torch.empty(sb // 2, dtype=torch.float16, device=dev)
    with torch.cuda.device(dev):
        st = lib.q4_pack_nibbles(rows.data_ptr(), scales.data_ptr(), wq.data_ptr(), ws.data_ptr(), N, K,
                                 _stream(dev))
    _lib.check(st, "q4_pack_nibbles")
    return Q4Weight(wq, ws, N, K)


def quantize(w: torch.Tensor):
    """Dense weights [N, K] (float32, bfloat16 or float16, on a GPU) ->
    canonical (codes uint8 [N, K], scales float16 [N, K/32]) for ``pack``.
    Per block of 32 weights of a row: d = absmax / 7 rounded once to fp16,
    code = clamp(round_half_even(w / d), -8, 7) + 8 (include/q4.h)."""
    lib = _lib.load()
    _need(w, "w", (torch.float32, torch.bfloat16, torch.float16), 2)
    N, K = w.shape
    kind = {torch.float32: _lib.Q4_F32, torch.bfloat16: _lib.Q4_BF16, torch.float16: _lib.Q4_F16}[w.dtype]
    codes = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    scales = torch.empty((N, max(K // 32, 0)), dtype=torch.float16, device=w.device)
    with torch.cuda.device(w.device):
        st = lib.q4_quantize(w.data_ptr(), kind, codes.data_ptr(), scales.data_ptr(), N, K, _stream(w.device))
    _lib.check(st, "q4_quantize")
    return codes, scales


def quantize_pack(w: torch.Tensor) -> Q4Weight:
    """quantize() then pack(): dense weights [N, K] -> Q4Weight."""
    return pack(*quantize(w))


def workspace_bytes(M: int, N: int, K: int, kernel: str = "auto") -> int:
    return int(_lib.load().q4_workspace_bytes(M, N, K, KERNELS[kernel]))


def linear(x: torch.Tensor, w: Q4Weight, out: torch.Tensor | None = None, kernel: str = "auto",
           workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """y = x . dequant(w)^T on the current stream of x's device.

    kernel: "auto" (crossover rule), "gemv" or "gemm" (forced).  The result
    bits do not depend on this choice.
    workspace: True (default) allocates the workspace the matrix-matrix
    kernel can use; False/None runs without one; a uint8 tensor is used as
    given.
    """
    lib = _lib.load()
    _need(x, "x", (torch.bfloat16, torch.float16), 2)
    dev = x.device
    if not isinstance(w, Q4Weight):
        raise TypeError("w must be a Q4Weight (see pack)")
    _need(w.codes, "w.codes", (torch.uint8,), 1, dev)
    _need(w.scales, "w.scales", (torch.float16,), 1, dev)
    M, K = x.shape
    N = w.N
    if K != w.K:
        raise ValueError("x has K=%d, weight has K=%d" % (K, w.K))
    cb, sb = packed_sizes(N, K)
    if w.codes.numel() != cb or w.scales.numel() * 2 != sb:
        raise ValueError("packed weight sizes do not match N=%d K=%d" % (N, K))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), 2, dev)
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [%d, %d]" % (M, N))
    if kernel not in KERNELS:
        raise ValueError("kernel must be one of %s" % sorted(KERNELS))
    ws_ptr, ws_len = None, 0
    if isinstance(workspace, torch.Tensor):
        _need(workspace, "workspace", (torch.uint8,), 1, dev)
        ws_ptr, ws_len = workspace.data_ptr(), workspace.numel()
    elif workspace:
        need = lib.q4_workspace_bytes(M, N, K, KERNELS[kernel])
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            ws_ptr, ws_len = ws.data_ptr(), need
    dtype = _lib.Q4_BF16 if x.dtype == torch.bfloat16 else _lib.Q4_F16
    with torch.cuda.device(dev):
        st = lib.q4_linear_ex(x.data_ptr(), dtype, w.codes.data_ptr(), w.scales.data_ptr(), out.data_ptr(),
                              M, N, K, KERNELS[kernel], ws_ptr, ws_len, _stream(dev))
    _lib.check(st, "q4_linear_ex")
    return out


def linear_noalloc(x: torch.Tensor, w: Q4Weight, out: torch.Tensor, kernel: str = "auto") -> torch.Tensor:
    """q4_linear_noalloc: like ``linear`` with the library's fixed scratch
    buffer as the workspace, so the call allocates nothing (``out`` must be
    given).  Calls that overlap in time on one GPU share that buffer and
    race."""
    lib = _lib.load()
    _need(x, "x", (torch.bfloat16, torch.float16), 2)
    dev = x.device
    if not isinstance(w, Q4Weight):
        raise TypeError("w must be a Q4Weight (see pack)")
    _need(w.codes, "w.codes", (torch.uint8,), 1, dev)
    _need(w.scales, "w.scales", (torch.float16,), 1, dev)
    M, K = x.shape
    if K != w.K:
        raise ValueError("x has K=%d, weight has K=%d" % (K, w.K))
    _need(out, "out", (torch.float32,), 2, dev)
    if tuple(out.shape) != (M, w.N):
        raise ValueError("out must be [%d, %d]" % (M, w.N))
    if kernel not in KERNELS:
        raise ValueError("kernel must be one of %s" % sorted(KERNELS))
    dtype = _lib.Q4_BF16 if x.dtype == torch.bfloat16 else _lib.Q4_F16
    with torch.cuda.device(dev):
        st = lib.q4_linear_noalloc(x.data_ptr(), dtype, w.codes.data_ptr(), w.scales.data_ptr(), out.data_ptr(),
                                   M, w.N, K, KERNELS[kernel], _stream(dev))
    _lib.check(st, "q4_linear_noalloc")
    return out


def linear_grouped(x: torch.Tensor, weights, outs=None, workspace: torch.Tensor | bool | None = True) -> list:
    """q4_linear_grouped: y_i = x . dequant(w_i)^T for 1..8 weights sharing
    x's K, in one launch of the matrix-vector kernel where the crossover rule
    picks it (else one call per weight, with ``workspace`` as in ``linear``:
    True allocates the largest one the calls can use).  Returns the outputs
    (allocated unless ``outs`` is given)."""
    lib = _lib.load()
    _need(x, "x", (torch.bfloat16, torch.float16), 2)
    dev = x.device
    weights = list(weights)
    if not 1 <= len(weights) <= _lib.GROUP_MAX:
        raise ValueError("linear_grouped takes 1..%d weights" % _lib.GROUP_MAX)
    M, K = x.shape
    if outs is None:
        outs = [torch.empty((M, w.N), dtype=torch.float32, device=dev) for w in weights]
    outs = list(outs)
    if len(outs) != len(weights):
        raise ValueError("one output per weight")
    items = (_lib.GroupItem * len(weights))()
    for i, (w, y) in enumerate(zip(weights, outs)):
        if not isinstance(w, Q4Weight):
            raise TypeError("weights must be Q4Weight objects")
        if w.K != K:
            raise ValueError("weight %d has K=%d, x has K=%d" % (i, w.K, K))
        _need(w.codes, "w.codes", (torch.uint8,), 1, dev)
        _need(w.scales, "w.scales", (torch.float16,), 1, dev)
        cb, sb = packed_sizes(w.N, K)
        if w.codes.numel() != cb or w.scales.numel() * 2 != sb:
            raise ValueError("packed weight %d sizes do not match N=%d K=%d" % (i, w.N, K))
        _need(y, "out", (torch.float32,), 2, dev)
        if tuple(y.shape) != (M, w.N):
            raise ValueError("out %d must be [%d, %d]" % (i, M, w.N))
        items[i] = _lib.GroupItem(w.codes.data_ptr(), w.scales.data_ptr(), y.data_ptr(), w.N)
    ws_ptr, ws_len = None, 0
    if isinstance(workspace, torch.Tensor):
        _need(workspace, "workspace", (torch.uint8,), 1, dev)
        ws_ptr, ws_len = workspace.data_ptr(), workspace.numel()
    elif workspace:
        need = max(lib.q4_workspace_bytes(M, w.N, K, _lib.Q4_AUTO) for w in weights)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            ws_ptr, ws_len = ws.data_ptr(), need
    dtype = _lib.Q4_BF16 if x.dtype == torch.bfloat16 else _lib.Q4_F16
    with torch.cuda.device(dev):
        st = lib.q4_linear_grouped(x.data_ptr(), dtype, items, len(weights), M, K, ws_ptr, ws_len, _stream(dev))
    _lib.check(st, "q4_linear_grouped")
    return outs


@dataclass
class Int8Matrix:
    """A packed matrix of 8-bit codes with one scale for each row (weights, or
    activations that several products share): ``codes`` int8
    [q4_int8_packed_bytes], ``scales`` float32 [rows], both on one GPU."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    K: int

    @property
    def device(self) -> torch.device:
        return self.codes.device


_DTYPES = {torch.float32: _lib.Q4_F32, torch.bfloat16: _lib.Q4_BF16, torch.float16: _lib.Q4_F16}


def _int8_bytes(rows: int, K: int) -> int:
    n = _lib.load().q4_int8_packed_bytes(rows, K)
    if n == 0:
        raise ValueError("bad shape %d x %d (K must be a positive multiple of 32, at most 131040)" % (rows, K))
    return n


def _need_int8(w, name: str, device=None):
    if not isinstance(w, Int8Matrix):
        raise TypeError("%s must be an Int8Matrix (see pack_int8)" % name)
    _need(w.codes, name + ".codes", (torch.int8,), 1, device)
    _need(w.scales, name + ".scales", (torch.float32,), 1, w.codes.device)
    tiles = -(-w.rows // 16) * 2 * -(-w.K // 128)  # (q4_int8_packed_bytes, without the call)
    if w.K % 32 or tiles < 1 or w.codes.numel() != 1024 * tiles or w.scales.numel() != w.rows:
        raise ValueError("%s does not hold %d x %d packed codes and %d scales" % (name, w.rows, w.K, w.rows))


def quantize_int8(w: torch.Tensor):
    """Dense rows [R, K] (float32, bfloat16 or float16, on a GPU) -> canonical
    (codes int8 [R, K], scales float32 [R]) for ``pack_int8``.  For each row
    s = absmax / 127 rounded once to float32, code =
    clamp(round_half_even(w / s), -127, 127); a row with an infinity or NaN
    gets s = NaN and codes 0 (include/q4.h)."""
    lib = _lib.load()
    _need(w, "w", tuple(_DTYPES), 2)
    R, K = w.shape
    codes = torch.empty((R, K), dtype=torch.int8, device=w.device)
    scales = torch.empty(R, dtype=torch.float32, device=w.device)
    _call(w.device, "q4_int8_quantize", lib.q4_int8_quantize, w.data_ptr(), _DTYPES[w.dtype], codes.data_ptr(),
          scales.data_ptr(), R, K)
    return codes, scales


def pack_int8(codes: torch.Tensor, scales: torch.Tensor) -> Int8Matrix:
    """codes int8 [R, K], scales float32 [R] -> Int8Matrix (the scales tensor
    is kept as given)."""
    lib = _lib.load()
    _need(codes, "codes", (torch.int8,), 2)
    _need(scales, "scales", (torch.float32,), 1, codes.device)
    R, K = codes.shape
    if scales.numel() != R:
        raise ValueError("scales must be [%d]" % R)
    packed = torch.empty(_int8_bytes(R, K), dtype=torch.int8, device=codes.device)
    _call(codes.device, "q4_int8_pack", lib.q4_int8_pack, codes.data_ptr(), packed.data_ptr(), R, K)
    return Int8Matrix(packed, scales, R, K)


def quantize_pack_int8(w: torch.Tensor) -> Int8Matrix:
    """quantize_int8() and pack_int8() in one kernel: dense rows [R, K] ->
    Int8Matrix (a weight, or activations for several ``linear_int8`` calls)."""
    lib = _lib.load()
    _need(w, "w", tuple(_DTYPES), 2)
    R, K = w.shape
    packed = torch.empty(_int8_bytes(R, K), dtype=torch.int8, device=w.device)
    scales = torch.empty(R, dtype=torch.float32, device=w.device)
    _call(w.device, "q4_int8_quantize_pack", lib.q4_int8_quantize_pack, w.data_ptr(), _DTYPES[w.dtype],
          packed.data_ptr(), scales.data_ptr(), R, K)
    return Int8Matrix(packed, scales, R, K)


def _need_out(out, shape, dtypes, dev):
    _need(out, "out", dtypes, 2, dev)
    if tuple(out.shape) != shape:
        raise ValueError("out must be [%d, %d]" % shape)


def _workspace(workspace, need: int, dev):
    """(tensor to keep, pointer, bytes) of a call's workspace."""
    if isinstance(workspace, torch.Tensor):
        _need(workspace, "workspace", (torch.uint8,), 1, dev)
        return workspace, workspace.data_ptr(), workspace.numel()
    if workspace and need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        return ws, ws.data_ptr(), need
    return None, None, 0


def linear_int8(x, w: Int8Matrix, out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """y[m, n] = (sum_k qx[m, k] qw[n, k]) sx[m] sw[n] on the current stream of
    x's device.

    x: bfloat16 or float16 [M, K], quantized row by row within the call, or an
    Int8Matrix (``quantize_pack_int8``) that several products share; the bits
    are the same.  out_dtype: float32, bfloat16 or float16 (``out``'s own if
    given).  workspace: True allocates what the call needs; a uint8 tensor is
    used as given; False/None for calls that need none.
    """
    lib = _lib.load()
    if not isinstance(x, Int8Matrix):
        _need(x, "x", (torch.bfloat16, torch.float16), 2)
        M, K = x.shape
        kind, x_ptr, xs_ptr = _DTYPES[x.dtype], x.data_ptr(), None
    else:
        _need_int8(x, "x")
        M, K = x.rows, x.K
        kind, x_ptr, xs_ptr = _lib.Q4_I8, x.codes.data_ptr(), x.scales.data_ptr()
    dev = x.device
    _need_int8(w, "w", dev)
    N = w.rows
    if K != w.K:
        raise ValueError("x has K=%d, weight has K=%d" % (K, w.K))
    if out is None:
        if out_dtype not in _DTYPES:
            raise TypeError("out_dtype must be one of %s" % (tuple(_DTYPES),))
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    else:
        _need_out(out, (M, N), _DTYPES, dev)
    _keep, ws_ptr, ws_len = _workspace(workspace, lib.q4_int8_workspace_bytes(M, N, K, kind), dev)
    _call(dev, "q4_int8_linear", lib.q4_int8_linear, x_ptr, kind, xs_ptr, w.codes.data_ptr(), w.scales.data_ptr(),
          out.data_ptr(), _DTYPES[out.dtype], M, N, K, ws_ptr, ws_len)
    return out


def _need_route(x, router, topk, bias):
    _need(x, "x", (torch.bfloat16, torch.float16), 2)
    dev = x.device
    _need(router, "router", (x.dtype, torch.float32), 2, dev)
    M, K = x.shape
    E = router.shape[0]
    if router.shape[1] != K:
        raise ValueError("x has K=%d, router has K=%d" % (K, router.shape[1]))
    if bias is not None:
        _need(bias, "bias", (torch.float32,), 1, dev)
        if bias.numel() != E:
            raise ValueError("bias must be [%d]" % E)
    if not 1 <= topk <= E:
        raise ValueError("topk=%d of %d experts" % (topk, E))
    return M, K, E


def _need_experts(x, w13, w2):
    """(experts, I) of an expert layer's weights for x [M, H]."""
    M, H = x.shape
    for name, w in (("w13", w13), ("w2", w2)):
        _need_q4(w, name, x.device)
    I = w2.K
    E = w2.N // H if H else 0
    if w13.K != H or E < 1 or w2.N != E * H or w13.N != E * 2 * I:
        raise ValueError("x [%d, %d] with w13 %d x %d and w2 %d x %d: w13 is (E 2 I) x H, w2 (E H) x I"
                         % (M, H, w13.N, w13.K, w2.N, w2.K))
    return E, I


def _need_q4(w, name: str, dev):
    if not isinstance(w, Q4Weight):
        raise TypeError("%s must be a Q4Weight (see pack)" % name)
    _need(w.codes, name + ".codes", (torch.uint8,), 1, dev)
    _need(w.scales, name + ".scales", (torch.float16,), 1, dev)
    tiles = -(-w.N // 16) * -(-w.K // 128)  # (q4_packed_code_bytes, without the calls)
    if w.K % 32 or tiles < 1 or w.codes.numel() != 1024 * tiles or w.scales.numel() != 64 * tiles:
        raise ValueError("packed %s sizes do not match N=%d K=%d" % (name, w.N, w.K))


def moe_route(x: torch.Tensor, router: torch.Tensor, topk: int, bias: torch.Tensor | None = None,
              renormalize: bool = True, workspace: torch.Tensor | bool | None = True):
    """The topk experts of each row and their weights, by the largest of
    softmax(x . router^T + bias): (ids int32 [M, topk], weights float32
    [M, topk]), largest first, equal ones by lower index; the weights are
    divided by their sum where ``renormalize``.

    x: bfloat16 or float16 [M, K]; router: [E, K], x's dtype or float32; bias:
    float32 [E] (-inf disables an expert; a slot without an expert gets id -1
    and weight 0).  The logits are 64-bit sums, so a row's choice does not
    depend on the batch (include/q4.h).
    """
    lib = _lib.load()
    M, K, E = _need_route(x, router, topk, bias)
    dev = x.device
    ids = torch.empty((M, topk), dtype=torch.int32, device=dev)
    weights = torch.empty((M, topk), dtype=torch.float32, device=dev)
    _keep, ws_ptr, ws_len = _workspace(workspace, lib.q4_moe_route_workspace_bytes(M, E, K), dev)
    _call(dev, "q4_moe_route", lib.q4_moe_route, x.data_ptr(), _DTYPES[x.dtype], router.data_ptr(),
          _DTYPES[router.dtype], None if bias is None else bias.data_ptr(), ids.data_ptr(), weights.data_ptr(), M,
          E, K, topk, int(renormalize), ws_ptr, ws_len)
    return ids, weights


def moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: Q4Weight, w2: Q4Weight,
                out: torch.Tensor | None = None, workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """y[m] = sum_j weights[m, j] (h . dequant(w2[e])^T) with e = ids[m, j],
    [g | u] = x[m] . dequant(w13[e])^T and h = silu(g) u: float32 [M, H].

    x: bfloat16 or float16 [M, H]; ids int32, weights float32 [M, topk] (ids
    outside the experts add nothing).  w13: the experts' gate rows and up rows
    packed as one weight of N = E 2 I rows, K = H; w2: N = E H rows, K = I
    (``pack`` of the stacked rows, or ``concat_n`` of the experts' weights).
    """
    lib = _lib.load()
    _need(x, "x", (torch.bfloat16, torch.float16), 2)
    dev = x.device
    M, H = x.shape
    _need(ids, "ids", (torch.int32,), 2, dev)
    _need(weights, "weights", (torch.float32,), 2, dev)
    topk = ids.shape[1]
    if ids.shape[0] != M or weights.shape != ids.shape:
        raise ValueError("ids and weights must be [%d, topk], got %s and %s"
                         % (M, tuple(ids.shape), tuple(weights.shape)))
    E, I = _need_experts(x, w13, w2)
    if out is None:
        out = torch.empty((M, H), dtype=torch.float32, device=dev)
    else:
        _need_out(out, (M, H), (torch.float32,), dev)
    _keep, ws_ptr, ws_len = _workspace(workspace, lib.q4_moe_experts_workspace_bytes(M, H, I, topk), dev)
    _call(dev, "q4_moe_experts", lib.q4_moe_experts, x.data_ptr(), _DTYPES[x.dtype], ids.data_ptr(),
          weights.data_ptr(), w13.codes.data_ptr(), w13.scales.data_ptr(), w2.codes.data_ptr(),
          w2.scales.data_ptr(), out.data_ptr(), M, E, H, I, topk, ws_ptr, ws_len)
    return out


def moe(x: torch.Tensor, router: torch.Tensor, w13: Q4Weight, w2: Q4Weight, topk: int,
        bias: torch.Tensor | None = None, renormalize: bool = True, out: torch.Tensor | None = None,
        workspace: torch.Tensor | bool | None = True) -> torch.Tensor:
    """The whole expert layer, ``moe_route`` and ``moe_experts`` in one call
    (fewer launches, the same bits): float32 [M, H]."""
    lib = _lib.load()
    M, H, E = _need_route(x, router, topk, bias)
    dev = x.device
    experts, I = _need_experts(x, w13, w2)
    if experts != E:
        raise ValueError("the router has %d experts, the weights %d" % (E, experts))
    if out is None:
        out = torch.empty((M, H), dtype=torch.float32, device=dev)
    else:
        _need_out(out, (M, H), (torch.float32,), dev)
    _keep, ws_ptr, ws_len = _workspace(workspace, lib.q4_moe_layer_workspace_bytes(M, E, H, I, topk), dev)
    _call(dev, "q4_moe_layer", lib.q4_moe_layer, x.data_ptr(), _DTYPES[x.dtype], router.data_ptr(),
          _DTYPES[router.dtype], None if bias is None else bias.data_ptr(), w13.codes.data_ptr(),
          w13.scales.data_ptr(), w2.codes.data_ptr(), w2.scales.data_ptr(), out.data_ptr(), M, E, H, I, topk,
          int(renormalize), ws_ptr, ws_len)
    return out


def get_crossover() -> int:
    return int(_lib.load().q4_get_crossover())


def set_crossover(T: int) -> None:
    _lib.check(_lib.load().q4_set_crossover(int(T)), "q4_set_crossover")


def segments(K: int) -> int:
    return int(_lib.load().q4_segments(int(K)))


def concat_n(weights) -> Q4Weight:
    """Packed weights of one K stacked along N, for fused launches (q|k|v,
    gate|up): one call then computes all of them.  The packed form is
    tile-major along N, so concatenating the packed buffers packs the
    concatenated rows; every part but the last must have N a multiple of
    16 (no padding rows inside).  Each output column keeps its bits: the
    reduction order depends on K only."""
    weights = list(weights)
    if not weights:
        raise ValueError("concat_n needs at least one weight")
    K = weights[0].K
    for i, w in enumerate(weights):
        if not isinstance(w, Q4Weight):
            raise TypeError("concat_n takes Q4Weight objects")
        if w.K != K:
            raise ValueError("all weights must share K (%d != %d)" % (w.K, K))
        if i + 1 < len(weights) and w.N % 16:
            raise ValueError("every part but the last needs N % 16 == 0 (part %d has N=%d)" % (i, w.N))
    codes = torch.cat([w.codes for w in weights])
    scales = torch.cat([w.scales for w in weights])
    return Q4Weight(codes, scales, sum(w.N for w in weights), K)


def split_n(w: Q4Weight, Ns) -> list:
    """Views of a packed weight as consecutive row blocks of Ns[i] rows
    (all but the last a multiple of 16; sum(Ns) == w.N): the inverse of
    concat_n, sharing w's memory."""
    Ns = [int(n) for n in Ns]
    if sum(Ns) != w.N or any(n < 1 for n in Ns) or any(n % 16 for n in Ns[:-1]):
        raise ValueError("row blocks %s do not split N=%d on 16-row tiles" % (Ns, w.N))
    out, c0, s0 = [], 0, 0
    for n in Ns:
        cb, sb = packed_sizes(n, w.K)
        out.append(Q4Weight(w.codes[c0:c0 + cb], w.scales[s0:s0 + sb // 2], n, w.K))
        c0 += cb
        s0 += sb // 2
    return out
