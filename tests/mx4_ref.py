"""Plain 64-bit computations of the microscaled 4-bit form, on the CPU."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def quantize(x):
    """x [R, K] -> (codes [R, K], one a byte, scale bytes [R, K / 32])."""
    R, K = x.shape
    d = x.double().reshape(R, K // 32, 32)
    bad = ~torch.isfinite(d).all(2)
    d = torch.where(bad[:, :, None], torch.zeros_like(d), d)
    top = d.abs().amax(2)
    e = torch.frexp(top)[1] - 3  # floor(log2(top)) - 2
    e = torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    a = torch.ldexp(d.abs(), -e[:, :, None])
    borders = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))
    codes = torch.zeros(d.shape, dtype=torch.uint8)
    for border, up in borders:  # a tie goes to the even code
        codes += ((a >= border) if up else (a > border)).to(torch.uint8)
    codes += 8 * torch.signbit(d).to(torch.uint8)
    codes[bad] = 0
    scales = (e + 127).to(torch.uint8)
    scales[bad] = 255
    return codes.reshape(R, K), scales


def values(codes, scales):
    """What codes and scale bytes stand for, [R, K] in 64 bits."""
    R, K = codes.shape
    v = torch.ldexp(E2M1[codes.long()].reshape(R, K // 32, 32), scales.to(torch.int32)[:, :, None] - 127)
    v[scales == 255] = float("nan")
    return v.reshape(R, K)


def nibbles(codes):
    """[R, K] one a byte -> [R, K / 2], even k in the low half."""
    return codes[:, 0::2] | codes[:, 1::2] << 4


def packed(codes, scales):
    """Canonical codes (one a byte) and scale bytes -> the packed bytes, element by element from the layout's
    definition."""
    R, K = codes.shape
    T, Q, G = -(-R // 16), -(-K // 128), -(-K // 512)
    c = torch.zeros((T * 16, Q * 128), dtype=torch.uint8)
    c[:R, :K] = codes
    s = torch.zeros((T * 16, G * 16), dtype=torch.uint8)
    s[:R, :K // 32] = scales
    row, k = torch.meshgrid(torch.arange(T * 16), torch.arange(0, Q * 128, 2), indexing="ij")
    at = (row // 16 * Q + k // 128) * 1024 + 16 * (16 * (k // 32 % 4) + row % 16) + k % 32 // 2
    out = torch.zeros(T * Q * 1024, dtype=torch.uint8)
    out[at.reshape(-1)] = nibbles(c).reshape(-1)
    row, b = torch.meshgrid(torch.arange(T * 16), torch.arange(G * 16), indexing="ij")
    at = (row // 16 * G + b // 16) * 256 + 4 * (16 * (b % 4) + row % 16) + b // 4 % 4
    outs = torch.zeros(T * G * 256, dtype=torch.uint8)
    outs[at.reshape(-1)] = s.reshape(-1)
    return out, outs


def product(x, w):
    """(x . w^T, the sum of the magnitudes) in 64 bits of value matrices."""
    return x @ w.T, x.abs() @ w.abs().T
