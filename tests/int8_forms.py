"""The forms of the 8-bit product and shapes that take them, for the tests."""
import ctypes

from bit_quantized_matmul_q4_amd import build

# form: (M, N, K) of dense x.  A tile form is "rows x columns"; "/s" where K is
# split.  Odd N, short last steps of K, rows past the last tile, and more than
# one band of four row tiles with every remainder (9, 11, 14, 17 and 13 of them).
FORMS = {
    "decode": [(1, 40, 18944), (1, 33, 20480), (2, 40, 9984), (2, 31, 10240), (3, 17, 6752), (3, 40, 64),
               (4, 100, 5120), (4, 31, 96), (4, 48, 4128)],
    "gemv": [(1, 21, 20512), (3, 8200, 64), (5, 40, 18944), (33, 300, 9984), (64, 33, 20480),
             (16, 24577, 64), (64, 24576, 32)],
    "64x64": [(65, 12001, 96), (333, 4863, 896), (17, 24577, 160), (48, 60001, 32), (64, 26000, 544)],
    "64x64/s": [(124, 301, 18944), (70, 33, 20512)],
    "128x64": [(1030, 3101, 160), (1400, 2503, 96), (1793, 1666, 544)],
    "128x64/s": [(25700, 60, 1056)],
    "128x128": [(65, 51300, 96), (128, 60001, 160), (2050, 3333, 288), (1030, 6401, 608)],
    "256x256": [(129, 51300, 64), (4100, 3301, 160), (3100, 4602, 416), (2600, 5121, 2080)],
}


def form_of(dense, M, N, K):
    """The form's name, and the rows a workgroup of the quantizer."""
    f = ctypes.CDLL(build.PROBE_LIB).q4probe_int8_form
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int)]
    r = (ctypes.c_int * 6)()
    f(int(dense), M, N, K, r)
    decode, gemv, bm, bn, split, rows = r
    name = "decode" if decode else "gemv" if gemv else "%dx%d" % (bm, bn) + ("/s" if split > 1 else "")
    return name, rows
