"""Microscaled 4-bit floating point in numpy, from the format's definition: what the tests of the
quantiser and the product compare with."""
import numpy as np

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def quantize(x):
    """(codes (M, K) of 0 to 15, scales (M, ceil(K / 32)) bytes) of x in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    nb = -(-K // 32)
    b = np.zeros((M, nb * 32))
    b[:, :K] = x
    b = b.reshape(M, nb, 32)
    peak = np.abs(b).max(2)
    bad = ~np.isfinite(peak)
    _, e = np.frexp(np.where(bad, 0, peak))               # peak = f 2^e, 1/2 <= f < 1
    scales = np.where(peak == 0, 0, np.maximum(e - 1 - 2 + 127, 0))
    scales = np.where(bad, 255, scales)
    y = np.where(bad[:, :, None], 0, b) / np.exp2(np.where(bad, 0, scales - 127.0))[:, :, None]
    size = np.abs(y)
    code = np.zeros(y.shape, dtype=np.int64)
    for c in range(1, 8):
        border = (VALUES[c - 1] + VALUES[c]) / 2
        code[(size > border) | ((size == border) & (c % 2 == 0))] = c
    code = np.where(np.signbit(y), code + 8, code)
    code[bad] = 0
    return code.reshape(M, nb * 32)[:, :K].astype(np.uint8), scales.astype(np.uint8)


def pack(codes):
    M, K = codes.shape
    even = np.zeros((M, K + K % 2), dtype=np.uint8)
    even[:, :K] = codes
    return even[:, 0::2] | even[:, 1::2] << 4


def unpack(q, K=None):
    codes = np.stack([q & 15, q >> 4], axis=2).reshape(q.shape[0], -1)
    return codes if K is None else codes[:, :K]


def values(codes, scales):
    """The numbers that codes and scales stand for, in 64 bits."""
    K = codes.shape[1]
    unit = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return VALUES[codes] * np.repeat(unit, 32, axis=1)[:, :K]
