"""Oracle for the 8-bit activation checkpoints (test infrastructure only).

[TSR] §9.5: the backward needs the rows that dispatch laid out, or redoes the
dispatch.  The pages name no format for what is kept; the reading taken here is
one power-of-two scale per 32 consecutive values of a row and e4m3 codes (OCP
FP8: 1 sign bit, 4 exponent bits of bias 7, 3 mantissa bits, all-ones is NaN).

Codes are found by searching the table of e4m3 values, not by rounding
arithmetic.  Pinned by tests/test_oracle_q8.py.
"""
import numpy as np

from . import bf16

BLOCK = 32


def e4m3_table():
    """Value of each of the 256 codes, from the format's definition."""
    c = np.arange(256)
    exp, man = (c >> 3) & 15, c & 7
    v = np.where(exp == 0, man / 8.0 * 2.0 ** -6, (1 + man / 8.0) * 2.0 ** (exp - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


TABLE = e4m3_table()
POSITIVE = TABLE[:127]                                  # ascending, 0 .. 448


def encode_magnitude(a):
    """Code of the e4m3 value nearest to a in [0, 448], ties to the even code."""
    hi = np.clip(np.searchsorted(POSITIVE, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = a - POSITIVE[lo], POSITIVE[hi] - a
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def scale_exponent(top):
    """The least k >= -127 with top <= 448 * 2^k."""
    top = np.asarray(top, np.float64)
    k = np.full(top.shape, -127, np.int64)
    for _ in range(255):
        k = np.where(top > np.ldexp(448.0, k), k + 1, k)
    return k


def store(bits):
    """(q, scale) of bf16 rows [rows, width]: uint8 codes and scale bytes."""
    x = bf16.bits_to_f64(bits)
    rows, width = x.shape
    nb = -(-width // BLOCK)
    pad = np.zeros((rows, nb * BLOCK))
    pad[:, :width] = x
    v = pad.reshape(rows, nb, BLOCK)
    finite = np.isfinite(v)
    k = scale_exponent(np.where(finite, np.abs(v), 0.0).max(axis=2))
    u = np.ldexp(np.where(finite, v, 0.0), -k[:, :, None])
    code = encode_magnitude(np.abs(u)) | np.where(np.signbit(u), 128, 0)
    code = np.where(finite, code, 127)
    return (code.reshape(rows, -1)[:, :width].astype(np.uint8), (k + 127).astype(np.uint8))


def load(q, scale):
    """float64 values that codes and scale bytes stand for."""
    rows, width = q.shape
    k = np.repeat(scale.astype(np.int64) - 127, BLOCK, axis=1)[:, :width]
    return np.ldexp(TABLE[q], k)


def load_bits(q, scale):
    return bf16.f64_to_bits(load(q, scale))
