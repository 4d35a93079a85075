"""Pins of the 8-bit checkpoint oracle: the format's table, scales, rounding, errors."""
import numpy as np
import torch

from oracle import bf16, q8


def test_table_is_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q8.TABLE, t, equal_nan=True)
    assert q8.POSITIVE[-1] == 448 and np.all(np.diff(q8.POSITIVE) > 0)


def test_scale_exponents():
    assert q8.scale_exponent([448.0, 448.1, 896.0, 1.0, 1.75, 1.76, 0.0]).tolist() == \
        [0, 1, 1, -8, -8, -7, -127]


def test_rounding_by_hand():
    # 17 lies between 16 and 18, 19 between 18 and 20: ties to the even code
    assert q8.POSITIVE[q8.encode_magnitude(np.array([17.0, 19.0, 17.01, 448.0, 0.0]))].tolist() == \
        [16.0, 20.0, 18.0, 448.0, 0.0]


def test_round_trip_error_and_exactness_in_bf16():
    g = np.random.default_rng(1)
    x = np.exp(3 * g.standard_normal((64, 72))) * np.sign(g.standard_normal((64, 72)))
    b = bf16.f64_to_bits(x)
    v = bf16.bits_to_f64(b)
    q, s = q8.store(b)
    assert s.shape == (64, 3)
    w = q8.load(q, s)
    k = np.repeat(s.astype(int) - 127, 32, axis=1)[:, :72]
    assert np.all(np.abs(w - v) <= np.maximum(2.0 ** -4 * np.abs(v), np.ldexp(1.0, k - 10)))
    assert np.array_equal(bf16.bits_to_f64(q8.load_bits(q, s)), w)
    # what is kept is kept again unchanged
    q2, s2 = q8.store(q8.load_bits(q, s))
    assert np.array_equal(q8.load(q2, s2), w)


def test_values_that_are_not_finite():
    b = np.array([[0x7F80, 0xFF80, 0x7FC1, 0x3F80, 0x8000, 0, 0x0001, 0x7F7F]], np.uint16)
    q, s = q8.store(b[:, :7])
    w = q8.load(q, s)[0]
    assert np.isnan(w[:3]).all() and w[3] == 1.0 and s[0, 0] == 127 - 8
    assert q[0, 4] == 128 and q[0, 5] == 0
    q, s = q8.store(b)
    assert s[0, 0] == 127 + 120 and np.isfinite(q8.load(q, s)[0, 7])
