"""Tolerances of the epilogue and dropout tests, derived from the arithmetic (no tests here).

h = 2^-24 is half an fp32 step, R = 2^-8 half a bf16 step, both relative to the value.

* z: a product of two bf16 values is exact in fp32; at most H + 16 additions (those of the
  matrix instructions, of the four waves and of the splits, the bias) of at most one step each:
  2 (H + 16) h (sum |x w| + |bias|).
* act: the exponential of an argument a that is itself rounded has a relative error of
  (4 |a| + 2) h, with |a| <= z^2 / 2 (gelu), |z| (silu), 1.6 |z| + 0.072 |z|^3 (gelu by tanh);
  the polynomial of the normal tail 8 h (4.7e-7), reciprocal, sums and products around them 16 h:
  (2 z^2 + 8 |z| + 0.3 |z|^3 + 32) h of the value, and an error dz of z gives slope * dz: the
  slopes are below 1.13, those of relu^2 below 2 (|z| + dz).  Where an exponential passes fp32's
  range the share is 0 instead of at most 2^-126.
* slopes: the same relative error on each of their two terms, twice for the products in them.
* dropout: its factor rounded once, one product: 2 h.  The residual: one addition, h.
* outputs: R or h of the value.
"""
import numpy as np

from oracle import epilogue as O

h, R = 2.0 ** -24, 2.0 ** -8


def round_tol(v, f32):
    return (h if f32 else R) * np.abs(v)


def z_tol(H, terms):
    return 2 * (H + 16) * h * terms


def act_cond(z):
    a = np.abs(z)
    return (2 * a * a + 8 * a + 0.3 * a ** 3 + 32) * h


def product_tol(z, dz, kind, factor, residual, f32):
    """Bound of |y - exact| from z (exact) and its own bound dz."""
    v = O.act(z, kind)
    slope = {O.NONE: 1.0, O.RELU: 1.0, O.RELU2: 2 * (np.abs(z) + dz)}.get(kind, 1.13)
    cond = 2 * h if kind in (O.NONE, O.RELU, O.RELU2) else act_cond(z)
    err = (slope * dz + cond * np.abs(v) + np.abs(z) * 2.0 ** -126 + 2 * h * np.abs(v)) * factor
    y = v * factor + (0 if residual is None else residual)
    err = err + h * (np.abs(v) * factor + np.abs(y))
    return (1 + R) * err + round_tol(y, f32)


def dz_tol(dy, pre, kind, factor):
    """Bounds of |dz - exact| before and after its rounding."""
    a, b = O.slope_terms(pre, kind)
    cond = 4 * h if kind in (O.NONE, O.RELU, O.RELU2) else 2 * act_cond(pre) + 8 * h
    err = np.abs(dy) * factor * ((np.abs(a) + np.abs(b)) * cond + (1 + np.abs(pre)) * 2.0 ** -126)
    exact = dy * factor * (a + b)
    return err, (1 + R) * err + R * np.abs(exact)


def close(got, want, tol, what):
    """|got - want| <= tol everywhere (NaN nowhere)."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        at = tuple(int(v) for v in np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d beyond their bound, first at %s: %r, want %r, bound %r" % (
            what, bad.sum(), bad.size, at, got[at], want[at], np.broadcast_to(tol, got.shape)[at]))
