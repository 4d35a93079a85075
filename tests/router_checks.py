"""Check of a router gradient that NaN cannot pass (shared by the CPU and the GPU tests).

The tolerance is that of the router's GPU tests: with h = 2^-24 and X the row's spread of
logits, a share is off by rel = (5 X + 48) h, a gradient by (3 rel + 48 h) times the sum of
the magnitudes it is made of (size), and by half a bf16 step where it is rounded to bf16.
"""
import numpy as np

h = 2.0 ** -24


def check_gradient(rel, got, want, size, bf16):
    """Every value of got is finite and within its tolerance of want, itself finite."""
    tol = (3 * rel + 48 * h) * size + 2 * 2.0 ** -126
    if bf16:
        tol = tol + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    assert np.isfinite(want).all() and np.isfinite(tol).all(), "the oracle has no finite value"
    good = np.isfinite(got)
    good[good] = np.abs(got[good] - want[good]) <= tol[good]
    assert good.all(), (np.argwhere(~good)[:5], got[~good][:5], want[~good][:5], tol[~good][:5])
