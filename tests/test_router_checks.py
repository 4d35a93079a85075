"""The check of the router's gradients fails on what it must fail on (CPU)."""
import numpy as np
import pytest

from oracle import router as O
from router_checks import check_gradient, h


def gradient(score):
    g = np.random.default_rng(3)
    T, E, K = 5, 12, 3
    z = g.standard_normal((T, E))
    ids = O.choose(z, None, K, score)
    cu = [0, 2, T]
    counts = O.balance(z, ids, cu, score)[0]
    return O.backward(z, ids, score, True, 1.5, g.standard_normal((T, K)), cu, counts,
                      g.standard_normal(2))


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID], ids=["softmax", "sigmoid"])
def test_planted_values_fail(score, bf16):
    want, size = gradient(score)
    rel = (5 * 15 + 48) * h
    check_gradient(rel, want.copy(), want, size, bf16)
    for bad in (np.nan, np.inf, -np.inf, want[3, 7] + (2.0 ** -6 if bf16 else 2.0 ** -10) * size[3, 7]):
        got = want.copy()
        got[3, 7] = bad
        with pytest.raises(AssertionError):
            check_gradient(rel, got, want, size, bf16)
    with pytest.raises(AssertionError):
        check_gradient(rel, np.full_like(want, np.nan), want, size, bf16)
    # an oracle without a finite value passes nothing either
    gone = want.copy()
    gone[0, 0] = np.nan
    with pytest.raises(AssertionError):
        check_gradient(rel, gone.copy(), gone, size, bf16)
