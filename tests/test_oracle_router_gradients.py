"""The router oracle's gradient where its arithmetic is delicate (CPU)."""
import numpy as np
import pytest

from oracle import router as O


def test_gradient_of_saturated_sigmoids():
    """The oracle's gradient at large logits, where 1 - s as a difference has no digits left.
    One expert beside one of score 1/2: d gate = s (1 - s) = e^-z / (1 + e^-z)^2, a function of
    e^-z alone; of the shares p = s / (s + 1/2), the loss with counts (1, 0) has gradient
    u p (1 - s) (1 - p).  A few roundings of float64: 2^-48 of the value."""
    zs = np.array([20.0, 34.638683, 37.5, 60.0, 300.0, 700.0])
    z = np.stack([zs, np.zeros_like(zs)], 1)
    n = len(zs)
    ids = np.zeros((n, 1), np.int64)
    t = np.exp(-zs)
    gate = O.backward(z, ids, O.SIGMOID, False, 1.0, np.ones((n, 1)))[0]
    want = t / (1 + t) ** 2
    assert np.all(np.abs(gate[:, 0] - want) <= 2.0 ** -48 * want) and not gate[:, 1].any()
    cu = list(range(n + 1))
    counts = np.tile([1, 0], (n, 1))
    loss = O.backward(z, ids, O.SIGMOID, False, 1.0, None, cu, counts, np.ones(n))[0]
    s = 1 / (1 + t)
    p = s / (s + 0.5)
    want = 2 * p * t / (1 + t) * (0.5 / (s + 0.5))
    assert np.all(np.abs(loss[:, 0] - want) <= 2.0 ** -48 * want)


@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renormalised"])
@pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID], ids=["softmax", "sigmoid"])
def test_repeated_ids_against_differences(score, renorm):
    """The oracle's gradient where a token names an expert more than once: each naming is a gate
    of its own.  Central differences with steps of 2^-17 leave 2^-34 / 6 of a third derivative
    and 2^-53 / 2^-17 of rounding: 2^-30 of values around 1 covers both."""
    g = np.random.default_rng(4)
    T, E, K = 4, 7, 5
    z = g.standard_normal((T, E))
    ids = g.integers(0, E, (T, K)).astype(np.int32)
    ids[0], ids[1, 2:] = 3, 6
    dg = g.standard_normal((T, K))

    def value(a):
        return 1.5 * (dg * O.gate_shares(a, ids, score, renorm)).sum()

    want = O.backward(z, ids, score, renorm, 1.5, dg)[0]
    d = 2.0 ** -17
    for t in range(T):
        for e in range(E):
            step = np.zeros_like(z)
            step[t, e] = d
            diff = (value(z + step) - value(z - step)) / (2 * d)
            assert abs(diff - want[t, e]) <= 2.0 ** -30
