"""Pins of the router oracle: closed forms, ties, masks, and central differences."""
import numpy as np
import pytest

from oracle import router as R

SCORES = [R.SOFTMAX, R.SIGMOID]


def test_scores_closed_forms():
    z = np.log(np.array([[1.0, 2.0, 5.0]]))
    s, p = R.scores(z, R.SOFTMAX)
    assert np.allclose(s, [[1 / 8, 2 / 8, 5 / 8]], rtol=1e-15) and np.array_equal(s, p)
    s, p = R.scores(z, R.SIGMOID)
    want = np.array([[1 / 2, 2 / 3, 5 / 6]])
    assert np.allclose(s, want, rtol=1e-15) and np.allclose(p, want / want.sum(), rtol=1e-15)
    # scores that underflow keep their ratios
    _, p = R.scores(np.array([[-1000.0, -1000.0 + np.log(3.0)]]), R.SIGMOID)
    assert np.allclose(p, [[0.25, 0.75]], rtol=1e-12)


def test_choice_ties_masks_and_bias():
    inf = np.inf
    z = np.array([[1.0, 3.0, 3.0, 2.0], [-inf, -inf, 0.0, -inf], [-inf] * 4,
                  [np.nan, -inf, 1.0, np.nan], [0.0, -0.0, 0.0, -0.0]])
    assert R.choose(z, None, 3, R.SOFTMAX).tolist() == [[1, 2, 3], [2, 0, 1], [0, 1, 2],
                                                       [2, 1, 0], [0, 1, 2]]
    z = np.zeros((1, 4))
    assert R.choose(z, np.array([0.0, 1.0, -1.0, 1.0]), 4, R.SIGMOID).tolist() == [[1, 3, 0, 2]]
    w = R.gate_shares(np.array([[-inf] * 4]), np.array([[0, 1]]), R.SOFTMAX, True)
    assert w.tolist() == [[0.0, 0.0]]


def test_balance_by_hand():
    z = np.zeros((5, 2))
    ids = np.array([[0], [0], [1], [0], [7]])
    counts, prob, loss = R.balance(z, ids, [0, 3, 3, 5], R.SOFTMAX)
    assert counts.tolist() == [[2, 1], [0, 0], [1, 0]]
    assert prob.tolist() == [[0.5, 0.5], [0, 0], [0.5, 0.5]]
    assert np.allclose(loss, [1.0, 0.0, 0.5])


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("which", ["gates", "loss", "both"])
def test_backward_against_central_differences(score, renorm, which):
    g = np.random.default_rng(5)
    T, E, K, scale = 7, 6, 3, 1.7
    z = g.standard_normal((T, E))
    bias = 0.1 * g.standard_normal(E)
    ids = R.choose(z, bias, K, score)
    cu = [0, 2, 2, 6]                                     # token 6 is in no sequence
    dg, dl = g.standard_normal((T, K)), g.standard_normal(3)
    counts, _, _ = R.balance(z, ids, cu, score)

    def value(zz):
        v = 0.0
        if which != "loss":
            v += (dg * scale * R.gate_shares(zz, ids, score, renorm)).sum()
        if which != "gates":
            v += (dl * R.balance(zz, ids, cu, score)[2]).sum()
        return v

    dz, size = R.backward(z, ids, score, renorm, scale, dg if which != "loss" else None, cu,
                          counts, dl if which != "gates" else None)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            a, b = z.copy(), z.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((value(a) - value(b)) / (2 * h) - dz[t, e]) < 1e-8
    assert np.all(np.abs(dz) <= size * (1 + 1e-12) + 1e-300)
