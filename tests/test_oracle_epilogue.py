"""Pins of oracle.epilogue (CPU)."""
import numpy as np
import pytest

from oracle import epilogue as O

ACTS = [O.NONE, O.RELU, O.GELU, O.GELU_TANH, O.SILU, O.RELU2]


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(counter, key, words):
    """The published test vectors of Philox4x32-10: zeros, ones, and the digits of pi."""
    assert tuple(int(v) for v in O.philox(counter, key)) == words


def test_numbers_follow_the_layout():
    zero = O.numbers((0, 0), np.arange(8))
    want = [w >> (16 * (i % 2)) & 0xFFFF for w in (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
            for i in range(2)]
    assert zero.tolist() == want
    # negative int64 values of rng are their two's complement words
    assert np.array_equal(O.numbers((-1, -2), np.arange(64)),
                          O.numbers((2 ** 64 - 1, 2 ** 64 - 2), np.arange(64)))


@pytest.mark.parametrize("p", [0.0, 0.1, 0.25, 0.5, 0.9, 1.0, 2.0 ** -18])
def test_share_and_mean(p):
    n = 1 << 20
    f = O.factor(p, (123456789, 7), np.arange(n))
    d = O.steps(p)
    assert d == round(65536 * float(np.float32(p)))
    share = d / 65536
    # five standard deviations of a share of n independent draws
    assert abs((f == 0).mean() - share) <= 5 * np.sqrt(share * (1 - share) / n)
    assert set(np.unique(f)) <= {0.0, 65536 / max(1, 65536 - d)}


def test_numbers_differ_by_seed_step_and_place():
    a = O.numbers((5, 9), np.arange(4096))
    for other in (O.numbers((6, 9), np.arange(4096)), O.numbers((5, 10), np.arange(4096)),
                  O.numbers((5 + (1 << 32), 9), np.arange(4096)),
                  O.numbers((5, 9 + (1 << 32)), np.arange(4096)),
                  O.numbers((5, 9), np.arange(4096) + 4096), O.numbers((5, 9), np.arange(4096) + (1 << 35))):
        assert (a == other).mean() < 0.01


@pytest.mark.parametrize("kind", ACTS)
def test_slopes_by_differences(kind):
    z = np.concatenate([np.linspace(-8, 8, 2001) + 1e-3, [-30.0, 25.0, 1e-6, -1e-6]])
    h = 1e-6
    z = z[np.abs(z) > 10 * h]                            # away from the corner of relu
    diff = (O.act(z + h, kind) - O.act(z - h, kind)) / (2 * h)
    assert np.abs(diff - O.slope(z, kind)).max() <= 1e-8 * (1 + np.abs(z).max())


def test_values():
    z = np.array([-2.0, 0.0, 1.0, 3.0])
    assert O.act(z, O.RELU).tolist() == [0, 0, 1, 3] and O.act(z, O.RELU2).tolist() == [0, 0, 1, 9]
    assert np.allclose(O.act(z, O.GELU), [-0.04550026389635842, 0, 0.8413447460685429, 2.9959502763],
                       atol=1e-9)
    u = np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    assert np.allclose(O.act(z, O.GELU_TANH), 0.5 * z * (1 + np.tanh(u)), atol=1e-15)
    assert np.allclose(O.act(z, O.SILU), z / (1 + np.exp(-z)), atol=1e-15)


def test_gradients_by_differences():
    g = np.random.default_rng(1)
    rows, n, E, rng = 12, 16, 3, (77, 5)
    expert = np.array([0] * 5 + [2] * 6 + [-1])
    z, dy, bias = g.standard_normal((rows, n)), g.standard_normal((rows, n)), g.standard_normal((E, n))
    own = np.where((expert >= 0)[:, None], bias[np.maximum(expert, 0)], 0)
    for kind in ACTS:
        loss = lambda b: (dy * O.forward(z + np.where((expert >= 0)[:, None], b[np.maximum(expert, 0)], 0),
                                         kind, 0.25, rng, z)).sum()
        dz, dbias = O.backward(dy, z + own, kind, 0.25, rng, expert, E)
        assert np.all(dbias[1] == 0)
        for e, c in ((0, 0), (2, 7), (2, 15)):
            step = np.zeros_like(bias)
            step[e, c] = 1e-6
            assert abs((loss(bias + step) - loss(bias - step)) / 2e-6 - dbias[e, c]) < 1e-6
    T, K = 6, 2
    y, gates = g.standard_normal((T * K, n)), g.random((T, K))
    route = g.permutation(T * K)
    route[3] = -1
    dout = g.standard_normal((T, n))
    loss = lambda yy, gg: (dout * O.combine(yy, gg, route, 0.5, rng)).sum()
    dy, dgates = O.combine_backward(dout, y, gates, route, 0.5, rng)
    assert dgates.reshape(-1)[3] == 0
    for t, k, c in ((0, 0, 3), (4, 1, 9)):
        step = np.zeros_like(gates)
        step[t, k] = 1e-6
        assert abs((loss(y, gates + step) - loss(y, gates - step)) / 2e-6 - dgates[t, k]) < 1e-6
        step = np.zeros_like(y)
        step[route.reshape(T, K)[t, k], c] = 1e-6
        assert abs((loss(y + step, gates) - loss(y - step, gates)) / 2e-6 - dy[t, k, c]) < 1e-6


def test_segment_experts():
    cu = np.array([[0, 2, 2, 3, 5], [0, 0, 4, 5, 5]])
    got = O.segment_experts(cu, np.array([[1, -1], [0, 0]]), 2, 6)
    assert got.tolist() == [0, 0, 1, -2, -2, -1, 1, 1, 1, 1, 0, -1]
