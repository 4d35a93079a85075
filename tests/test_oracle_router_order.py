"""The oracle's choice where masks, NaN and infinities meet, by hand (CPU)."""
import numpy as np
import pytest

from oracle import router as O

nan, inf = np.nan, np.inf


@pytest.mark.parametrize("score,z,bias,want", [
    # numbers by size, then masked, then NaN
    (O.SIGMOID, [0, -inf, nan, 2, 1], None, [3, 4, 0, 1, 2]),
    (O.SIGMOID, [0, -inf, nan, 2, 1], [0, 9, 9, 0, 0], [3, 4, 0, 1, 2]),
    # a live expert of bias -inf comes before a masked one of any bias
    (O.SIGMOID, [-inf, 0, -inf, 1, 2], [5, -inf, 0, -inf, 0], [4, 1, 3, 0, 2]),
    (O.SOFTMAX, [-inf, 0, -inf, 1, 2], [5, -inf, 0, -inf, 0], [4, 1, 3, 0, 2]),
    # one NaN logit makes every score of a softmax row NaN: live ones by id, masked, NaN
    (O.SOFTMAX, [nan, -inf, 0, 2, 1], [0, 0, 0, 0, 0], [2, 3, 4, 1, 0]),
    # so does +inf
    (O.SOFTMAX, [0, -inf, inf, 2, nan], [0, 0, 0, 0, 0], [0, 2, 3, 1, 4]),
    (O.SIGMOID, [0, -inf, inf, 2, nan], [0, 0, 0, 0, 0], [2, 3, 0, 1, 4]),
    # a NaN bias: after the numbers, before the masked
    (O.SIGMOID, [0, -inf, 1, 2, nan], [0, nan, nan, 0, 0], [3, 0, 2, 1, 4]),
    # infinite biases are numbers; +inf - inf never enters a score plus bias
    (O.SIGMOID, [0, 3, 1, 2, -inf], [inf, -inf, 0, inf, inf], [0, 3, 2, 1, 4]),
    (O.SOFTMAX, [-inf, -inf, nan, -inf, -inf], [0, 1, 2, 3, nan], [0, 1, 3, 4, 2])])
def test_order(score, z, bias, want):
    b = None if bias is None else np.array(bias, np.float64)
    with np.errstate(invalid="ignore"):
        for K in range(1, 6):
            got = O.choose(np.array([z], np.float64), b, K, score)
            assert got.tolist() == [want[:K]]
