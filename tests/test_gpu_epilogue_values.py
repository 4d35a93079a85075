"""Values of the product with an epilogue and of its backward that are known without a tolerance
of their own: infinities, NaN and zeros in every row.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
from epilogue_checks import R, close, h
from gpu_helpers import announce, free
from oracle import epilogue as O
from test_gpu_epilogue import Out, f64, matrix, workspace

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


def same(got, want, tol, what):
    """close, where NaN and infinities have to stand in the same places."""
    got, want = np.broadcast_arrays(np.asarray(got, np.float64), np.asarray(want, np.float64))
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf]), what
    ok = np.isfinite(want)
    close(got[ok], want[ok], np.broadcast_to(tol, want.shape)[ok], what)


# every tile of the product, with the k axis whole and in parts
@pytest.mark.parametrize("S,H,Hp", [(3, 16, 8), (1300, 16, 8), (2, 728, 24), (13, 7160, 392), (943, 360, 1080),
                                    (567, 3376, 536), (2406, 432, 824), (1485, 3824, 1392), (4100, 1000, 520),
                                    (6881, 360, 7016), (653, 7064, 5520)])
@pytest.mark.parametrize("kind", range(6))
def test_special_values_in_every_row(S, H, Hp, kind):
    """The values as bias on zero products: each row is the function of the bias.

    The share that a function multiplies by is 0 or 1 here, off by one unit of the hardware
    reciprocal, 2 h, and the product by h; squares and pre are rounded once.
    """
    vals = np.array([INF, -INF, NAN, 0.0, -0.0, 1e30, -1e30, 3e38])
    k = matrix(S, H, Hp, kind, f32=True, pre=True, seed=1)
    k.x.zero_()
    k.bias[0] = torch.from_numpy(np.resize(vals, Hp)).float()
    k()
    k.y.check()
    k.pre.check()
    z = f64(k.bias)[0]
    with np.errstate(invalid="ignore", over="ignore"):
        want = O.act(z, kind).astype(np.float32).astype(np.float64)
        same(f64(k.y.t), want[None], 4 * h * np.abs(want)[None], "y")
        same(f64(k.pre.t), z[None], R * np.abs(z)[None], "pre")


@pytest.mark.parametrize("S", [1, 9, 5000])
@pytest.mark.parametrize("kind", range(6))
def test_gradients_that_are_not_finite(kind, S):
    """dz is a product: infinity times a slope of 0 is NaN, as NaN times any slope is."""
    pre = np.array([-3.0, -0.0, 0.0, 2.0, -1.0, 0.5, 4.0, NAN])
    dy = np.array([INF, -INF, NAN, 1.0])
    announce("gradients that are not finite", kind, S)
    Hp = 32
    c = mx.make_cfg(1, S, 1, 1, 8, Hp, 0, mx.MODE_INFER)
    zt = torch.from_numpy(np.tile(pre, 4)).to("cuda", torch.bfloat16).repeat(S, 1)
    dt = torch.from_numpy(np.repeat(dy, 8)).to("cuda", torch.float32).repeat(S, 1)
    dz, db = Out(S, Hp, torch.bfloat16), Out(1, Hp, torch.float32)
    ec = mx.make_epilogue_cfg(kind, 0.0, True)
    mx.moe_epilogue_backward(c, ec, None, dt, zt, None, dz.t, db.t, workspace(c, ec))
    torch.cuda.synchronize()
    dz.check()
    db.check()
    slope = O.slope(np.tile(pre, 4), kind)
    if kind != O.NONE:                                     # without an activation pre is not read
        slope[np.isnan(np.tile(pre, 4))] = NAN
    with np.errstate(invalid="ignore"):
        want = np.repeat(dy, 8) * slope
    same(f64(dz.t), want[None], 1.1 * R * np.abs(want)[None], "dz")
    finite = np.isfinite(want)
    assert np.array_equal(np.isfinite(f64(db.t))[0], finite)
    assert np.array_equal(np.isnan(f64(db.t))[0], np.isnan(want))
