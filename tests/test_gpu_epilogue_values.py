"""Values of the product with an epilogue and of its backward that are known without a tolerance
of their own: infinities, NaN and zeros.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
from epilogue_checks import R, close
from gpu_helpers import announce, free
from oracle import epilogue as O
from test_gpu_epilogue import Out, f64, workspace

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
