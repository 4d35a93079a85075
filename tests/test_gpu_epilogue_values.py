"""Values of the product with an epilogue and of its backward that are known without a tolerance
of their own: infinities, NaN and zeros in every row, and sums of whole numbers past 2^31 values.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
from epilogue_checks import R, close, h
from gpu_helpers import announce, free
from oracle import epilogue as O
from test_gpu_epilogue import Out, f64, matrix, rng_of, workspace

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


def test_bias_gradients_past_32_bits():
    """More than 2^31 values without an activation, dy 1/2 and half of them dropped: dz is 0 or
    1, so the biases' gradients are counts below 2^24, which fp32 sums without an error."""
    E, Hp, S = 4, 2048, (1 << 31) // 2048 // 4 + 176
    announce("bias gradients past 32 bits", E, Hp, S)
    c = mx.make_cfg(4, S, E, 1, 8, Hp, 0, mx.MODE_INFER)     # S Hp 2 < 4 GiB a rank
    plan = mx.Plan(c)
    # every rank has rows of every expert, cut anywhere, one segment without rows, and a rest
    cu = torch.tensor([[0, 3, 100003, 100003, S], [0, 0, 131071, 131099, S - 5], [0, S // 2, S // 2 + 1, S - 1, S],
                       [0, 77777, 155555, 200000, S - 300]], dtype=torch.int32)
    plan.cu_seqlens[:20].copy_(cu.reshape(-1))
    ec = mx.make_epilogue_cfg(O.NONE, 0.5)
    dy = torch.full((4 * S, Hp), 0.5, dtype=torch.bfloat16, device="cuda")
    assert dy.numel() > 1 << 31
    db, rng = torch.empty((E, Hp), device="cuda"), rng_of(12, 34)
    mx.moe_epilogue_backward(c, ec, plan, dy, None, rng, dy, db, workspace(c, ec))
    torch.cuda.synchronize()
    rows = 4 * S
    at = np.concatenate([np.arange(4), np.arange(rows // 2 - 2, rows // 2 + 2), np.arange(rows - 4, rows)])
    got = f64(dy.index_select(0, torch.from_numpy(at).cuda()))
    assert np.array_equal(got, 0.5 * O.row_factor(0.5, [12, 34], at, Hp))
    for e in range(E):
        count = torch.zeros(Hp, dtype=torch.int64, device="cuda")
        for r in range(4):
            lo, hi = (r * S + int(v) for v in cu[r, e:e + 2])
            for a in range(lo, hi, 1 << 15):
                count += (dy[a:min(hi, a + (1 << 15))] != 0).sum(0)
        assert int(count.max()) < 1 << 24
        assert torch.equal(db[e].double(), count.double()), e
