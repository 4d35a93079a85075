"""Gradients of the router by a check that NaN cannot pass.

The forms of tests/test_gpu_router.py are run again with it, and masks, far logits and rows of
nothing at widths of several registers per lane, in both types.  The tolerance is that module's.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import test_gpu_router as R
from gpu_helpers import free
from oracle import router as O
from router_checks import check_gradient

pytestmark = pytest.mark.gpu

SCORES = pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID], ids=["softmax", "sigmoid"])
TYPES = pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])


def strict(z, got, want, size, score, bf16):
    check_gradient(R.rel_of(z, score), got, want, size, bf16)


@pytest.fixture(autouse=True)
def _gpu(monkeypatch):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    monkeypatch.setattr(R, "check_backward", strict)
    free()
    yield
    free()


@TYPES
@SCORES
@pytest.mark.parametrize("shape", R.SHAPES, ids=str)
def test_shapes(shape, score, bf16):
    R.test_forward_and_backward(shape, score, bf16)


@SCORES
def test_masks_ties_and_extremes(score):
    R.test_masks_ties_and_extremes(score)


@TYPES
def test_given_ids(bf16):
    R.test_given_ids(bf16)


def test_large_batch():
    R.test_gradient_in_place_and_large_batch()


def hard_rows(E, K, seed):
    """Rows that take the kernels' other paths, with the masks at the row's ends too."""
    g = np.random.default_rng(seed)
    inf, low = np.inf, np.float32(-3.3895314e38)            # the lowest bf16 value
    n = lambda: g.standard_normal(E)                         # noqa: E731
    rows = [n(), np.full(E, -inf), np.full(E, low), np.full(E, 3.0), n() + 200, n() - 200,
            n() * 1e4, n() * 1e30, np.linspace(-80, -40, E), np.where(g.random(E) < 0.9, -inf, n())]
    for live in (1, K, K + 1):
        r = np.full(E, -inf)
        r[g.permutation(E)[:live]] = g.standard_normal(live)
        rows.append(r)
    first, last = np.full(E, -inf), np.full(E, -inf)
    first[0] = last[E - 1] = -50.0
    half = n()
    half[E // 2:] = low
    return np.array(rows + [first, last, half, n()], np.float32)


@TYPES
@SCORES
@pytest.mark.parametrize("E,K", [(130, 5), (384, 8), (897, 16), (1536, 3), (2047, 6)])
def test_masks_in_wide_rows(E, K, score, bf16):
    zt = torch.from_numpy(hard_rows(E, K, E))
    zt = zt.to(torch.bfloat16) if bf16 else zt
    z, T = zt.double().numpy(), zt.shape[0]
    assert np.isfinite(z[z != -np.inf]).all()
    c = R.cfg_of(1, T, E, K)
    g = np.random.default_rng(E + 1)
    cu = np.array([0, 1, 7, T - 1], np.int32)
    dg, dl = (g.standard_normal(n).astype(np.float32) for n in ((T, K), 3))
    bias = (0.3 * g.standard_normal(E)).astype(np.float32)
    for renorm, b in ((0, None), (1, None), (0, bias), (1, bias)):
        rc = mx.make_router_cfg(score, renorm, 1.0, bf16, 3)
        got = R.run_forward(c, rc, zt.cuda(), None if b is None else R.on_gpu(b, torch.float32),
                            R.on_gpu(cu, torch.int32), True)
        ids = R.check_forward(z, b, got, c, rc, cu)
        counts = O.balance(z, ids, cu, score)[0]
        for use_g, use_l in ((1, 1), (1, 0), (0, 1)):
            want, size = O.backward(z, ids, score, bool(renorm), 1.0, dg if use_g else None, cu,
                                    counts, dl if use_l else None)
            got = R.run_backward(c, rc, zt.cuda(), R.on_gpu(ids, torch.int32) if use_g else None,
                                 R.on_gpu(dg, torch.float32) if use_g else None,
                                 R.on_gpu(cu, torch.int32), R.on_gpu(counts, torch.int32),
                                 R.on_gpu(dl, torch.float32) if use_l else None)
            strict(z, got, want, size, score, bf16)
            assert np.all(got[1] == 0)                       # a row of nothing has no gradient
            assert np.all(got[z == -np.inf] == 0)            # nor has a masked expert


@TYPES
@SCORES
@pytest.mark.parametrize("E", [7, 384])
def test_in_place(E, score, bf16):
    """dlogits over logits, bit for bit as apart: gates, loss and both, with rows that take the
    path for far logits."""
    K, n = 3, 2
    zt = torch.from_numpy(np.concatenate([hard_rows(E, K, E), hard_rows(E, K, E + 1)]))
    zt = zt.to(torch.bfloat16) if bf16 else zt
    z, T = zt.double().numpy(), zt.shape[0]
    c = R.cfg_of(1, T, E, K)
    g = np.random.default_rng(E)
    ids = O.choose(z, None, K, score)
    cu = np.array([1, 9, T - 2], np.int32)
    counts = R.on_gpu(O.balance(z, ids, cu, score)[0], torch.int32)
    ids, cu = R.on_gpu(ids, torch.int32), R.on_gpu(cu, torch.int32)
    dg, dl = R.on_gpu(g.standard_normal((T, K)), torch.float32), R.on_gpu(g.standard_normal(n), torch.float32)
    for renorm in (0, 1):
        rc = mx.make_router_cfg(score, renorm, 2.0, bf16, n)
        for args in ((ids, dg, cu, counts, dl), (ids, dg, None, None, None),
                     (None, None, cu, counts, dl)):
            want = R.run_backward(c, rc, zt.cuda(), *args)
            zg = zt.cuda()
            mx.moe_router_backward(c, rc, zg, *args, zg)
            torch.cuda.synchronize()
            assert np.array_equal(zg.double().cpu().numpy(), want)


@TYPES
@SCORES
def test_expert_named_twice(score, bf16):
    """Each naming is a gate of its own; their parts add at the expert's logit."""
    T, E, K = 40, 30, 6
    g = np.random.default_rng(12)
    zt, z = R.make_logits(T, E, bf16, 13)
    ids = g.integers(0, E, (T, K)).astype(np.int32)
    ids[:, 1] = ids[:, 0]
    ids[:10, 3:] = ids[:10, :1]                             # five of six the same
    ids[10:20] = ids[10:20, :1]                             # all the same
    ids[20:25, 2] = -1
    c = R.cfg_of(1, T, E, K)
    dg = g.standard_normal((T, K)).astype(np.float32)
    for renorm in (0, 1):
        rc = mx.make_router_cfg(score, renorm, 1.5, bf16, 1)
        want, size = O.backward(z, ids, score, bool(renorm), 1.5, dg)
        got = R.run_backward(c, rc, zt.cuda(), R.on_gpu(ids, torch.int32),
                             R.on_gpu(dg, torch.float32), None, None, None)
        strict(z, got, want, size, score, bf16)
