"""Ids where masks, NaN and infinities of logits and biases meet in one row, against the oracle."""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import test_gpu_router as R
from gpu_helpers import announce, free
from oracle import router as O

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


def rows(E, seed):
    """Rows with every mix of masks, NaN and both infinities, and one without any."""
    g = np.random.default_rng(seed)
    out = [g.standard_normal(E)]
    for mask in (0.0, 0.3, 0.9):
        for nan in (0, 1, E // 3):
            for inf in (0, 1, 3):
                r = g.standard_normal(E)
                r[g.random(E) < mask] = -np.inf
                r[g.permutation(E)[:nan]] = np.nan
                r[g.permutation(E)[:inf]] = np.inf
                out.append(r)
    none = np.full(E, -np.inf)
    none[E // 2] = np.nan                                   # masked ones and one NaN
    return np.array(out + [none], np.float32)


def biases(E, seed):
    g = np.random.default_rng(seed)
    plain = (0.2 * g.standard_normal(E)).astype(np.float32)
    wild = plain.copy()
    for v in (np.nan, np.inf, -np.inf, 3.4028235e38, -3.4028235e38):
        wild[g.permutation(E)[:max(1, E // 12)]] = v
    low = plain.copy()
    low[g.random(E) < 0.8] = -np.inf                        # live ones behind live ones
    return {"none": None, "zero": np.zeros(E, np.float32), "plain": plain, "wild": wild, "low": low}


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(24, 5), (24, 24), (65, 12), (384, 8), (897, 30)])
def test_ids(E, K, score, bf16):
    zt = torch.from_numpy(rows(E, E + K))
    zt = zt.to(torch.bfloat16) if bf16 else zt
    z, T = zt.double().numpy(), zt.shape[0]
    c = R.cfg_of(1, T, E, K)
    rc = mx.make_router_cfg(score, 1, 1.0, bf16, 1)
    for name, b in biases(E, K).items():
        announce("router order", E, K, score, bf16, name)
        with np.errstate(invalid="ignore"):
            want = O.choose(z, b, K, score)
        bg = None if b is None else R.on_gpu(b, torch.float32)
        for stats in (False, True):
            got = R.run_forward(c, rc, zt.cuda(), bg, None, stats)
            assert np.array_equal(got["ids"], want), (name, stats)
        counts = np.bincount(want.reshape(-1), minlength=E)
        assert np.array_equal(got["counts"][0], counts), name
