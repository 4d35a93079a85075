"""Counts, mean shares, loss and gradient at sizes where the sums are joined in parts.

A call's tokens go to workgroups of 8 ceil(T / 4096) tokens where it chooses (8 ceil(T / 8192)
where it does not).  Their sums are joined by one workgroup a sequence, by one for each 64
experts, or, with 256 or more workgroups a sequence, in eight parts first.  40,001 tokens take
all of these, several tokens a wave, and end in a workgroup of one token.  Tolerances are those
of tests/test_gpu_router.py.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import test_gpu_router as R
from gpu_helpers import announce, free
from oracle import router as O
from router_checks import check_gradient

pytestmark = pytest.mark.gpu

T = 40001


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


def loss_of(c, rc, z, ids, cu):
    """counts, prob and loss of moe_balance_loss, from a soiled workspace."""
    n, E = rc.nseq, c.E
    out = [R.Guarded(n * E, torch.int32), R.Guarded(n * E, torch.float32),
           R.Guarded(n, torch.float32)]
    ws = torch.full((mx.moe_router_workspace_size(c, rc),), 0xFF, dtype=torch.uint8, device="cuda")
    mx.moe_balance_loss(c, rc, z, ids, cu, *[o.t for o in out], ws)
    torch.cuda.synchronize()
    for o in out:
        o.check()
    counts, prob, loss = (o.t.cpu().numpy() for o in out)
    return {"counts": counts.reshape(n, E), "prob": prob.reshape(n, E), "loss": loss}


# one sequence of everything, one without the ends, eight parts of ragged ones with an empty one
# among them, one part, one that a single workgroup holds beside long ones
CUTS = {"all": None, "inner": [5, T - 7], "ragged3": [0, 17001, 17001, T - 1],
        "ragged7": [3, 4, 1000, 9001, 9001, 20000, 39990, T - 2], "short": [0, 20003, 20010, T]}


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("E", [65, 128, 130])
@pytest.mark.parametrize("cut", sorted(CUTS))
def test_forty_thousand_tokens(cut, E, bf16):
    announce("joins", cut, E, bf16)
    K, score = 5, O.SIGMOID if cut in ("inner", "ragged7") else O.SOFTMAX
    c = R.cfg_of(1, T, E, K)
    cu = np.array([0, T] if CUTS[cut] is None else CUTS[cut], np.int32)
    cug = None if CUTS[cut] is None else R.on_gpu(cu, torch.int32)
    n = len(cu) - 1
    zt, z = R.make_logits(T, E, bf16, E + n, 2.0)
    zg = zt.cuda()
    rc = mx.make_router_cfg(score, 1, 1.5, bf16, n)
    g = np.random.default_rng(E)
    # ids of a router of the program's own
    given = g.integers(0, E, (T, K)).astype(np.int32)
    counts, prob, loss = O.balance(z, given, cu, score)
    got = loss_of(c, rc, zg, R.on_gpu(given, torch.int32), cug)
    assert np.array_equal(got["counts"], counts)
    R.check_sums(z, got, c, rc, prob, loss)
    # chosen with the loss, without a bias and with one
    for bias in (None, (0.1 * g.standard_normal(E)).astype(np.float32)):
        bg = None if bias is None else R.on_gpu(bias, torch.float32)
        ids = R.check_forward(z, bias, R.run_forward(c, rc, zg, bg, cug, True), c, rc, cu)
    # forward only
    for b in (None, bg):
        R.check_forward(z, None if b is None else bias, R.run_forward(c, rc, zg, b, None, False), c,
                        rc, None)
    counts = O.balance(z, ids, cu, score)[0]
    dg = g.standard_normal((T, K)).astype(np.float32)
    dl = g.standard_normal(n).astype(np.float32)
    want, size = O.backward(z, ids, score, True, 1.5, dg, cu, counts, dl)
    got = R.run_backward(c, rc, zg, R.on_gpu(ids, torch.int32), R.on_gpu(dg, torch.float32), cug,
                         R.on_gpu(counts, torch.int32), R.on_gpu(dl, torch.float32))
    check_gradient(R.rel_of(z, score), got, want, size, bf16)


@pytest.mark.parametrize("S,E,nseq", [(9001, 1100, 1), (9001, 1100, 530), (300, 2048, 900)])
def test_more_experts_than_one_workgroup_joins(S, E, nseq):
    K = 3
    c = R.cfg_of(1, S, E, K)
    cu = R.cuts(S, nseq, 5, tail=3) if nseq > 1 else np.array([2, S - 3], np.int32)
    zt, z = R.make_logits(S, E, True, 6)
    rc = mx.make_router_cfg(O.SOFTMAX, 0, 1.0, True, nseq)
    given = np.random.default_rng(1).integers(0, E, (S, K)).astype(np.int32)
    counts, prob, loss = O.balance(z, given, cu, O.SOFTMAX)
    got = loss_of(c, rc, zt.cuda(), R.on_gpu(given, torch.int32), R.on_gpu(cu, torch.int32))
    assert np.array_equal(got["counts"], counts)
    R.check_sums(z, got, c, rc, prob, loss)


def test_as_many_sequences_as_a_call_takes():
    """2^20 sequences, almost all of them empty, and the gradient through them."""
    S, E, K, n = 5000, 8, 2, 1 << 20
    c = R.cfg_of(1, S, E, K)
    rc = mx.make_router_cfg(O.SIGMOID, 1, 1.0, False, n)
    cu = R.cuts(S, n, 8, tail=2)
    zt, z = R.make_logits(S, E, False, 9)
    cug = R.on_gpu(cu, torch.int32)
    got = R.run_forward(c, rc, zt.cuda(), None, cug, True)
    ids = R.check_forward(z, None, got, c, rc, cu)
    g = np.random.default_rng(2)
    dg, dl = g.standard_normal((S, K)).astype(np.float32), g.standard_normal(n).astype(np.float32)
    want, size = O.backward(z, ids, O.SIGMOID, True, 1.0, dg, cu, got["counts"], dl)
    got = R.run_backward(c, rc, zt.cuda(), R.on_gpu(ids, torch.int32), R.on_gpu(dg, torch.float32),
                         cug, R.on_gpu(got["counts"], torch.int32), R.on_gpu(dl, torch.float32))
    check_gradient(R.rel_of(z, O.SIGMOID), got, want, size, False)
