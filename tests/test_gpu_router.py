"""Router, balance loss and their gradients against the float64 oracle.

Tolerances, from the arithmetic, with h = 2^-24 (half an fp32 step, relative):

* a score's exponential: its argument x is rounded (|x| h), multiplied by
  log2 e, itself rounded (0.2 h), (|x| h again) and exponentiated (1 ulp = 2 h):
  (2.2 |x| + 2) h.  |x| is at most X = the largest |z - max z| of the row among
  finite logits (sigmoid: the largest |z|), counted up to 110, past which the
  score is 0 in fp32, and from 15 on: a softmax whose largest logit lies
  between -15 and 13 is not shifted by it, which lengthens |x| by 15 at most;
* the sum over E experts, whose terms are off by as much: P <= 32 additions in
  a lane and 6 across lanes, and the reciprocal and products that follow, 4
  more: a share is off by rel = (5 X + 2 + 32 + 6 + 8) h at most;
* what fp32 cannot hold (scores below 2^-126) is 2^-126 absolute;
* the sums over a sequence: one wave adds at most chunk / 8 tokens, then 8
  waves; the join is float64.  chunk = 8 ceil(T / 4096) at most;
* the gradient is a sum of terms whose magnitudes the oracle adds up (size);
  each is a product of up to 3 rounded shares and 6 roundings, and its mean
  over experts adds 40 more: (3 rel + 48 h) size.  A bf16 result adds half a
  step, 2^-8 |dz|.
"""
import ctypes

import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import workloads as W
from gpu_helpers import announce, free
from oracle import router as O

pytestmark = pytest.mark.gpu

h = 2.0 ** -24
TINY_ABS = 2.0 ** -126
SENT = 0x5A


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


def cfg_of(R, S, E, K):
    return mx.make_cfg(R, S, E, K, 8, 8, 0, mx.MODE_INFER)


def on_gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=dtype)


class Guarded:
    """An output tensor with 64 bytes of sentinel before and behind it."""

    def __init__(self, n, dtype):
        size = torch.empty((), dtype=dtype).element_size()
        pad = 64
        self.raw = torch.full((2 * pad + n * size,), SENT, dtype=torch.uint8, device="cuda")
        self.t = self.raw[pad:pad + n * size].view(dtype)
        self.pad, self.end = pad, pad + n * size

    def check(self):
        assert torch.all(self.raw[:self.pad] == SENT) and torch.all(self.raw[self.end:] == SENT)


def spread(z, score):
    """X of the module's comment, per row."""
    f = np.where(np.isfinite(z), z, np.nan)
    if score == O.SIGMOID:
        x = np.nan_to_num(np.abs(f)).max(axis=1)
    else:
        x = np.where(np.isnan(f), -np.inf, f).max(axis=1) - np.where(np.isnan(f), np.inf, f).min(axis=1)
    return np.clip(x, 15.0, 110.0)[:, None]


def rel_of(z, score):
    return (5 * spread(z, score) + 48) * h


def run_forward(c, rc, z, bias, cu, stats):
    T = c.R * c.S
    out = {"ids": Guarded(T * c.K, torch.int32), "gates": Guarded(T * c.K, torch.float32)}
    args = {}
    if stats:
        out["counts"] = Guarded(rc.nseq * c.E, torch.int32)
        out["prob"] = Guarded(rc.nseq * c.E, torch.float32)
        out["loss"] = Guarded(rc.nseq, torch.float32)
        n = mx.moe_router_workspace_size(c, rc)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # garbage: NaN, -1
        args = {"cu_tokens": cu, "counts": out["counts"].t, "prob": out["prob"].t,
                "loss": out["loss"].t, "workspace": ws}
    mx.moe_router(c, rc, z, bias, out["ids"].t, out["gates"].t, **args)
    torch.cuda.synchronize()
    for g in out.values():
        g.check()
    got = {k: g.t.cpu().numpy() for k, g in out.items()}
    got["ids"] = got["ids"].reshape(T, c.K)
    got["gates"] = got["gates"].reshape(T, c.K)
    if stats:
        got["counts"] = got["counts"].reshape(rc.nseq, c.E)
        got["prob"] = got["prob"].reshape(rc.nseq, c.E)
    return got


def make_logits(T, E, bf16, seed, scale=1.0):
    g = np.random.default_rng(seed)
    z = (scale * g.standard_normal((T, E))).astype(np.float32)
    t = torch.from_numpy(z)
    if bf16:
        t = t.to(torch.bfloat16)
    return t, t.to(torch.float64).numpy()


def cuts(T, nseq, seed, head=0, tail=0):
    g = np.random.default_rng(seed)
    c = np.sort(g.integers(head, max(head, T - tail) + 1, nseq + 1)).astype(np.int32)
    if nseq == 1 and not head and not tail:
        c[:] = [0, T]
    return c


def check_forward(z, bias, got, c, rc, cu):
    ids = O.choose(z, bias, c.K, rc.score)
    assert np.array_equal(got["ids"], ids)
    zk = np.take_along_axis(z, ids, 1)
    want = rc.scale * O.gate_shares(z, ids, rc.score, bool(rc.renormalize))
    rel = rel_of(zk if rc.renormalize else z, rc.score)
    scale = abs(rc.scale)
    assert np.all(np.abs(got["gates"] - want) <= rel * np.abs(want) + scale * TINY_ABS)
    if "loss" not in got:
        return ids
    counts, prob, loss = O.balance(z, ids, cu, rc.score)
    assert np.array_equal(got["counts"], counts)
    check_sums(z, got, c, rc, prob, loss)
    return ids


def check_sums(z, got, c, rc, prob, loss):
    T = c.R * c.S
    chunk = 8 * -(-T // 4096)
    r = float(rel_of(z, rc.score).max(initial=0)) + (chunk / 8 + 8) * h
    assert np.all(np.abs(got["prob"] - prob) <= r * prob + TINY_ABS)
    assert np.all(np.abs(got["loss"] - loss) <= (r + 8 * h) * loss + TINY_ABS)


def check_backward(z, got, want, size, score, bf16):
    rel = 3 * rel_of(z, score) + 48 * h
    tol = rel * size + 2 * TINY_ABS
    if bf16:
        tol = tol + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


def run_backward(c, rc, z, ids, dgates, cu, counts, dloss):
    T = c.R * c.S
    out = Guarded(T * c.E, z.dtype)
    mx.moe_router_backward(c, rc, z, ids, dgates, cu, counts, dloss, out.t)
    torch.cuda.synchronize()
    out.check()
    return out.t.to(torch.float64).cpu().numpy().reshape(T, c.E)


SHAPES = [  # R, S, E, K, nseq
    (1, 1, 1, 1, 1), (1, 1, 8, 8, 3), (2, 3, 8, 3, 2), (1, 33, 7, 2, 5), (1, 5, 65, 64, 2),
    (3, 11, 129, 5, 9), (8, 9, 384, 8, 4), (4, 13, 520, 12, 70), (1, 9, 897, 16, 1),
    (2, 8, 1280, 3, 2), (1, 6, 2048, 64, 2), (1, 5, 2047, 40, 3), (8, 520, 64, 4, 37),
    # rows that fill the lanes, of every register count, and rows that nearly do
    (1, 19, 128, 6, 3), (1, 9, 256, 4, 2), (2, 5, 512, 4, 1), (1, 9, 768, 5, 2), (1, 5, 896, 16, 3),
    (1, 7, 1024, 8, 2), (1, 4, 1023, 9, 2), (1, 6, 702, 33, 2), (1, 3, 1536, 2, 1),
    # more sequences than 512, most of them of a token or none
    (1, 700, 130, 4, 600), (1, 90, 1100, 3, 520),
    # the least experts of every register count, even and odd
    (1, 3, 2, 2, 1), (1, 9, 130, 4, 2), (1, 9, 258, 4, 2), (1, 7, 386, 6, 2), (1, 7, 514, 6, 2),
    (1, 5, 770, 7, 2), (1, 5, 898, 7, 2), (1, 5, 1026, 7, 2), (1, 5, 1282, 7, 2),
    (1, 5, 257, 4, 2), (1, 5, 513, 6, 2), (1, 3, 769, 5, 2), (1, 3, 1025, 5, 2), (1, 3, 1281, 5, 2),
]


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, score, bf16):
    R, S, E, K, nseq = shape
    T = R * S
    announce("router", shape, score, bf16)
    c = cfg_of(R, S, E, K)
    zt, z = make_logits(T, E, bf16, 31 + E, 2.0)
    zg = zt.cuda()
    g = np.random.default_rng(E + T)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    dg = g.standard_normal((T, K)).astype(np.float32)
    dl = g.standard_normal(nseq).astype(np.float32)
    for renorm in (0, 1):
        for b in (None, bias):
            rc = mx.make_router_cfg(score, renorm, 2.5, bf16, nseq)
            cu = cuts(T, nseq, E + renorm, head=min(2, T - 1) if nseq > 3 else 0,
                      tail=1 if nseq > 1 and T > 3 else 0)
            cug = on_gpu(cu, torch.int32)
            bg = None if b is None else on_gpu(b, torch.float32)
            ids = check_forward(z, b, run_forward(c, rc, zg, bg, cug, True), c, rc, cu)
            check_forward(z, b, run_forward(c, rc, zg, bg, None, False), c, rc, None)
            counts = O.balance(z, ids, cu, score)[0]
            idg, cg = on_gpu(ids, torch.int32), on_gpu(counts, torch.int32)
            for use_g, use_l in ((1, 1), (1, 0), (0, 1)):
                want, size = O.backward(z, ids, score, bool(renorm), 2.5, dg if use_g else None,
                                        cu, counts, dl if use_l else None)
                if use_g and not use_l:
                    args = (idg, on_gpu(dg, torch.float32), None, None, None)
                elif use_l and not use_g:
                    args = (None, None, cug, cg, on_gpu(dl, torch.float32))
                else:
                    args = (idg, on_gpu(dg, torch.float32), cug, cg, on_gpu(dl, torch.float32))
                check_backward(z, run_backward(c, rc, zg, *args), want, size, score, bf16)


@pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID], ids=["softmax", "sigmoid"])
def test_masks_ties_and_extremes(score):
    """Masked experts, rows of nothing, equal logits, zeros of both signs, far logits."""
    E, K = 24, 6
    inf = np.inf
    g = np.random.default_rng(3)
    rows = [np.full(E, -inf), np.full(E, np.float32(-3.4028235e38)), np.full(E, 7.0), np.zeros(E)]
    for live in (1, 3, K, K + 1):                          # fewer live experts than K, and just
        r = np.full(E, -inf)
        r[g.permutation(E)[:live]] = g.standard_normal(live)
        rows.append(r)
    low = np.full(E, np.float32(-3.4028235e38))             # masks of the type's lowest value
    low[[5, 11]] = [0.5, 0.25]
    rows.append(low)
    rows.append(np.where(g.random(E) < 0.5, 0.0, -0.0))
    rows.append(np.repeat(g.standard_normal(E // 4), 4))    # ties of four
    rows.append(g.standard_normal(E) * 1e4)
    rows.append(g.standard_normal(E) - 200.0)               # every sigmoid underflows
    rows.append(g.standard_normal(E) + 200.0)               # every sigmoid is 1
    rows.append(np.linspace(-80, -40, E))                   # either side of the sigmoid's switch
    rows.append(np.linspace(-1, 1, E) * np.float32(3e38))
    z = np.array(rows, np.float32)
    T = len(rows)
    c = cfg_of(1, T, E, K)
    cu = np.array([0, 1, T - 2, T], np.int32)
    dg = g.standard_normal((T, K)).astype(np.float32)
    dl = g.standard_normal(3).astype(np.float32)
    bias = (0.3 * g.standard_normal(E)).astype(np.float32)
    bias[3], bias[4] = 50.0, -50.0
    for renorm, b in ((0, None), (1, None), (0, bias), (1, np.zeros(E, np.float32))):
        rc = mx.make_router_cfg(score, renorm, 1.0, False, 3)
        z64 = z.astype(np.float64)
        got = run_forward(c, rc, on_gpu(z, torch.float32),
                          None if b is None else on_gpu(b, torch.float32),
                          on_gpu(cu, torch.int32), True)
        ids = check_forward(z64, b, got, c, rc, cu)
        assert np.isfinite(got["gates"]).all() and np.all(got["gates"][0] == 0)
        counts = O.balance(z64, ids, cu, score)[0]
        want, size = O.backward(z64, ids, score, bool(renorm), 1.0, dg, cu, counts, dl)
        b = run_backward(c, rc, on_gpu(z, torch.float32), on_gpu(ids, torch.int32),
                         on_gpu(dg, torch.float32), on_gpu(cu, torch.int32),
                         on_gpu(counts, torch.int32), on_gpu(dl, torch.float32))
        check_backward(z64, b, want, size, score, False)
        assert np.all(b[0] == 0)                            # a row of nothing has no gradient


@pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID], ids=["softmax", "sigmoid"])
def test_nan_and_infinite_logits(score):
    """Ids stay K distinct experts; what NaN enters is NaN, other rows are untouched."""
    E, K, T = 40, 5, 8
    g = np.random.default_rng(9)
    z = g.standard_normal((T, E)).astype(np.float32)
    z[1, 7] = np.nan
    z[3] = np.nan
    z[4, 1:] = np.nan
    z[5, 9] = np.inf
    z[6, ::2] = np.nan
    c = cfg_of(1, T, E, K)
    rc = mx.make_router_cfg(score, 0, 1.0, False, 1)
    for b in (None, np.zeros(E, np.float32)):
        got = run_forward(c, rc, on_gpu(z, torch.float32),
                          None if b is None else on_gpu(b, torch.float32), None, True)
        for t in range(T):
            assert len(set(got["ids"][t])) == K and got["ids"][t].min() >= 0
            assert got["ids"][t].max() < E
        clean = [0, 2, 7]
        z64 = z.astype(np.float64)
        ids = O.choose(z64, b, K, score)
        assert np.array_equal(got["ids"][clean], ids[clean])
        assert np.isfinite(got["gates"][clean]).all()
        if b is None or score == O.SIGMOID:
            assert np.array_equal(got["ids"], ids)
        if score == O.SOFTMAX:
            assert np.isnan(got["gates"][[1, 3, 4, 6]]).all()
        assert np.isnan(got["loss"]).all() and np.isnan(got["prob"]).any()


@pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID], ids=["softmax", "sigmoid"])
def test_bias_orders_scores_nearer_than_fp32(score):
    """Scores plus bias that differ by far less than an fp32 step are ordered as float64 has
    them, at the border of the choice and inside it."""
    T, E, K = 64, 48, 4
    g = np.random.default_rng(17)
    z = g.standard_normal((T, E)).astype(np.float32)
    s = O.scores(z.astype(np.float64), score)[0]
    # biases that bring six experts of row 0 level at 1.5, then the same logits in every row
    z[:] = z[0]
    bias = np.zeros(E, np.float32)
    for i, e in enumerate((3, 9, 20, 21, 33, 47)):
        bias[e] = np.float32(1.5 - s[0, e])
    z[1:, 9] = np.nextafter(z[1:, 9], np.float32(9))        # one step in one logit
    z[T // 2:, 33] = np.nextafter(z[T // 2:, 33], np.float32(-9))
    key = O.scores(z.astype(np.float64), score)[0] + bias
    six = np.sort(key[:, [3, 9, 20, 21, 33, 47]], axis=1)
    assert np.diff(six, axis=1).max() < 2.0 ** -22          # level to fp32
    c = cfg_of(1, T, E, K)
    rc = mx.make_router_cfg(score, 1, 1.0, False, 1)
    got = run_forward(c, rc, on_gpu(z, torch.float32), on_gpu(bias, torch.float32), None, True)
    assert np.array_equal(got["ids"], O.choose(z.astype(np.float64), bias, K, score))


def test_saturated_sigmoids_with_bias():
    """Scores that round to 1 in fp32 and in float64: float64's order, then the lowest id."""
    E, K = 16, 5
    z = np.array([[20, 21, 18, 19, 30, 31, 60, 61, 70, 50, 45, 17, 16, 15, 14, 13]], np.float32)
    c = cfg_of(1, 1, E, K)
    rc = mx.make_router_cfg(O.SIGMOID, 1, 1.0, False, 1)
    bias = np.zeros(E, np.float32)
    got = run_forward(c, rc, on_gpu(z, torch.float32), on_gpu(bias, torch.float32), None, False)
    assert np.array_equal(got["ids"], O.choose(z.astype(np.float64), bias, K, O.SIGMOID))


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_given_ids(bf16):
    """moe_balance_loss with repeated ids and ids outside the experts; gradient likewise."""
    T, E, K, nseq = 77, 30, 4, 6
    g = np.random.default_rng(23)
    zt, z = make_logits(T, E, bf16, 5)
    ids = g.integers(-2, E + 2, (T, K)).astype(np.int32)
    ids[:, 1] = ids[:, 0]
    ids[5], ids[6] = 2 ** 31 - 1, -2 ** 31
    cu = cuts(T, nseq, 4, head=3, tail=5)
    for score in (O.SOFTMAX, O.SIGMOID):
        c = cfg_of(1, T, E, K)
        rc = mx.make_router_cfg(score, 1, 1.0, bf16, nseq)
        counts, prob, loss = (Guarded(nseq * E, torch.int32), Guarded(nseq * E, torch.float32),
                              Guarded(nseq, torch.float32))
        ws = torch.full((mx.moe_router_workspace_size(c, rc),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        idg, cug = on_gpu(ids, torch.int32), on_gpu(cu, torch.int32)
        mx.moe_balance_loss(c, rc, zt.cuda(), idg, cug, counts.t, prob.t, loss.t, ws)
        torch.cuda.synchronize()
        for o in (counts, prob, loss):
            o.check()
        wc, wp, wl = O.balance(z, ids, cu, score)
        assert np.array_equal(counts.t.cpu().numpy().reshape(nseq, E), wc)
        check_sums(z, {"prob": prob.t.cpu().numpy().reshape(nseq, E), "loss": loss.t.cpu().numpy()},
                   c, rc, wp, wl)
        dg = g.standard_normal((T, K)).astype(np.float32)
        dl = g.standard_normal(nseq).astype(np.float32)
        # without repeats: K distinct experts are what the gates' gradient is defined for
        only = ids.copy()
        only[:, 1] = -1
        for renorm in (0, 1):
            rc = mx.make_router_cfg(score, renorm, 1.5, bf16, nseq)
            ok = only.copy()
            for t in range(T):
                _, first = np.unique(ok[t], return_index=True)
                ok[t, [k for k in range(K) if k not in first]] = -1
            want, size = O.backward(z, ok, score, bool(renorm), 1.5, dg, cu, wc, dl)
            b = run_backward(c, rc, zt.cuda(), on_gpu(ok, torch.int32), on_gpu(dg, torch.float32),
                             cug, on_gpu(wc, torch.int32), on_gpu(dl, torch.float32))
            check_backward(z, b, want, size, score, bf16)


def test_gradient_in_place_and_large_batch():
    """dlogits over logits, at a size where every wave walks several tokens."""
    R, S, E, K, nseq = 8, 4100, 96, 6, 11
    T = R * S
    zt, z = make_logits(T, E, False, 8)
    c = cfg_of(R, S, E, K)
    rc = mx.make_router_cfg(O.SOFTMAX, 1, 1.0, False, nseq)
    cu = cuts(T, nseq, 1, tail=9)
    zg, cug = zt.cuda(), on_gpu(cu, torch.int32)
    got = run_forward(c, rc, zg, None, cug, True)
    ids = check_forward(z, None, got, c, rc, cu)
    g = np.random.default_rng(2)
    dg = g.standard_normal((T, K)).astype(np.float32)
    dl = g.standard_normal(nseq).astype(np.float32)
    want, size = O.backward(z, ids, O.SOFTMAX, True, 1.0, dg, cu, got["counts"], dl)
    args = (on_gpu(ids, torch.int32), on_gpu(dg, torch.float32), cug,
            on_gpu(got["counts"], torch.int32), on_gpu(dl, torch.float32))
    apart = run_backward(c, rc, zg, *args)
    check_backward(z, apart, want, size, O.SOFTMAX, False)
    mx.moe_router_backward(c, rc, zg, *args, zg)
    torch.cuda.synchronize()
    assert np.array_equal(zg.double().cpu().numpy(), apart)
    # the same inputs give the same bits
    zg = zt.cuda()
    again = run_forward(c, rc, zg, None, cug, True)
    for k in got:
        assert np.array_equal(got[k], again[k]), k


def test_gradient_against_differences():
    """Central differences of the kernels' own loss and gates, on a few logits.

    The loss is fp32: its steps of h0 = 2^-5 leave a rounding of about
    2^-24 * 2 / (2 h0) of the value per term and a curvature of h0^2 / 6 of the
    third derivative, below 2^-10 of the largest term together.
    """
    T, E, K = 6, 12, 3
    zt, z = make_logits(T, E, False, 44)
    c = cfg_of(1, T, E, K)
    rc = mx.make_router_cfg(O.SIGMOID, 1, 1.0, False, 2)
    cu = on_gpu(np.array([0, 2, 6], np.int32), torch.int32)
    g = np.random.default_rng(7)
    dg = g.standard_normal((T, K)).astype(np.float32)
    dl = g.standard_normal(2).astype(np.float32)
    got = run_forward(c, rc, zt.cuda(), None, cu, True)
    ids = on_gpu(got["ids"], torch.int32)
    dz = run_backward(c, rc, zt.cuda(), ids, on_gpu(dg, torch.float32), cu,
                      on_gpu(got["counts"], torch.int32), on_gpu(dl, torch.float32))

    def value(a):
        o = run_forward(c, rc, torch.from_numpy(a).cuda(), None, cu, True)
        if not (np.array_equal(o["ids"], got["ids"])):
            return None
        return float((o["gates"].astype(np.float64) * dg).sum() + (o["loss"] * dl.astype(np.float64)).sum())

    h0, seen = 2.0 ** -5, 0
    for t in range(T):
        for e in range(0, E, 3):
            a, b = zt.numpy().copy(), zt.numpy().copy()
            a[t, e] += np.float32(h0)
            b[t, e] -= np.float32(h0)
            va, vb = value(a), value(b)
            if va is None or vb is None:                    # the step changes the choice
                continue
            seen += 1
            width = float(a[t, e]) - float(b[t, e])
            assert abs((va - vb) / width - dz[t, e]) < 2.0 ** -9
    assert seen > 10


def test_no_tokens():
    c = cfg_of(2, 0, 8, 2)
    rc = mx.make_router_cfg(O.SOFTMAX, 1, 1.0, False, 2)
    z = torch.empty((0, 8), device="cuda")
    got = run_forward(c, rc, z, None, torch.zeros(3, dtype=torch.int32, device="cuda"), True)
    assert not got["counts"].any() and not got["prob"].any() and not got["loss"].any()
    mx.moe_router_backward(c, rc, z, torch.empty(0, dtype=torch.int32, device="cuda"),
                           torch.empty(0, device="cuda"), None, None, None, z)


def test_rows_of_one_wave_in_any_order():
    """The bound that a wave's last row left behind must not matter: rows of far apart sizes
    and signs follow each other, many more than waves."""
    g = np.random.default_rng(29)
    E, K, T = 128, 8, 1024 * 40
    z = g.standard_normal((T, E)).astype(np.float32)
    z *= (10.0 ** g.integers(-30, 31, (T, 1))).astype(np.float32)
    z += (g.integers(-1, 2, (T, 1)) * 10.0 ** g.integers(-10, 30, (T, 1))).astype(np.float32)
    z[g.random(T) < 0.05] = -np.inf
    z[g.random(T) < 0.05] = 0.0
    c = cfg_of(8, T // 8, E, K)
    rc = mx.make_router_cfg(O.SOFTMAX, 1, 1.0, False, 1)
    got = run_forward(c, rc, on_gpu(z, torch.float32), None, None, True)
    assert np.array_equal(got["ids"], O.choose(z.astype(np.float64), None, K, O.SOFTMAX))
    bias = np.zeros(E, np.float32)
    few = slice(0, 4096)
    c = cfg_of(8, 512, E, K)
    for score in (O.SOFTMAX, O.SIGMOID):
        rc = mx.make_router_cfg(score, 1, 1.0, False, 1)
        got = run_forward(c, rc, on_gpu(z[few], torch.float32), on_gpu(bias, torch.float32), None,
                          True)
        want = O.choose(z[few].astype(np.float64), bias, K, score)
        # Scores in float64 come from an exponential, a sum or 1 + x, and a division, each off
        # by an ulp or two (2^-52): where neighbours among the K + 1 largest are nearer than
        # 8 * 2^-52 of the score without being equal logits, float64 itself has no order, and
        # only the chosen scores are compared.
        s = O.scores(z[few].astype(np.float64), score)[0]
        more = O.choose(z[few].astype(np.float64), bias, K + 1, score)
        sk = np.take_along_axis(s, more, 1)
        zk = np.take_along_axis(z[few], more, 1)
        near = (sk[:, :-1] - sk[:, 1:] <= 8 * 2.0 ** -52 * sk[:, :-1]) & (zk[:, :-1] != zk[:, 1:])
        clear = ~near.any(axis=1)
        assert clear.mean() > 0.5
        assert np.array_equal(got["ids"][clear], want[clear])
        sg = np.take_along_axis(s, got["ids"], 1)
        assert np.all(np.abs(sg - sk[:, :-1]) <= 16 * 2.0 ** -52 * sk[:, :-1])


@pytest.mark.parametrize("E,K,bf16", [(2048, 8, False), (60, 3, True)])
def test_captured_calls_equal_eager(E, K, bf16):
    """Forward with the loss and backward captured once, replayed on new logits and sequences;
    2,048 experts take more LDS than a launch gets unasked."""
    R, S, nseq = 2, 150, 4
    T = R * S
    c = cfg_of(R, S, E, K)
    rc = mx.make_router_cfg(O.SIGMOID, 1, 1.5, bf16, nseq)
    dt = torch.bfloat16 if bf16 else torch.float32
    z, bias = torch.zeros((T, E), dtype=dt, device="cuda"), torch.zeros(E, device="cuda")
    cu = torch.zeros(nseq + 1, dtype=torch.int32, device="cuda")
    ids, gates = torch.zeros((T, K), dtype=torch.int32, device="cuda"), torch.zeros((T, K), device="cuda")
    counts, prob = torch.zeros((nseq, E), dtype=torch.int32, device="cuda"), torch.zeros((nseq, E), device="cuda")
    loss, dl, dg = torch.zeros(nseq, device="cuda"), torch.ones(nseq, device="cuda"), torch.ones((T, K), device="cuda")
    ws = torch.zeros(mx.moe_router_workspace_size(c, rc), dtype=torch.uint8, device="cuda")
    dz = torch.zeros_like(z)

    def step():
        mx.moe_router(c, rc, z, bias, ids, gates, cu, counts, prob, loss, ws)
        mx.moe_router_backward(c, rc, z, ids, dg, cu, counts, dl, dz)

    def out():
        torch.cuda.synchronize()
        return [t.clone() for t in (ids, gates, counts, prob, loss, dz.view(torch.int16) if bf16 else dz)]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2, 3):
        r = np.random.default_rng(seed)
        z.copy_(torch.from_numpy(r.standard_normal((T, E))))
        bias.copy_(torch.from_numpy(0.1 * r.standard_normal(E)))
        dg.copy_(torch.from_numpy(r.standard_normal((T, K))))
        cu.copy_(torch.from_numpy(cuts(T, nseq, seed, tail=5)))
        torch.cuda.synchronize()
        g.replay()
        a = out()
        step()
        b = out()
        g.replay()
        for x, y, w in zip(a, b, out()):
            assert torch.equal(x, y) and torch.equal(y, w)


def test_one_device(monkeypatch):
    c = cfg_of(1, 4, 8, 2)
    rc = mx.make_router_cfg(O.SOFTMAX, 1)
    z = torch.zeros((4, 8), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        mx.moe_router(c, rc, z, None, ids, torch.zeros((4, 2), device="cuda:0"))


def test_binding_refuses_wrong_tensors():
    c = cfg_of(1, 4, 8, 2)
    rc = mx.make_router_cfg(O.SOFTMAX, 1)
    z = torch.zeros((4, 8), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    gates = torch.zeros((4, 2), device="cuda")
    with pytest.raises(TypeError):
        mx.moe_router(c, rc, z.to(torch.bfloat16), None, ids, gates)
    with pytest.raises(TypeError):
        mx.moe_router(c, rc, z, None, ids.long(), gates)
    with pytest.raises(ValueError):
        mx.moe_router(c, rc, z.t(), None, ids, gates)
    with pytest.raises(ValueError):
        mx.moe_router(c, rc, z[:3], None, ids, gates)
    with pytest.raises(ValueError):
        mx.moe_router(c, rc, z.cpu(), None, ids, gates)
    with pytest.raises(ValueError):
        mx.moe_router(c, rc, z, torch.zeros(7, device="cuda"), ids, gates)
    with pytest.raises(mx.MoeError) as e:                   # loss without counts
        mx.moe_router(c, rc, z, None, ids, gates, loss=torch.zeros(1, device="cuda"),
                      workspace=torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == mx.MOE_EINVAL
