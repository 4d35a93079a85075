"""The router and the calls on codes where offsets pass 2^31 values.

The rows at the start, on either side of the border and at the end are compared with the oracle
or with calls whose tensors are small; the rest, equal by construction, on the GPU.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import test_gpu_q8 as Q
import test_gpu_router as R
import workloads as W
from gpu_helpers import announce, bits, free
from oracle import bf16, q8, swiglu
from oracle import router as O
from router_checks import check_gradient

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


@pytest.mark.parametrize("bf16_logits", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("score,use_bias", [(O.SOFTMAX, False), (O.SIGMOID, True)],
                         ids=["softmax", "sigmoid-bias"])
def test_router(score, use_bias, bf16_logits):
    """Rows of zeros but for a few; three sequences, of the first, the border and the last."""
    E, K, n = 514, 6, 3
    T = (1 << 31) // E + 1001
    announce("router past 2^31", T, E, score, bf16_logits)
    c = R.cfg_of(1, T, E, K)
    rc = mx.make_router_cfg(score, 1, 1.5, bf16_logits, n)
    dt = torch.bfloat16 if bf16_logits else torch.float32
    z = torch.zeros((T, E), dtype=dt, device="cuda")
    mid = (1 << 31) // E                                    # its row holds value 2^31
    spans = [(0, 9), (mid - 5, mid + 6), (T - 7, T)]
    rows = np.concatenate([np.arange(a, b) for a, b in spans])
    zt, zr = R.make_logits(len(rows), E, bf16_logits, 3, 2.0)
    z[torch.from_numpy(rows).cuda()] = zt.cuda()
    g = np.random.default_rng(4)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32) if use_bias else None
    bg = None if bias is None else R.on_gpu(bias, torch.float32)
    ids, gates = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    # the sequences in one call need ascending ends: tokens between them are sequences 1 and 3
    ends = np.array([0, 9, mid - 5, mid + 6, T - 7, T], np.int32)
    rc5 = mx.make_router_cfg(score, 1, 1.5, bf16_logits, 5)
    ws = torch.empty(mx.moe_router_workspace_size(c, rc5), dtype=torch.uint8, device="cuda")
    counts = torch.empty((5, E), dtype=torch.int32, device="cuda")
    prob, loss = torch.empty((5, E), device="cuda"), torch.empty(5, device="cuda")
    cu = R.on_gpu(ends, torch.int32)
    mx.moe_router(c, rc5, z, bg, ids, gates, cu, counts, prob, loss, ws)
    torch.cuda.synchronize()
    at = torch.from_numpy(rows).cuda()
    got = {"ids": ids[at].cpu().numpy(), "gates": gates[at].cpu().numpy()}
    want = O.choose(zr, bias, K, score)
    assert np.array_equal(got["ids"], want)
    zk = np.take_along_axis(zr, want, 1)
    rel = R.rel_of(zk, score)
    share = 1.5 * O.gate_shares(zr, want, score, True)
    assert np.all(np.abs(got["gates"] - share) <= rel * share + 2.0 ** -125)
    # rows of zeros: the same K experts, gates of 1.5 / K
    same = O.choose(np.zeros((1, E)), bias, K, score)[0]
    off = torch.ones(T, dtype=torch.bool, device="cuda")
    off[at] = False
    rest = (ids == torch.from_numpy(same).cuda()).all(1) & (gates - 1.5 / K).abs().le(1e-6).all(1)
    assert bool((rest | ~off).all())
    cn, first = counts.cpu().numpy(), 0
    for q, (a, b) in zip((0, 2, 4), spans):
        part = slice(first, first + b - a)
        first += b - a
        wc, wp, wl = O.balance(zr[part], want[part], [0, b - a], score)
        assert np.array_equal(cn[q], wc[0])
        R.check_sums(zr[part], {"prob": prob[q:q + 1].cpu().numpy(), "loss": loss[q:q + 1].cpu().numpy()},
                     c, rc, wp, wl)
    # Equal shares: sum f / E = 1.  The module tests/test_gpu_router.py derives the bound: a share
    # is off by (5 X + 48) h with X = 15, a wave adds chunk / 8 of them, here ceil(T / 4096) =
    # 1,021, each addition off by h at most (and by the same amount where all terms are equal),
    # 8 waves and the loss's own roundings 16 more.
    far = (5 * 15 + 48 + -(-T // 4096) + 16) * R.h
    for q, m in ((1, mid - 14), (3, T - mid - 13)):
        flat = np.zeros(E, np.int64)
        flat[same] = m
        assert np.array_equal(cn[q], flat)
        assert abs(loss[q].item() - 1.0) <= far
    dg = g.standard_normal((len(rows), K)).astype(np.float32)
    dl = np.array([1.5, 0, -2.0, 0, 0.5], np.float32)
    dgates = torch.zeros((T, K), device="cuda")
    dgates[at] = torch.from_numpy(dg).cuda()
    mx.moe_router_backward(c, rc5, z, ids, dgates, cu, counts, R.on_gpu(dl, torch.float32), z)
    torch.cuda.synchronize()
    dz, first = z[at].double().cpu().numpy(), 0
    for q, (a, b) in zip((0, 2, 4), spans):
        part = slice(first, first + b - a)
        first += b - a
        w, size = O.backward(zr[part], want[part], score, True, 1.5, dg[part], [0, b - a],
                             cn[q:q + 1], dl[q:q + 1])
        check_gradient(R.rel_of(zr[part], score), dz[part], w, size, bf16_logits)
    assert bool(((z == 0).all(1) | ~off).all())


def test_dispatch_and_combine():
    """65,536 tokens of 7,168 and of 4,104 values to 8 places each: 3.8 and 2.2 G values."""
    R_, S, E, K = 8, 8192, 64, 8
    T = R_ * S
    gen = torch.Generator(device="cuda").manual_seed(5)
    route = torch.randperm(T * K, generator=gen, device="cuda").to(torch.int32)

    def planned(H, Hp):
        c = mx.make_cfg(R_, S, E, K, H, Hp, 0, mx.MODE_INFER)
        plan = mx.Plan(c)
        plan.route.copy_(route)
        return c, plan

    def codes(rows, width):
        q = torch.empty((rows, width), dtype=torch.uint8, device="cuda")
        for lo in range(0, rows, 1 << 16):                  # no NaN codes: 0 .. 119 and signs
            part = q[lo:lo + (1 << 16)]
            part.random_(0, 120, generator=gen)
            part[:, ::3] += 128
        s = torch.empty((rows, Q.blocks(width)), dtype=torch.uint8, device="cuda")
        return q, s.random_(110, 130, generator=gen)

    announce("dispatch past 2^31")
    c, plan = planned(7168, 8)
    xq, xs = codes(T, 7168)
    x = torch.empty((T, 7168), dtype=torch.bfloat16, device="cuda")
    xp = torch.empty((T * K, 7168), dtype=torch.bfloat16, device="cuda")
    mx.moe_q8_load(T, 7168, xq, xs, x)
    mx.moe_dispatch_q8(c, plan, xq, xs, xp)
    torch.cuda.synchronize()
    at = route.long().view(T, K)
    for lo in range(0, T, 4096):
        for k in range(K):
            assert torch.equal(xp[at[lo:lo + 4096, k]].view(torch.int16), x[lo:lo + 4096].view(torch.int16))
    del xp, x, xq, xs
    free()
    announce("combine past 2^31")
    Hp = 4104
    c, plan = planned(8, Hp)
    yq, ys = codes(T * K, Hp)
    y = torch.empty((T * K, Hp), dtype=torch.bfloat16, device="cuda")
    mx.moe_q8_load(T * K, Hp, yq, ys, y)
    dout = torch.randn((T, Hp), generator=gen, device="cuda").to(torch.bfloat16)
    gates = torch.rand((T, K), generator=gen, device="cuda")
    dy, dg = torch.empty((T * K, Hp), dtype=torch.bfloat16, device="cuda"), torch.empty((T, K), device="cuda")
    mx.moe_combine_backward_q8(c, plan, dout, yq, ys, gates, dy, dg)
    torch.cuda.synchronize()
    h = 2.0 ** -24
    for lo in range(0, T, 4096):
        d = dout[lo:lo + 4096].double()
        for k in range(K):
            r = at[lo:lo + 4096, k]
            # a float64 product of 8 and 24 bits is exact, and so is its distance from dy: half a
            # bf16 step at most (torch's cast from float64 passes through float32 and rounds twice)
            want = d * gates[lo:lo + 4096, k:k + 1].double()
            step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -126))) - 7)
            assert bool(((dy[r].double() - want).abs() <= step / 2).all())
            terms = d * y[r].double()
            tol = (Hp / 64 + 16) * h * terms.abs().sum(1)
            assert bool(((dg[lo:lo + 4096, k].double() - terms.sum(1)).abs() <= tol).all())


def test_swiglu_backward():
    """524,288 rows of 2 x 2,056 values, all alike but those at the border and the ends."""
    R_, S, E, K, Hp = 8, 8192, 64, 8, 2056
    rows = R_ * S * K
    announce("swiglu backward past 2^31")
    c = mx.make_cfg(R_, S, E, K, 8, Hp, 0, mx.MODE_INFER)
    mid = (1 << 31) // (2 * Hp)
    pick = [0, 1, mid - 1, mid, mid + 1, rows - 2, rows - 1]
    h13, d = Q.activations(len(pick), 2 * Hp, 31), Q.activations(len(pick), Hp, 32)
    hq, hs = q8.store(h13.reshape(2 * len(pick), Hp))
    q = torch.full((rows, 2 * Hp), 0x38, dtype=torch.uint8, device="cuda")       # 1.0
    s = torch.full((rows, 2 * Q.blocks(Hp)), 127, dtype=torch.uint8, device="cuda")
    dact = torch.ones((rows, Hp), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor(pick, device="cuda")
    q[at] = torch.from_numpy(hq.reshape(len(pick), -1)).cuda()
    s[at] = torch.from_numpy(hs.reshape(len(pick), -1)).cuda()
    dact[at] = W.from_bits(d, "cuda")
    dh = torch.empty((rows, 2 * Hp), dtype=torch.bfloat16, device="cuda")
    mx.moe_swiglu_backward_q8(c, q, s, dact, dh, dact)
    torch.cuda.synchronize()
    kept = q8.load(hq, hs).reshape(len(pick), 2 * Hp)
    g, u, df = kept[:, :Hp], kept[:, Hp:], bf16.bits_to_f64(d)
    want = np.concatenate(swiglu.swiglu_backward_f64(g, u, df), 1)
    got = bf16.bits_to_f64(bits(dh[at]))
    assert np.all(np.abs(got - want) <= Q.swiglu_tolerance(g, u, df, want))
    act = swiglu.silu(g) * u
    tol = (4 * np.minimum(np.abs(g), 200) + 40) * 2.0 ** -24 * np.abs(act) + 2.0 ** -8 * np.abs(act) + \
        2.0 ** -126 * (1 + np.abs(g)) * (1 + np.abs(u))
    assert np.all(np.abs(bf16.bits_to_f64(bits(dact[at])) - act) <= tol)
    off = torch.ones(rows, dtype=torch.bool, device="cuda")
    off[at] = False
    assert bool(((dh[:, :Hp] == dh[2, 0]).all(1) | ~off).all()) and bool(((dh[:, Hp:] == dh[2, Hp]).all(1) | ~off).all())
    assert bool(((dact == dact[2, 0]).all(1) | ~off).all())
    one = 1 / (1 + np.exp(-1.0))
    assert abs(dh[2, 0].item() - one * (2 - one)) < 2.0 ** -7 and abs(dh[2, Hp].item() - one) < 2.0 ** -8
