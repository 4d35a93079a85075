"""Dropout alone and around the combine, and the combine's gradients through it, against the
oracle.

Tolerances, with h = 2^-24 and R = 2^-8 (half a step of fp32 and bf16): dropout is one product
by a rounded factor and one addition, 2 h |v| f + h |out|, and the output's rounding.  The sum
over K routes adds 2 (K + 1) h sum |g y|.  dy: two products, 3 h, and its rounding; dgates: a
lane adds 8 products per group and at most Hp / 512 + 1 groups, seven additions join the lanes
and one each pass: 2 (Hp / 64 + 32) h sum |d y|.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import workloads as W
from epilogue_checks import R, close, h, round_tol
from gpu_helpers import announce, cfgs, free, gpu_plan
from oracle import epilogue as O
from test_gpu_epilogue import Out, f64, normal, rng_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


def dtype_of(f32):
    return torch.float32 if f32 else torch.bfloat16


@pytest.mark.parametrize("rows,width", [(1, 8), (3, 1000), (8, 7168), (257, 520), (4099, 72), (1, 40000), (20000, 8)])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True], ids=["alone", "residual"])
def test_dropout(rows, width, f32, residual):
    announce("dropout", rows, width, f32, residual)
    for p in (0.0, 0.1, 0.5, 1.0):
        src = normal(rows, f32, rows, width)
        res = normal(rows + 1, f32, rows, width) if residual else None
        rng = rng_of(-rows, width << 32)
        out = Out(rows, width, dtype_of(f32))
        dc = mx.make_dropout_cfg(p, f32)
        mx.moe_dropout(dc, rows, width, src, res, rng if p else None, out.t)
        torch.cuda.synchronize()
        out.check()
        f = O.row_factor(p, rng.tolist(), np.arange(rows), width)
        v = f64(src) * f
        want = v + (f64(res) if residual else 0)
        close(f64(out.t), want, (1 + R) * (2 * h * np.abs(v) + h * np.abs(want)) + round_tol(want, f32), "dst")
        assert np.all(f64(out.t)[f == 0] == (f64(res)[f == 0] if residual else 0))
        # in place on either tensor: the same bits
        for which in ("src", "residual")[:1 + residual]:
            a, b = src.clone(), None if res is None else res.clone()
            dst = a if which == "src" else b
            mx.moe_dropout(dc, rows, width, a, b, rng, dst)
            torch.cuda.synchronize()
            assert torch.equal(dst, out.t)


def test_dropout_is_its_own_backward():
    """<dropout(u), v> = <u, dropout(v)>: fp32, sums in 64 bits; each value two roundings off."""
    rows, width = 100, 520
    u, v, rng = normal(1, True, rows, width), normal(2, True, rows, width), rng_of(4, 5)
    du, dv = torch.empty_like(u), torch.empty_like(v)
    dc = mx.make_dropout_cfg(0.3, True)
    mx.moe_dropout(dc, rows, width, u, None, rng, du)
    mx.moe_dropout(dc, rows, width, v, None, rng, dv)
    torch.cuda.synchronize()
    a, b = (f64(du) * f64(v)), (f64(u) * f64(dv))
    assert np.abs(a - b).max() <= 4 * h * np.abs(a).max() and 0.25 < (a == 0).mean() < 0.35


def test_dropped_values_are_zero_whatever_they_were():
    src = torch.full((64, 64), float("inf"), device="cuda")
    src[1::2] = float("nan")
    rng, dst = rng_of(1, 1), torch.empty_like(src)
    mx.moe_dropout(mx.make_dropout_cfg(0.5, True), 64, 64, src, None, rng, dst)
    torch.cuda.synchronize()
    f = O.row_factor(0.5, [1, 1], np.arange(64), 64)
    got = f64(dst)
    assert np.all(got[f == 0] == 0)
    assert np.all(np.isinf(got[0::2][f[0::2] > 0])) and np.all(np.isnan(got[1::2][f[1::2] > 0]))


def test_dropout_past_32_bits():
    rows, width = (1 << 31) // 4096 + 33, 4096
    src, rng = torch.full((rows, width), 1.0, dtype=torch.bfloat16, device="cuda"), rng_of(3, 1 << 62)
    mx.moe_dropout(mx.make_dropout_cfg(0.5), rows, width, src, None, rng, src)
    torch.cuda.synchronize()
    mid = (1 << 31) // width
    at = np.concatenate([np.arange(3), np.arange(mid - 2, mid + 2), np.arange(rows - 3, rows)])
    assert np.array_equal(f64(src.index_select(0, torch.from_numpy(at).cuda())),
                          O.row_factor(0.5, [3, 1 << 62], at, width))
    share = float((src == 0).sum().item()) / src.numel()
    assert abs(share - 0.5) <= 5 * 0.5 / src.numel() ** 0.5


def plan_of(shape, ids="uniform"):
    picked = (W.routing_hot(shape) if ids == "hot" else W.routing_uniform(shape, 4)[0]).copy()
    if ids == "failed":
        picked[0, 0] = shape.E
    if ids == "twice":
        picked[::3, 1] = picked[::3, 0]
    return gpu_plan(shape, picked)


@pytest.mark.parametrize("ids", ["uniform", "hot", "failed", "twice"])
@pytest.mark.parametrize("shape", [
    W.TINY, W.TINY.with_(S=125, Hp=1000), W.TINY.with_(S=1, Hp=8), W.TINY.with_(R=2, B=4, S=33, K=7, Hp=2056),
    W.TINY.with_(R=1, B=8, S=9, Hp=520), W.TINY.with_(S=5, Hp=1032), W.TINY.with_(R=1, B=8, S=3, Hp=4104),
    W.TINY.with_(R=1, B=8, S=2, Hp=8200), W.TINY.with_(R=1, B=0, mode=1, S=3, E=64, K=64, Hp=72)], ids=str)
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_combine(shape, ids, f32):
    if ids == "twice" and shape.K == 1:
        pytest.skip("one route a token")
    announce("combine", shape, ids, f32)
    c, _ = cfgs(shape)
    plan, v = plan_of(shape, ids)
    route = v["route"].astype(np.int64)
    T, K, Hp, rows = shape.tokens, shape.K, shape.Hp, shape.R * shape.SK
    y = normal(1, False, rows, Hp)
    gates = normal(2, True, T, K)
    gates[0, 0] = 0.0
    res, dout = normal(3, f32, T, Hp), normal(4, f32, T, Hp)
    yn, gn, rn, dn = f64(y), f64(gates), f64(res), f64(dout)
    for p, with_res in ((0.0, False), (0.1, True), (0.5, False), (1.0, True)):
        rng = rng_of(77, T)
        r = rng.tolist()
        dc = mx.make_dropout_cfg(p, f32)
        out = Out(T, Hp, dtype_of(f32))
        mx.moe_combine_dropout(c, dc, plan, y, gates, res if with_res else None, rng if p else None, out.t)
        dy, dg = Out(rows, Hp, torch.bfloat16), Out(T, K, torch.float32)
        mx.moe_combine_dropout_backward(c, dc, plan, dout, y, gates, rng if p else None, dy.t, dg.t)
        torch.cuda.synchronize()
        f = O.row_factor(p, r, np.arange(T), Hp)
        add = rn if with_res else None
        want = O.combine(yn, gn, route, p, r, add)
        mag = O.combine(np.abs(yn), np.abs(gn), route, p, r)
        out.check()
        close(f64(out.t), want, (1 + R) * (2 * (K + 3) * h * mag + h * np.abs(want)) + round_tol(want, f32), "out")
        gy, gg = O.combine_backward(dn, yn, gn, route, p, r)
        _, gmag = O.combine_backward(np.abs(dn), np.abs(yn), gn, route, p, r)
        dg.check()
        close(f64(dg.t), gg, 2 * (Hp / 64 + 32) * h * gmag, "dgates")
        live = route >= 0
        assert np.all(f64(dg.t).reshape(-1)[~live] == 0)
        got = f64(dy.t)
        where = route[live]
        flat = gy.reshape(T * K, Hp)[live]
        close(got[where], flat, (3 * h * (1 + R) + R) * np.abs(flat), "dy")
        rest = np.setdiff1d(np.arange(rows), where)
        dy.check(torch.from_numpy(rest).cuda())
        # in place: the sum over its residual, the gates' gradient over the gates
        if with_res:
            buf = res.clone()
            mx.moe_combine_dropout(c, dc, plan, y, gates, buf, rng if p else None, buf)
            torch.cuda.synchronize()
            assert torch.equal(buf, out.t)
        buf = gates.clone()
        mx.moe_combine_dropout_backward(c, dc, plan, dout, y, buf, rng if p else None, dy.t, buf)
        torch.cuda.synchronize()
        assert torch.equal(buf, dg.t)


def test_combine_without_dropout_is_combine():
    """bf16, p = 0, no residual: the sums of moe_combine, bit for bit; and its gradients' gates."""
    s = W.TINY.with_(S=64, Hp=1000)
    c, _ = cfgs(s)
    plan, _ = plan_of(s)
    y, gates = normal(1, False, s.R * s.SK, s.Hp), normal(2, True, s.tokens, s.K)
    a, b = (torch.empty((s.tokens, s.Hp), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mx.moe_combine(c, plan, y, gates, a)
    mx.moe_combine_dropout(c, mx.make_dropout_cfg(), plan, y, gates, None, None, b)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_binding_refuses():
    dc = mx.make_dropout_cfg(0.5)
    t = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    rng = rng_of(1, 1)
    with pytest.raises(TypeError):
        mx.moe_dropout(dc, 4, 64, t.float(), None, rng, t)
    with pytest.raises(TypeError):
        mx.moe_dropout(dc, 4, 64, t, None, rng.int(), t)
    with pytest.raises(ValueError):
        mx.moe_dropout(dc, 8, 64, t, None, rng, t)
    with pytest.raises(ValueError):
        mx.moe_dropout(dc, 4, 64, t, None, rng.cpu(), t)
    with pytest.raises(ValueError):
        mx.moe_dropout(dc, 4, 64, torch.zeros((64, 4), dtype=torch.bfloat16, device="cuda").t(), None, rng, t)
    with pytest.raises(mx.MoeError):
        mx.moe_dropout(dc, 4, 64, t, None, None, t)
