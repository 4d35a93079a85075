"""Calls on codes: tensors that lie next to each other or may share memory, scales that no store
writes, and the same call again."""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import test_gpu_q8 as Q
import workloads as W
from gpu_helpers import bits, cfgs, free, gpu_plan
from oracle import bf16, q8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


def side_by_side(*parts):
    """Tensors of (n, dtype) cut from one allocation, each where the last one ends (on the next
    16-byte boundary)."""
    sizes = [-(-n * torch.empty((), dtype=d).element_size() // 16) * 16 for n, d in parts]
    raw = torch.zeros(sum(sizes), dtype=torch.uint8, device="cuda")
    out, at = [], 0
    for (n, d), size in zip(parts, sizes):
        out.append(raw[at:at + n * torch.empty((), dtype=d).element_size()].view(d))
        at += size
    return out


# one wave a token, and four
@pytest.mark.parametrize("shape", [W.TINY.with_(Hp=40, S=37), W.TINY.with_(Hp=1032, S=19)],
                         ids=["H40", "H1032"])
def test_combine_backward_in_place_and_side_by_side(shape):
    c, _ = cfgs(shape)
    ids, gates = W.routing_uniform(shape, salt=5)
    plan, _ = gpu_plan(shape, ids)
    rows, T, K, Hp = shape.R * shape.SK, shape.tokens, shape.K, shape.Hp
    q0, s0 = Q.store(Q.activations(rows, Hp, 11))
    d0 = W.from_bits(Q.activations(T, Hp, 12), "cuda")
    g0 = torch.from_numpy(np.ascontiguousarray(gates)).cuda()
    dy0 = torch.zeros((rows, Hp), dtype=torch.bfloat16, device="cuda")
    dg0 = torch.zeros((T, K), device="cuda")
    mx.moe_combine_backward_q8(c, plan, d0, q0, s0, g0, dy0, dg0)
    d, dy, q, dg, s, g = side_by_side((T * Hp, torch.bfloat16), (rows * Hp, torch.bfloat16),
                                      (rows * Hp, torch.uint8), (T * K, torch.float32),
                                      (s0.numel(), torch.uint8), (T * K, torch.float32))
    for to, of in ((d, d0), (q, q0), (s, s0), (g, g0)):
        to.copy_(of.reshape(-1))
    mx.moe_combine_backward_q8(c, plan, d, q, s, g, dy, dg)
    torch.cuda.synchronize()
    assert torch.equal(dy.view(torch.int16), dy0.view(torch.int16).reshape(-1))
    assert torch.equal(dg, dg0.reshape(-1)) and torch.equal(g, g0.reshape(-1))
    dy.zero_()
    mx.moe_combine_backward_q8(c, plan, d, q, s, g, dy, g)  # dgates over gates
    torch.cuda.synchronize()
    assert torch.equal(dy.view(torch.int16), dy0.view(torch.int16).reshape(-1))
    assert torch.equal(g, dg0.reshape(-1))


def test_dispatch_side_by_side():
    shape = W.TINY.with_(H=72, Hp=40, S=37)
    c, _ = cfgs(shape)
    ids, _ = W.routing_uniform(shape, salt=2)
    plan, _ = gpu_plan(shape, ids)
    rows, H = shape.R * shape.SK, shape.H
    q0, s0 = Q.store(Q.activations(shape.tokens, H, 7))
    want = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    mx.moe_dispatch_q8(c, plan, q0, s0, want)
    q, xp, s = side_by_side((q0.numel(), torch.uint8), (rows * H, torch.bfloat16),
                            (s0.numel(), torch.uint8))
    q.copy_(q0)
    s.copy_(s0)
    mx.moe_dispatch_q8(c, plan, q, s, xp)
    torch.cuda.synchronize()
    assert torch.equal(xp.view(torch.int16), want.view(torch.int16).reshape(-1))


def test_projection_over_another_ranks_rows():
    """Rank 1's act may lie where rank 0's rows of xperm were; the other tensors side by side."""
    shape = W.TINY.with_(H=72, Hp=40, S=37)
    c, _ = cfgs(shape)
    ids, _ = W.routing_uniform(shape, salt=8)
    plan, _ = gpu_plan(shape, ids)
    rows, n, H, Hp, bf = shape.R * shape.SK, shape.SK, shape.H, shape.Hp, torch.bfloat16
    nb = Q.blocks(Hp)
    c13 = mx.make_cfg(shape.R, shape.S, shape.E, shape.K, H, 2 * Hp, shape.B, shape.mode)
    x = W.randn_bf16((shape.tokens, H), 1, "cuda")
    w = W.randn_bf16((shape.E, H, 2 * Hp), 2, "cuda")
    wp = torch.zeros((shape.R * shape.B, H, 2 * Hp), dtype=bf, device="cuda")
    ws0 = torch.empty(mx.moe_gemm_workspace_size(c), dtype=torch.uint8, device="cuda")
    mx.moe_prefetch_weight(c13, plan, w, wp)
    xp0 = torch.zeros((rows, H), dtype=bf, device="cuda")
    mx.moe_dispatch(c, plan, x, xp0)
    act0, q0, s0 = (torch.zeros(rows * Hp, dtype=bf, device="cuda"),
                    torch.zeros(rows * 2 * Hp, dtype=torch.uint8, device="cuda"),
                    torch.zeros(rows * 2 * nb, dtype=torch.uint8, device="cuda"))
    mx.moe_grouped_gemm_swiglu_q8(c, xp0, w, wp, plan.cu_seqlens, act0, q0, s0, 0, shape.R, ws0)
    both, q, ws, s = side_by_side((n * Hp + rows * H, bf), (rows * 2 * Hp, torch.uint8),
                                  (ws0.numel(), torch.uint8), (rows * 2 * nb, torch.uint8))
    xp, act = both[n * Hp:], both[:rows * Hp]
    assert n * Hp * 2 % 16 == 0 and Hp <= H
    xp.copy_(xp0.reshape(-1))
    mx.moe_grouped_gemm_swiglu_q8(c, xp, w, wp, plan.cu_seqlens, act, q, s, 1, 2, ws)
    torch.cuda.synchronize()
    part = slice(n * Hp, 2 * n * Hp)
    assert torch.equal(act[part].view(torch.int16), act0[part].view(torch.int16))
    assert torch.equal(q[n * 2 * Hp:2 * n * 2 * Hp], q0[n * 2 * Hp:2 * n * 2 * Hp])
    assert torch.equal(s[n * 2 * nb:2 * n * 2 * nb], s0[n * 2 * nb:2 * n * 2 * nb])


@pytest.mark.parametrize("shape", [W.TINY.with_(R=1, E=24, S=11, K=4, B=24, H=520, Hp=72),
                                   W.SKEWED.with_(S=256, Hp=520)], ids=["few-rows", "skewed"])
def test_projection_repeats_and_rounds_once(shape):
    """The same bits call after call, whatever its buffers held; and every gate and up that is
    kept is the bf16 next to the float64 product, but for the fp32 sum's own error.

    A sum of H exact products in fp32 is off by H h sum |x w| at most, in any order, and its
    rounding to bf16 by half a step, 2^-8 of the value.
    """
    c, _ = cfgs(shape)
    ids, _ = W.routing_uniform(shape, salt=3)
    plan, _ = gpu_plan(shape, ids)
    rows, H, Hp, E = shape.R * shape.SK, shape.H, shape.Hp, shape.E
    c13 = mx.make_cfg(shape.R, shape.S, E, shape.K, H, 2 * Hp, shape.B, shape.mode)
    w = W.randn_bf16((E, H, 2 * Hp), 2, "cuda")
    wp = torch.zeros((shape.R * shape.B, H, 2 * Hp), dtype=torch.bfloat16, device="cuda")
    xp = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mx.moe_gemm_workspace_size(c), dtype=torch.uint8, device="cuda")
    mx.moe_prefetch_weight(c13, plan, w, wp)
    mx.moe_dispatch(c, plan, W.randn_bf16((shape.tokens, H), 1, "cuda"), xp)
    act = torch.empty((rows, Hp), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((rows, 2 * Hp), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, 2 * Q.blocks(Hp)), dtype=torch.uint8, device="cuda")
    seen = []
    for soil in (0x00, 0xFF, 0x7F, 0x5A):
        for t in (act.view(torch.uint8), q, s, ws):
            t.fill_(soil)
        mx.moe_grouped_gemm_swiglu_q8(c, xp, w, wp, plan.cu_seqlens, act, q, s, 0, shape.R, ws)
        torch.cuda.synchronize()
        seen.append((act.view(torch.int16).clone(), q.clone(), s.clone()))
        assert all(torch.equal(a, b) for a, b in zip(seen[0], seen[-1]))
    h13 = torch.zeros((rows, 2 * Hp), dtype=torch.bfloat16, device="cuda")
    mx.moe_grouped_gemm_swiglu(c, xp, w, wp, plan.cu_seqlens, act, h13, 0, shape.R, ws)
    q0, s0 = Q.store(bits(h13).reshape(2 * rows, Hp))
    assert torch.equal(q.reshape(-1), q0) and torch.equal(s.reshape(-1), s0)
    v = {k: t.cpu().numpy() for k, t in plan.views().items()}
    cu, slot = v["cu_seqlens"].reshape(shape.R, -1), v["slot_expert"]
    some = 0
    for r in range(shape.R):
        for j in range(cu.shape[1] - 1):
            lo, hi = r * shape.SK + cu[r, j], r * shape.SK + cu[r, j + 1]
            if hi == lo:
                continue
            some += 1
            x, we = xp[lo:hi].double(), w[j if j < E else int(slot[r, j - E])].double()
            exact, size = x @ we, x.abs() @ we.abs()
            tol = 2.0 ** -8 * exact.abs() + 1.01 * H * 2.0 ** -24 * size
            assert bool(((h13[lo:hi].double() - exact).abs() <= tol).all())
    assert some > 10


def test_scales_that_no_store_writes():
    """Scale bytes 248 to 255 under every code: 2^121 to 2^127, and an infinite scale."""
    q = np.repeat(np.arange(256, dtype=np.uint8)[None], 8, axis=0)
    s = np.repeat(np.arange(248, 256, dtype=np.uint8)[:, None], 8, axis=1)
    out = torch.empty((8, 256), dtype=torch.bfloat16, device="cuda")
    mx.moe_q8_load(8, 256, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), out)
    torch.cuda.synchronize()
    got, want = bf16.bits_to_f64(bits(out)), q8.load(q, s)
    want[7] = np.where(want[7] == 0, np.nan, np.copysign(np.inf, want[7]))       # byte 255
    want[7, [127, 255]] = np.nan                            # NaN under any scale
    want[want >= 2.0 ** 128] = np.inf
    want[want <= -2.0 ** 128] = -np.inf
    assert np.array_equal(got, want, equal_nan=True)


def test_largest_scale_of_a_store():
    """The largest finite bf16 magnitude: scale byte 247."""
    b = np.full((1, 32), 0x7F7F, np.uint16)
    b[0, 1::2] = 0xFF7F
    q, s = Q.store(b)
    wq, ws = q8.store(b)
    assert ws.max() == 247
    assert np.array_equal(s.cpu().numpy(), ws.reshape(-1)) and np.array_equal(q.cpu().numpy(), wq.reshape(-1))
