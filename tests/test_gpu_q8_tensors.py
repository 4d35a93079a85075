"""Calls on tensors that lie next to each other, and those that may share memory."""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import test_gpu_q8 as Q
import workloads as W
from gpu_helpers import cfgs, free, gpu_plan

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
