"""One MoE layer's training step through the new entry points and the old ones together.

Router (with the balance loss) -> plan -> prefetch -> dispatch -> SwiGLU projection that
keeps codes -> second projection -> combine, and back: combine from y's codes, data and
weight gradients, the activation's backward from h13's codes, the dispatch redone from x's
codes, and the router's gradient of gates and loss.

Against the oracle's chain in float64 arithmetic with the same roundings.  Between the two,
values differ where an fp32 sum lands on the other side of a bf16 rounding (relative 2^-8,
about one in a hundred), and one in sixteen of those lands on the other side of a code's
(2^-3 of the value at most): in the 2-norm of a tensor that is 2^-8 per step and
2^-3 * sqrt(1/1600) = 3e-3, so five chained steps stay below 2e-2, the projections' own bar.
A wrong row, block, scale or sign is of order 1.

The same step is captured once and replayed with new inputs: bit for bit the eager run.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import workloads as W
from gpu_helpers import announce, bits, cfgs, free
from oracle import bf16, dataflow, q8, router, swiglu
from oracle.plan import Cfg, make_plan

pytestmark = pytest.mark.gpu

SCALE = 1.5


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


class Layer:
    """Buffers and calls of one layer; widths H -> 2 H' -> H' -> H."""

    def __init__(self, s, score, seed=0, nseq=3):
        self.s, self.score, self.nseq = s, score, nseq
        args = (s.R, s.S, s.E, s.K)
        self.c = mx.make_cfg(*args, s.H, s.Hp, s.B, s.mode)                # H, H'
        self.c13 = mx.make_cfg(*args, s.H, 2 * s.Hp, s.B, s.mode)
        self.c2 = mx.make_cfg(*args, s.Hp, s.H, s.B, s.mode)
        self.rc = mx.make_router_cfg(score, 1, SCALE, False, nseq)
        T, rows, H, Hp, E = s.tokens, s.R * s.SK, s.H, s.Hp, s.E
        f = lambda *d: torch.zeros(d, device="cuda")
        b = lambda *d: torch.zeros(d, dtype=torch.bfloat16, device="cuda")
        u = lambda *d: torch.zeros(d, dtype=torch.uint8, device="cuda")
        i = lambda *d: torch.zeros(d, dtype=torch.int32, device="cuda")
        blk = lambda n: -(-n // 32)
        self.x, self.logits, self.bias, self.dout = b(T, H), f(T, E), f(E), b(T, H)
        self.cu, self.dloss = i(nseq + 1), f(nseq)
        self.w13 = (W.randn_bf16((E, H, 2 * Hp), seed + 1, "cuda").float() / H ** 0.5).bfloat16()
        self.w2 = (W.randn_bf16((E, Hp, H), seed + 2, "cuda").float() / Hp ** 0.5).bfloat16()
        self.ids, self.gates = i(T, s.K), f(T, s.K)
        self.counts, self.prob, self.loss = i(nseq, E), f(nseq, E), f(nseq)
        self.rws = u(mx.moe_router_workspace_size(self.c, self.rc))
        self.plan = mx.Plan(self.c)
        self.p13, self.p2 = b(max(1, s.R * s.B), H, 2 * Hp), b(max(1, s.R * s.B), Hp, H)
        self.ws = u(mx.moe_gemm_workspace_size(self.c))
        self.xq, self.xs, self.xp = u(T, H), u(T, blk(H)), b(rows, H)
        self.act, self.hq, self.hs = b(rows, Hp), u(rows, 2 * Hp), u(rows, 2 * blk(Hp))
        self.y, self.yq, self.ys, self.out = b(rows, H), u(rows, H), u(rows, blk(H)), b(T, H)
        self.dy, self.dgates, self.dact, self.dh13 = b(rows, H), f(T, s.K), b(rows, Hp), b(rows, 2 * Hp)
        self.g13, self.gp13 = f(E, H, 2 * Hp), f(max(1, s.R * s.B), H, 2 * Hp)
        self.g2, self.gp2 = f(E, Hp, H), f(max(1, s.R * s.B), Hp, H)
        self.dxp, self.dx, self.dlogits = b(rows, H), b(T, H), f(T, E)

    def fill(self, seed):
        """New inputs in the same buffers."""
        s, g = self.s, np.random.default_rng(seed)
        T = s.tokens
        self.x.copy_(W.randn_bf16((T, s.H), 100 + seed, "cuda"))
        self.dout.copy_(W.randn_bf16((T, s.H), 200 + seed, "cuda"))
        self.logits.copy_(torch.from_numpy(1.5 * g.standard_normal((T, s.E))))
        self.bias.copy_(torch.from_numpy(0.1 * g.standard_normal(s.E)))
        self.dloss.copy_(torch.from_numpy(g.random(self.nseq) + 0.5))
        cu = np.sort(g.integers(0, T + 1, self.nseq + 1))
        cu[0] = 0
        self.cu.copy_(torch.from_numpy(cu))

    def __call__(self):
        s, p, R, T, rows = self.s, self.plan, self.s.R, self.s.tokens, self.s.R * self.s.SK
        mx.moe_router(self.c, self.rc, self.logits, self.bias, self.ids, self.gates, self.cu,
                      self.counts, self.prob, self.loss, self.rws)
        mx.moe_plan_run(self.c, self.ids, p)
        mx.moe_prefetch_weight(self.c13, p, self.w13, self.p13)
        mx.moe_prefetch_weight(self.c2, p, self.w2, self.p2)
        mx.moe_q8_store(T, s.H, self.x, self.xq, self.xs)
        mx.moe_dispatch(self.c, p, self.x, self.xp)
        mx.moe_grouped_gemm_swiglu_q8(self.c, self.xp, self.w13, self.p13, p.cu_seqlens, self.act,
                                      self.hq, self.hs, 0, R, self.ws)
        mx.moe_grouped_gemm(self.c2, self.act, self.w2, self.p2, p.cu_seqlens, self.y, 0, R, self.ws)
        mx.moe_combine(self.c2, p, self.y, self.gates, self.out)
        mx.moe_q8_store(rows, s.H, self.y, self.yq, self.ys)
        # backward: xp, act and y of the forward are not read any more
        mx.moe_combine_backward_q8(self.c2, p, self.dout, self.yq, self.ys, self.gates, self.dy,
                                   self.dgates)
        mx.moe_grouped_gemm_dgrad(self.c2, self.dy, self.w2, self.p2, p.cu_seqlens, self.dact, 0, R,
                                  self.ws)
        mx.moe_swiglu_backward_q8(self.c, self.hq, self.hs, self.dact, self.dh13, self.act)
        mx.moe_grouped_gemm_wgrad(self.c2, p, self.act, self.dy, self.g2, self.gp2, self.ws)
        mx.moe_reduce_grad(self.c2, p, self.g2, self.gp2)
        mx.moe_dispatch_q8(self.c, p, self.xq, self.xs, self.xp)
        mx.moe_grouped_gemm_wgrad(self.c13, p, self.xp, self.dh13, self.g13, self.gp13, self.ws)
        mx.moe_reduce_grad(self.c13, p, self.g13, self.gp13)
        mx.moe_grouped_gemm_dgrad(self.c13, self.dh13, self.w13, self.p13, p.cu_seqlens, self.dxp, 0,
                                  R, self.ws)
        mx.moe_dispatch_backward(self.c13, p, self.dxp, self.dx)
        mx.moe_router_backward(self.c, self.rc, self.logits, self.ids, self.dgates, self.cu,
                               self.counts, self.dloss, self.dlogits)

    OUT = ("ids", "gates", "counts", "prob", "loss", "out", "dgates", "g2", "g13", "dx", "dlogits",
           "hq", "hs", "yq", "ys", "xq", "xs")

    def outputs(self):
        torch.cuda.synchronize()
        return {k: getattr(self, k).clone() for k in self.OUT}


def near(got, want, what, tol=2e-2):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= tol, (what, rel)


@pytest.mark.parametrize("score", [router.SOFTMAX, router.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", [W.TINY.with_(H=72, Hp=40, S=37), W.TINY.with_(S=64, H=264, Hp=136),
                                   W.SKEWED.with_(S=64, H=128, Hp=64)],
                         ids=["tiny-odd", "tiny", "skewed"])
def test_step_against_the_oracle(shape, score):
    announce("training layer", shape.name, shape.H, shape.Hp, score)
    s = shape
    L = Layer(s, score)
    L.fill(1)
    L()
    got = {k: v.cpu() for k, v in L.outputs().items()}
    oc = Cfg(s.R, s.S, s.E, s.K, s.H, s.Hp, s.B, s.mode)
    oc13 = Cfg(s.R, s.S, s.E, s.K, s.H, 2 * s.Hp, s.B, s.mode)
    oc2 = Cfg(s.R, s.S, s.E, s.K, s.Hp, s.H, s.B, s.mode)
    z, bias = L.logits.double().cpu().numpy(), L.bias.cpu().numpy()
    cu = L.cu.cpu().numpy()
    ids = router.choose(z, bias, s.K, score)
    gates = (SCALE * router.gate_shares(z, ids, score, True)).astype(np.float32)
    counts, prob, loss = router.balance(z, ids, cu, score)
    assert np.array_equal(got["ids"].numpy(), ids) and np.array_equal(got["counts"].numpy(), counts)
    plan = make_plan(ids, oc)
    x, w13, w2, dout = bits(L.x), bits(L.w13), bits(L.w2), bits(L.dout)
    p13, p2 = dataflow.prefetch(w13, plan, oc13), dataflow.prefetch(w2, plan, oc2)
    xp = dataflow.dispatch(x, plan, oc)
    act, h13 = swiglu.swiglu_gemm(xp, w13, p13, plan, oc)
    y = dataflow.grouped_gemm(act, w2, p2, plan, oc2)
    out = dataflow.combine(y, gates, plan, oc2)
    rows, Hp = s.R * s.SK, s.Hp
    h13k = q8.load_bits(*q8.store(h13.reshape(2 * rows, Hp))).reshape(rows, 2 * Hp)
    yk, xk = q8.load_bits(*q8.store(y)), q8.load_bits(*q8.store(x))
    dy, dgates = dataflow.combine_backward(dout, yk, gates, plan, oc2)
    dact = dataflow.dgrad(dy, w2, p2, plan, oc2)
    dh13 = swiglu.swiglu_backward(h13k, dact)
    hk = bf16.bits_to_f64(h13k)
    act2 = bf16.f64_to_bits(swiglu.silu(hk[:, :Hp]) * hk[:, Hp:])
    g2, _ = dataflow.reduce_grad(*dataflow.wgrad(act2, dy, plan, oc2), plan, oc2)
    xpk = dataflow.dispatch(xk, plan, oc)
    g13, _ = dataflow.reduce_grad(*dataflow.wgrad(xpk, dh13, plan, oc13), plan, oc13)
    dx = dataflow.dispatch_backward(dataflow.dgrad(dh13, w13, p13, plan, oc13), plan, oc13)
    dz, _ = router.backward(z, ids, score, True, SCALE, dgates, cu, counts,
                            L.dloss.double().cpu().numpy())
    near(got["gates"], gates, "gates", 1e-5)
    near(got["prob"], prob, "prob", 1e-5)
    near(got["loss"], loss, "loss", 1e-5)
    near(bf16.bits_to_f64(bits(got["out"])), bf16.bits_to_f64(out), "out")
    near(got["dgates"], dgates, "dgates")
    near(got["g2"], g2, "g2")
    near(got["g13"], g13, "g13")
    near(bf16.bits_to_f64(bits(got["dx"])), bf16.bits_to_f64(dx), "dx")
    near(got["dlogits"], dz, "dlogits")


@pytest.mark.parametrize("shape", [W.TINY.with_(H=72, Hp=40, S=37), W.SKEWED], ids=["tiny", "skewed"])
def test_captured_step_equals_eager(shape):
    L = Layer(shape, router.SIGMOID)
    L.fill(1)
    L()                                        # eager warm-up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L()
    torch.cuda.synchronize()
    for seed in (2, 3, 4):
        L.fill(seed)
        torch.cuda.synchronize()
        g.replay()
        first = L.outputs()
        L()                                    # eager, same buffers and inputs
        eager = L.outputs()
        g.replay()
        again = L.outputs()
        for k in L.OUT:
            a, b, c = (d[k].view(torch.int16) if d[k].dtype == torch.bfloat16 else d[k]
                       for d in (first, eager, again))
            assert torch.equal(a, b) and torch.equal(b, c), (seed, k)


def test_two_streams_at_once():
    """Two layers, each on a stream of its own with buffers of its own, equal each alone."""
    a, b = Layer(W.SKEWED.with_(S=256), router.SOFTMAX, 0), Layer(W.SKEWED.with_(S=256), router.SIGMOID, 9)
    a.fill(5)
    b.fill(6)
    want = []
    for L in (a, b):
        L()
        want.append(L.outputs())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a()
        with torch.cuda.stream(s2):
            b()
    torch.cuda.synchronize()
    for L, w in ((a, want[0]), (b, want[1])):
        got = L.outputs()
        for k in L.OUT:
            x, y = (t.view(torch.int16) if t.dtype == torch.bfloat16 else t for t in (got[k], w[k]))
            assert torch.equal(x, y), k
