"""One MoE layer with biased experts, a shared expert and dropout, forward and backward.

logits = x Wr + br (fp32) -> router -> plan -> prefetch -> dispatch -> gelu(x W1 + b1) ->
h W2 + b2 -> out = s + dropout(sum gates y), s = x + (silu(x S1 + c1) S2 + c2), and back to
every weight, bias and x, through the product's epilogue, its backward, and combine with dropout
and the entry points around them.

Against the oracle's chain in float64 arithmetic with the same roundings.  Between the two,
values differ where an fp32 sum lands on the other side of a bf16 rounding (relative 2^-8, about
one in a hundred): 4e-4 per step in the 2-norm of a tensor, so ten chained steps stay below
2e-2, the projections' own bar.  A wrong row, bias, mask or sign is of order 1.

The same step is captured once and replayed with new inputs and new random numbers: bit for bit
the eager run.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import workloads as W
from gpu_helpers import announce, bits, cfgs, free
from oracle import bf16, dataflow, router
from oracle import epilogue as O
from oracle.plan import Cfg, make_plan

pytestmark = pytest.mark.gpu

P = 0.2


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


class Layer:
    """Buffers and calls; widths H -> H' -> H in the experts, H -> H' -> H in the shared one."""

    def __init__(self, s, seed=0):
        self.s = s
        T, rows, H, Hp, E = s.tokens, s.R * s.SK, s.H, s.Hp, s.E
        args = (s.R, s.S, E, s.K)
        self.c1 = mx.make_cfg(*args, H, Hp, s.B, s.mode)
        self.c2 = mx.make_cfg(*args, Hp, H, s.B, s.mode)
        one = lambda a, b, B=0, mode=mx.MODE_INFER: mx.make_cfg(1, T, 1, 1, a, b, B, mode)
        self.cr, self.cs1, self.cs2 = one(H, E), one(H, Hp), one(Hp, H)
        # weight gradients are of training configurations, with a slot that nothing uses
        self.tr, self.ts1, self.ts2 = (one(a, b, 1, mx.MODE_TRAIN) for a, b in ((H, E), (H, Hp), (Hp, H)))
        self.rc = mx.make_router_cfg(mx.SCORE_SOFTMAX, 1, 1.5)
        self.er = mx.make_epilogue_cfg(mx.ACT_NONE, 0.0, True)
        self.e0, self.eg = mx.make_epilogue_cfg(), mx.make_epilogue_cfg(mx.ACT_GELU)
        self.es = mx.make_epilogue_cfg(mx.ACT_SILU)
        self.dc = mx.make_dropout_cfg(P)
        f = lambda *d: torch.zeros(d, device="cuda")
        b = lambda *d: torch.zeros(d, dtype=torch.bfloat16, device="cuda")
        w = lambda n, *d: (W.randn_bf16(d, seed + n, "cuda").float() / d[-2] ** 0.5).bfloat16()
        self.x, self.dout, self.rng = b(T, H), b(T, H), torch.zeros(2, dtype=torch.int64, device="cuda")
        self.wr, self.w1, self.w2 = w(1, 1, H, E), w(2, E, H, Hp), w(3, E, Hp, H)
        self.s1, self.s2 = w(4, 1, H, Hp), w(5, 1, Hp, H)
        self.br, self.b1, self.b2, self.k1, self.k2 = f(1, E), f(E, Hp), f(E, H), f(1, Hp), f(1, H)
        self.ids, self.gates = torch.zeros((T, s.K), dtype=torch.int32, device="cuda"), f(T, s.K)
        self.plan, self.solo = mx.Plan(self.c1), mx.Plan(self.tr)
        self.cu1 = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        slots = max(1, s.R * s.B)
        self.p1, self.p2 = b(slots, H, Hp), b(slots, Hp, H)
        pairs = ((self.c1, self.eg), (self.c2, self.e0), (self.cr, self.er), (self.cs1, self.es), (self.cs2, self.e0))
        self.ws = torch.empty(max(mx.moe_epilogue_workspace_size(*p) for p in pairs), dtype=torch.uint8, device="cuda")
        self.gws = torch.empty(max(mx.moe_gemm_workspace_size(c) for c in (self.c1, self.tr)), dtype=torch.uint8,
                               device="cuda")
        self.logits, self.xp, self.pre1, self.h1, self.y = f(T, E), b(rows, H), b(rows, Hp), b(rows, Hp), b(rows, H)
        self.spre, self.sh, self.sout, self.out = b(T, Hp), b(T, Hp), b(T, H), b(T, H)
        self.dy, self.dgates, self.dh1, self.dxp, self.dx = b(rows, H), f(T, s.K), b(rows, Hp), b(rows, H), b(T, H)
        self.dlogits, self.dl16, self.dxr = f(T, E), b(T, E), b(T, H)
        self.dsh, self.dxs = b(T, Hp), b(T, H)
        self.db1, self.db2, self.dbr, self.dk1, self.dk2 = f(E, Hp), f(E, H), f(1, E), f(1, Hp), f(1, H)
        self.g1, self.gp1, self.g2, self.gp2 = f(E, H, Hp), f(slots, H, Hp), f(E, Hp, H), f(slots, Hp, H)
        self.gr, self.gs1, self.gs2 = f(1, H, E), f(1, H, Hp), f(1, Hp, H)
        self.spare = f(1, H, max(E, Hp, H))
        mx.moe_plan_run(self.tr, torch.zeros(T, dtype=torch.int32, device="cuda"), self.solo)

    def fill(self, seed):
        g = np.random.default_rng(seed)
        self.x.copy_(W.randn_bf16(tuple(self.x.shape), 100 + seed, "cuda"))
        self.dout.copy_(W.randn_bf16(tuple(self.dout.shape), 200 + seed, "cuda"))
        self.rng.copy_(torch.tensor([123 + seed, seed]))
        for n in ("br", "b1", "b2", "k1", "k2"):
            t = getattr(self, n)
            t.copy_(torch.from_numpy(0.5 * g.standard_normal(tuple(t.shape))))

    def one(self, cfg, ec, x, w, bias, residual, y, pre=None):
        mx.moe_grouped_gemm_epilogue(cfg, ec, None, x, w, None, bias, residual, None, y, pre, 0, 1, self.ws)

    def __call__(self):
        p, R = self.plan, self.s.R
        self.one(self.cr, self.er, self.x, self.wr, self.br, None, self.logits)
        mx.moe_router(self.c1, self.rc, self.logits, None, self.ids, self.gates)
        mx.moe_plan_run(self.c1, self.ids, p)
        mx.moe_prefetch_weight(self.c1, p, self.w1, self.p1)
        mx.moe_prefetch_weight(self.c2, p, self.w2, self.p2)
        mx.moe_dispatch(self.c1, p, self.x, self.xp)
        mx.moe_grouped_gemm_epilogue(self.c1, self.eg, p, self.xp, self.w1, self.p1, self.b1, None, None, self.h1,
                                     self.pre1, 0, R, self.ws)
        mx.moe_grouped_gemm_epilogue(self.c2, self.e0, p, self.h1, self.w2, self.p2, self.b2, None, None, self.y, None,
                                     0, R, self.ws)
        self.one(self.cs1, self.es, self.x, self.s1, self.k1, None, self.sh, self.spre)
        self.one(self.cs2, self.e0, self.sh, self.s2, self.k2, self.x, self.sout)
        mx.moe_combine_dropout(self.c2, self.dc, p, self.y, self.gates, self.sout, self.rng, self.out)
        # backward of the experts
        mx.moe_combine_dropout_backward(self.c2, self.dc, p, self.dout, self.y, self.gates, self.rng, self.dy,
                                        self.dgates)
        mx.moe_epilogue_backward(self.c2, self.e0, p, self.dy, None, None, None, self.db2, self.ws)
        mx.moe_grouped_gemm_wgrad(self.c2, p, self.h1, self.dy, self.g2, self.gp2, self.gws)
        mx.moe_reduce_grad(self.c2, p, self.g2, self.gp2)
        mx.moe_grouped_gemm_dgrad(self.c2, self.dy, self.w2, self.p2, p.cu_seqlens, self.dh1, 0, R, self.gws)
        mx.moe_epilogue_backward(self.c1, self.eg, p, self.dh1, self.pre1, None, self.dh1, self.db1, self.ws)
        mx.moe_grouped_gemm_wgrad(self.c1, p, self.xp, self.dh1, self.g1, self.gp1, self.gws)
        mx.moe_reduce_grad(self.c1, p, self.g1, self.gp1)
        mx.moe_grouped_gemm_dgrad(self.c1, self.dh1, self.w1, self.p1, p.cu_seqlens, self.dxp, 0, R, self.gws)
        mx.moe_dispatch_backward(self.c1, p, self.dxp, self.dx)
        # of the router's projection
        mx.moe_router_backward(self.c1, self.rc, self.logits, self.ids, self.dgates, None, None, None, self.dlogits)
        mx.moe_epilogue_backward(self.cr, self.er, None, self.dlogits, None, None, self.dl16, self.dbr, self.ws)
        mx.moe_grouped_gemm_wgrad(self.tr, self.solo, self.x, self.dl16, self.gr, self.spare, self.gws)
        mx.moe_grouped_gemm_dgrad(self.cr, self.dl16, self.wr, None, self.cu1, self.dxr, 0, 1, self.gws)
        # of the shared expert
        mx.moe_epilogue_backward(self.cs2, self.e0, None, self.dout, None, None, None, self.dk2, self.ws)
        mx.moe_grouped_gemm_wgrad(self.ts2, self.solo, self.sh, self.dout, self.gs2, self.spare, self.gws)
        mx.moe_grouped_gemm_dgrad(self.cs2, self.dout, self.s2, None, self.cu1, self.dsh, 0, 1, self.gws)
        mx.moe_epilogue_backward(self.cs1, self.es, None, self.dsh, self.spre, None, self.dsh, self.dk1, self.ws)
        mx.moe_grouped_gemm_wgrad(self.ts1, self.solo, self.x, self.dsh, self.gs1, self.spare, self.gws)
        mx.moe_grouped_gemm_dgrad(self.cs1, self.dsh, self.s1, None, self.cu1, self.dxs, 0, 1, self.gws)

    OUT = ("logits", "ids", "gates", "out", "sout", "dgates", "db1", "db2", "dbr", "dk1", "dk2", "g1", "g2", "gr", "gs1",
           "gs2", "dx", "dxr", "dxs")

    def outputs(self):
        torch.cuda.synchronize()
        return {k: getattr(self, k).clone() for k in self.OUT}


def rounded(v):
    return bf16.bits_to_f64(bf16.f64_to_bits(v))


def near(got, want, what, tol=2e-2):
    got = got.double().cpu().numpy().reshape(-1)
    want = np.asarray(want, np.float64).reshape(-1)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= tol, (what, rel)


@pytest.mark.parametrize("shape", [W.TINY.with_(H=72, Hp=40, S=37), W.TINY.with_(S=1),
                                   W.SKEWED.with_(S=64, H=128, Hp=64)], ids=["tiny-odd", "one-token", "skewed"])
def test_step_against_the_oracle(shape):
    s = shape
    announce("biased layer", s)
    L = Layer(s)
    L.fill(1)
    L()
    got = L.outputs()
    v = lambda t: bf16.bits_to_f64(bits(t)) if t.dtype == torch.bfloat16 else t.double().cpu().numpy()
    oc1 = Cfg(s.R, s.S, s.E, s.K, s.H, s.Hp, s.B, s.mode)
    oc2 = Cfg(s.R, s.S, s.E, s.K, s.Hp, s.H, s.B, s.mode)
    x, dout, rng = v(L.x), v(L.dout), L.rng.tolist()
    near(got["logits"], x @ v(L.wr)[0] + v(L.br), "logits", 1e-4)
    z = v(got["logits"])
    ids = router.choose(z, None, s.K, router.SOFTMAX)
    assert np.array_equal(got["ids"].cpu().numpy(), ids)
    gates = (1.5 * router.gate_shares(z, ids, router.SOFTMAX, True)).astype(np.float32)
    plan = make_plan(ids, oc1)
    expert = O.segment_experts(plan.cu_seqlens, plan.slot_expert, s.E, s.SK)
    route = plan.route.astype(np.int64)
    xp = np.zeros((s.R * s.SK, s.H))
    xp[route] = np.repeat(x, s.K, 0)
    per_row = lambda a, w: np.stack([a[i] @ w[e] for i, e in enumerate(expert)])
    w1, w2 = v(L.w1), v(L.w2)
    z1 = per_row(xp, w1) + v(L.b1)[expert]
    h1 = rounded(O.act(z1, O.GELU))
    pre1 = rounded(z1)
    y = rounded(per_row(h1, w2) + v(L.b2)[expert])
    zs = x @ v(L.s1)[0] + v(L.k1)
    sh, spre = rounded(O.act(zs, O.SILU)), rounded(zs)
    sout = rounded(sh @ v(L.s2)[0] + v(L.k2) + x)
    near(got["sout"], sout, "sout")
    near(got["out"], O.combine(y, gates.astype(np.float64), route, P, rng, sout), "out")
    dyr, dgates = O.combine_backward(dout, y, gates.astype(np.float64), route, P, rng)
    near(got["dgates"], dgates, "dgates")
    dy = np.zeros_like(y)
    dy[route] = rounded(dyr.reshape(-1, s.H))
    rows_of = lambda a, b, E: np.stack([a[expert == e].T @ b[expert == e] for e in range(E)])
    near(got["db2"], np.stack([dy[expert == e].sum(0) for e in range(s.E)]), "db2")
    near(got["g2"], rows_of(h1, dy, s.E), "g2")
    dh = rounded(per_row(dy, np.swapaxes(w2, 1, 2)))
    dz1, db1 = O.backward(dh, pre1, O.GELU, 0.0, [0, 0], expert, s.E)
    near(got["db1"], db1, "db1")
    dz1 = rounded(dz1)
    near(got["g1"], rows_of(xp, dz1, s.E), "g1")
    dxp = rounded(per_row(dz1, np.swapaxes(w1, 1, 2)))
    near(got["dx"], dxp[route].reshape(s.tokens, s.K, s.H).sum(1), "dx")
    dl, _ = router.backward(z, ids, router.SOFTMAX, True, 1.5, dgates, None, None, None)
    near(got["dbr"], dl.sum(0, keepdims=True), "dbr")
    near(got["gr"], x.T @ rounded(dl), "gr")
    near(got["dxr"], rounded(dl) @ v(L.wr)[0].T, "dxr")
    near(got["dk2"], dout.sum(0), "dk2")
    near(got["gs2"], sh.T @ dout, "gs2")
    ds = rounded(dout @ v(L.s2)[0].T) * O.slope(spre, O.SILU)
    near(got["dk1"], ds.sum(0), "dk1")
    near(got["gs1"], x.T @ rounded(ds), "gs1")
    near(got["dxs"], rounded(ds) @ v(L.s1)[0].T, "dxs")


@pytest.mark.parametrize("shape", [W.TINY.with_(H=72, Hp=40, S=37), W.SKEWED.with_(S=128)], ids=["tiny", "skewed"])
def test_captured_step_equals_eager(shape):
    L = Layer(shape)
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
