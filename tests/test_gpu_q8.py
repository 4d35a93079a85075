"""8-bit activation checkpoints against the oracle.

Codes, scale bytes, restored rows, dispatched rows, dy and the projection's
kept h13 are exact.  Tolerances of the rest, with h = 2^-24:

* SwiGLU gradients: the sigmoid's exponential has a relative error of
  (2 |gate| + 2) h, the reciprocal and the sums around it 4 h more, the
  products after it 6 h; 1 + gate (1 - s) is a difference whose terms are 1 and
  |gate|, each off by those: (4 |gate| + 40) h |d act up s| (1 + |gate|) in all,
  and half a bf16 step, 2^-8 of the value.  Where e^-gate passes fp32's range s
  is 0 instead of at most 2^-127: 2^-126 |d act| (1 + |up|) (1 + |gate|) more.
* dgates: a lane adds 8 products per vector and CU <= 4 vectors a pass, 6
  additions join the lanes and one each pass: (H' / 64 + 16) h sum |dout y|.
* act of the projection: the bar of the bf16 projection, 2e-2 of the row.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import workloads as W
from gpu_helpers import announce, bits, cfgs, free, gpu_plan, rows_close
from oracle import bf16, dataflow, q8, swiglu
from oracle.plan import make_plan

pytestmark = pytest.mark.gpu

h = 2.0 ** -24
SENT = 0xA5


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


class Guarded:
    """uint8 or bf16 output of n elements with sentinel bytes around it."""

    def __init__(self, n, dtype):
        size = torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((128 + n * size,), SENT, dtype=torch.uint8, device="cuda")
        self.t = self.raw[64:64 + n * size].view(dtype)
        self.end = 64 + n * size

    def check(self):
        assert torch.all(self.raw[:64] == SENT) and torch.all(self.raw[self.end:] == SENT)


def blocks(width):
    return -(-width // 32)


def store(b):
    """GPU codes and scales of a bf16 bit array, checked for stray writes."""
    rows, width = b.shape
    q, s = Guarded(rows * width, torch.uint8), Guarded(rows * blocks(width), torch.uint8)
    mx.moe_q8_store(rows, width, W.from_bits(b, "cuda"), q.t, s.t)
    torch.cuda.synchronize()
    q.check()
    s.check()
    return q.t, s.t


def host(q, s, rows, width):
    return q.cpu().numpy().reshape(rows, width), s.cpu().numpy().reshape(rows, blocks(width))


def same_codes(q, want):
    nan = (want & 127) == 127
    assert np.array_equal((q & 127) == 127, nan)
    assert np.array_equal(q[~nan], want[~nan])


def activations(rows, width, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, width)) * np.exp(2 * g.standard_normal((rows, 1)))
    x[:, g.integers(0, width, 1 + width // 50)] *= 64
    return bf16.f64_to_bits(x)


SHAPES = [(1, 8), (3, 16), (5, 24), (7, 32), (2, 40), (33, 64), (257, 72), (64, 520), (130, 1000),
          (9, 2048), (41, 7168), (1, 40960), (1025, 8)]


@pytest.mark.parametrize("rows,width", SHAPES)
def test_store_and_load(rows, width):
    b = activations(rows, width, rows + width)
    q, s = store(b)
    wq, ws = q8.store(b)
    gq, gs = host(q, s, rows, width)
    assert np.array_equal(gs, ws)
    same_codes(gq, wq)
    out = Guarded(rows * width, torch.bfloat16)
    mx.moe_q8_load(rows, width, q, s, out.t)
    torch.cuda.synchronize()
    out.check()
    assert np.array_equal(bits(out.t).reshape(rows, width), q8.load_bits(wq, ws))


@pytest.mark.parametrize("width", [8, 32])
def test_every_bf16_value(width):
    """Each of the 65,536 bit patterns alone in a block, and among neighbours."""
    if width == 8:
        b = np.zeros((65536, 8), np.uint16)
        b[:, 3] = np.arange(65536)
    else:
        b = np.arange(65536, dtype=np.uint16).reshape(-1, 32)
    q, s = store(b)
    wq, ws = q8.store(b)
    gq, gs = host(q, s, *b.shape)
    assert np.array_equal(gs, ws)
    same_codes(gq, wq)


def test_every_code_under_every_scale():
    q = np.repeat(np.arange(256, dtype=np.uint8)[None], 248, axis=0)
    s = np.repeat(np.arange(248, dtype=np.uint8)[:, None], 8, axis=1)
    out = torch.empty((248, 256), dtype=torch.bfloat16, device="cuda")
    mx.moe_q8_load(248, 256, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), out)
    torch.cuda.synchronize()
    got, want = bf16.bits_to_f64(bits(out)), q8.load(q, s)
    small = np.ldexp(1.0, -133)                            # bf16's last place, of k near -127
    exact = np.isnan(want) | (np.round(want / small) * small == want)
    # bf16 has infinity where a code's value passes its largest number (k = 120, no store's)
    want[want >= 2.0 ** 128] = np.inf
    want[want <= -2.0 ** 128] = -np.inf
    assert np.array_equal(got[exact], want[exact], equal_nan=True)
    assert np.all(np.abs(got[~exact] - want[~exact]) < small)      # codes that no store makes


def test_rows_past_two_gib():
    """A flat offset of more than 2^31 values: the last rows, and those at the border."""
    rows, width = (1 << 31) // 8192 + 3, 8192
    src = torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
    src.fill_(0.75)
    pick = [0, rows - 4, rows - 3, rows - 1]
    b = activations(4, width, 3)
    for i, r in enumerate(pick):
        src[r] = W.from_bits(b[i], "cuda")
    q = torch.empty((rows, width), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, blocks(width)), dtype=torch.uint8, device="cuda")
    mx.moe_q8_store(rows, width, src, q, s)
    src.zero_()
    mx.moe_q8_load(rows, width, q, s, src)
    torch.cuda.synchronize()
    wq, ws = q8.store(b)
    for i, r in enumerate(pick):
        assert np.array_equal(q[r].cpu().numpy(), wq[i]) and np.array_equal(s[r].cpu().numpy(), ws[i])
        assert np.array_equal(bits(src[r]), q8.load_bits(wq, ws)[i])
    assert torch.all(src[1] == 0.75) and torch.all(src[rows - 2] == 0.75)


def test_no_rows():
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    mx.moe_q8_store(0, 8, torch.empty(0, dtype=torch.bfloat16, device="cuda"), e, e)
    mx.moe_q8_load(0, 8, e, e, torch.empty(0, dtype=torch.bfloat16, device="cuda"))


LAYERS = [W.TINY, W.TINY.with_(S=1), W.TINY.with_(H=72, Hp=40, S=37),
          W.TINY.with_(R=1, E=5, K=5, S=19, B=5, H=2056, Hp=1032),
          W.TINY.with_(R=2, E=16, K=12, S=24, B=8, H=264, Hp=2600),
          W.TINY.with_(S=20, H=9160, Hp=520), W.SKEWED.with_(S=128)]


def layer_id(s):
    return "%s-S%d-E%d-K%d-H%d-%d" % (s.name, s.S, s.E, s.K, s.H, s.Hp)


@pytest.mark.parametrize("shape", LAYERS, ids=layer_id)
def test_dispatch_from_codes(shape):
    c, oc = cfgs(shape)
    ids, _ = W.routing_uniform(shape, salt=2)
    plan, _ = gpu_plan(shape, ids)
    b = activations(shape.tokens, shape.H, 7)
    q, s = store(b)
    rows = shape.R * shape.SK
    out = Guarded(rows * shape.H, torch.bfloat16)
    mx.moe_dispatch_q8(c, plan, q, s, out.t)
    torch.cuda.synchronize()
    out.check()
    want = dataflow.dispatch(q8.load_bits(*q8.store(b)), make_plan(ids, oc), oc)
    assert np.array_equal(bits(out.t).reshape(rows, shape.H), want)


def test_after_a_failed_plan():
    """No route: xperm and dy keep what they held, dgates are zero."""
    shape = W.TINY
    c, _ = cfgs(shape)
    ids, _ = W.routing_uniform(shape)
    ids = ids.copy()
    ids[3, 1] = shape.E
    plan, g = gpu_plan(shape, ids)
    assert int(g["status"][2]) & mx.STATUS_BAD_ID
    rows = shape.R * shape.SK
    q, s = store(activations(shape.tokens, shape.H, 1))
    xp = torch.full((rows * shape.H * 2,), SENT, dtype=torch.uint8, device="cuda")
    mx.moe_dispatch_q8(c, plan, q, s, xp.view(torch.bfloat16))
    yq, ys = store(activations(rows, shape.Hp, 2))
    dy = torch.full((rows * shape.Hp * 2,), SENT, dtype=torch.uint8, device="cuda")
    dg = torch.full((shape.tokens, shape.K), 3.0, device="cuda")
    mx.moe_combine_backward_q8(c, plan, W.randn_bf16((shape.tokens, shape.Hp), 4, "cuda"), yq, ys,
                               torch.ones_like(dg), dy.view(torch.bfloat16), dg)
    torch.cuda.synchronize()
    assert torch.all(xp == SENT) and torch.all(dy == SENT) and torch.all(dg == 0)


@pytest.mark.parametrize("shape", LAYERS, ids=layer_id)
def test_combine_backward_from_codes(shape):
    c, oc = cfgs(shape)
    ids, gates = W.routing_uniform(shape, salt=5)
    plan, _ = gpu_plan(shape, ids)
    ref = make_plan(ids, oc)
    rows = shape.R * shape.SK
    yb = activations(rows, shape.Hp, 11)
    db = activations(shape.tokens, shape.Hp, 12)
    q, s = store(yb)
    dy, dg = Guarded(rows * shape.Hp, torch.bfloat16), Guarded(shape.tokens * shape.K, torch.float32)
    mx.moe_combine_backward_q8(c, plan, W.from_bits(db, "cuda"), q, s,
                               torch.from_numpy(gates).cuda(), dy.t, dg.t)
    torch.cuda.synchronize()
    dy.check()
    dg.check()
    kept = q8.load_bits(*q8.store(yb))
    wdy, wdg = dataflow.combine_backward(db, kept, gates, ref, oc)
    assert np.array_equal(bits(dy.t).reshape(rows, shape.Hp), wdy)
    d, y = bf16.bits_to_f64(db), bf16.bits_to_f64(kept)
    route = ref.route.reshape(-1, shape.K)
    got = dg.t.cpu().numpy().reshape(-1, shape.K)
    for k in range(shape.K):
        terms = np.abs(d * y[route[:, k]]).sum(1)
        assert np.all(np.abs(got[:, k] - wdg[:, k]) <= (shape.Hp / 64 + 16) * h * terms)


def swiglu_tolerance(g, u, d, want):
    s = swiglu.sigmoid(g)
    n = g.shape[1]
    lost = 2.0 ** -126 * np.abs(d) * (1 + np.abs(u)) * (1 + np.abs(g))
    rel = (4 * np.minimum(np.abs(g), 200) + 40) * h
    t = np.empty_like(want)
    t[:, :n] = rel * np.abs(d * u) * s * (1 + np.abs(g)) + lost
    t[:, n:] = rel * np.abs(d * g) * s + lost
    return t + 2.0 ** -8 * np.abs(want) + 2.0 ** -133


def check_swiglu_backward(c, shape, q, s, h13_bits, dact_bits, in_place):
    rows, Hp = shape.R * shape.SK, shape.Hp
    dact = W.from_bits(dact_bits, "cuda")
    dh, act = Guarded(rows * 2 * Hp, torch.bfloat16), Guarded(rows * Hp, torch.bfloat16)
    if in_place:
        act.t.copy_(dact.reshape(-1))
        mx.moe_swiglu_backward_q8(c, q, s, act.t, dh.t, act.t)
    else:
        mx.moe_swiglu_backward_q8(c, q, s, dact, dh.t, act.t)
    torch.cuda.synchronize()
    dh.check()
    act.check()
    kept = q8.load(*q8.store(h13_bits.reshape(2 * rows, Hp))).reshape(rows, 2 * Hp)
    g, u, d = kept[:, :Hp], kept[:, Hp:], bf16.bits_to_f64(dact_bits)
    dg, du = swiglu.swiglu_backward_f64(g, u, d)
    want = np.concatenate([dg, du], 1)
    got = bf16.bits_to_f64(bits(dh.t)).reshape(rows, 2 * Hp)
    assert np.all(np.abs(got - want) <= swiglu_tolerance(g, u, d, want))
    a = swiglu.silu(g) * u
    tol = (4 * np.minimum(np.abs(g), 200) + 40) * h * np.abs(a) + 2.0 ** -8 * np.abs(a) + \
        2.0 ** -126 * (1 + np.abs(g)) * (1 + np.abs(u))
    assert np.all(np.abs(bf16.bits_to_f64(bits(act.t)).reshape(rows, Hp) - a) <= tol)
    # without act the gradients are the same bits
    dh2 = Guarded(rows * 2 * Hp, torch.bfloat16)
    mx.moe_swiglu_backward_q8(c, q, s, dact, dh2.t)
    torch.cuda.synchronize()
    assert torch.equal(dh.t.view(torch.int16), dh2.t.view(torch.int16))


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "act-over-dact"])
@pytest.mark.parametrize("shape", LAYERS, ids=layer_id)
def test_swiglu_backward_from_codes(shape, in_place):
    c, _ = cfgs(shape)
    rows, Hp = shape.R * shape.SK, shape.Hp
    h13 = activations(rows, 2 * Hp, 21)
    h13[0, :8] = bf16.f64_to_bits(np.array([-200.0, 200, -88, 88, -1.2784645, 0, -0.0, 1e4]))
    q, s = store(h13.reshape(2 * rows, Hp))
    check_swiglu_backward(c, shape, q, s, h13, activations(rows, Hp, 22), in_place)


PROJECTIONS = [W.TINY, W.TINY.with_(H=72, Hp=40, S=37), W.TINY.with_(B=1, mode=1, Hp=136),
               W.TINY.with_(R=2, E=4, S=300, K=2, B=2, H=264, Hp=200),
               W.TINY.with_(S=1, H=8, Hp=8), W.SKEWED.with_(S=256, Hp=520)]


@pytest.mark.parametrize("shape", PROJECTIONS, ids=layer_id)
def test_projection_that_keeps_codes(shape):
    """act and codes bit for bit those of the bf16 projection and a store of its h13; the
    codes' values near the float64 product; rows of other ranks untouched."""
    c, oc = cfgs(shape)
    ids, _ = W.routing_uniform(shape, salt=8)
    plan, _ = gpu_plan(shape, ids)
    ref = make_plan(ids, oc)
    rows, H, Hp = shape.R * shape.SK, shape.H, shape.Hp
    c13 = mx.make_cfg(shape.R, shape.S, shape.E, shape.K, H, 2 * Hp, shape.B, shape.mode)
    x = W.randn_bf16((shape.tokens, H), 1, "cuda")
    w = W.randn_bf16((shape.E, H, 2 * Hp), 2, "cuda")
    wp = torch.zeros((max(1, shape.R * shape.B), H, 2 * Hp), dtype=torch.bfloat16, device="cuda")
    xp = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mx.moe_gemm_workspace_size(c), dtype=torch.uint8, device="cuda")
    mx.moe_prefetch_weight(c13, plan, w, wp)
    mx.moe_dispatch(c, plan, x, xp)
    act0 = torch.zeros((rows, Hp), dtype=torch.bfloat16, device="cuda")
    h13 = torch.zeros((rows, 2 * Hp), dtype=torch.bfloat16, device="cuda")
    mx.moe_grouped_gemm_swiglu(c, xp, w, wp, plan.cu_seqlens, act0, h13, 0, shape.R, ws)
    act, q, s = (Guarded(rows * Hp, torch.bfloat16), Guarded(rows * 2 * Hp, torch.uint8),
                 Guarded(rows * 2 * blocks(Hp), torch.uint8))
    mx.moe_grouped_gemm_swiglu_q8(c, xp, w, wp, plan.cu_seqlens, act.t, q.t, s.t, 0, shape.R, ws)
    torch.cuda.synchronize()
    for o in (act, q, s):
        o.check()
    assert torch.equal(act.t.view(torch.int16), act0.view(torch.int16).reshape(-1))
    wq, wsc = store(bits(h13).reshape(2 * rows, Hp))
    assert torch.equal(q.t, wq) and torch.equal(s.t, wsc)
    ract, rh = swiglu.swiglu_gemm(bits(xp), bits(w), bits(wp).reshape(shape.R, -1, H, 2 * Hp)
                                  if shape.B else None, ref, oc)
    rows_close(bits(act.t).reshape(rows, Hp), ract)
    kept = q8.load(*host(q.t, s.t, 2 * rows, Hp)).reshape(rows, 2 * Hp)
    v = bf16.bits_to_f64(rh)
    k = np.repeat(host(q.t, s.t, 2 * rows, Hp)[1].astype(int) - 127, 32, axis=1)[:, :Hp]
    step = np.ldexp(1.0, k - 10).reshape(rows, 2 * Hp)
    # 2^-4 of the value for the code, and the projection's own bar
    bar = 2e-2 * np.abs(v).max(axis=1, keepdims=True)
    assert np.all(np.abs(kept - v) <= 2.0 ** -4 * np.abs(v) + step + 1.1 * bar)
    if shape.R > 1:
        act, q, s = (torch.full((n,), SENT, dtype=torch.uint8, device="cuda") for n in
                     (rows * Hp * 2, rows * 2 * Hp, rows * 2 * blocks(Hp)))
        mx.moe_grouped_gemm_swiglu_q8(c, xp, w, wp, plan.cu_seqlens, act.view(torch.bfloat16), q, s,
                                      1, 2, ws)
        torch.cuda.synchronize()
        SK = shape.SK
        assert torch.equal(q[SK * 2 * Hp:2 * SK * 2 * Hp], wq[SK * 2 * Hp:2 * SK * 2 * Hp])
        n = 2 * blocks(Hp) * SK
        assert torch.equal(s[n:2 * n], wsc[n:2 * n])
        assert torch.all(s[:n] == SENT) and torch.all(s[2 * n:] == SENT)
        assert torch.all(q[:SK * 2 * Hp] == SENT) and torch.all(q[2 * SK * 2 * Hp:] == SENT)
        assert torch.all(act[:SK * Hp * 2] == SENT) and torch.all(act[2 * SK * Hp * 2:] == SENT)


def test_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((4, 64), dtype=torch.uint8, device="cuda")
    s = torch.zeros((4, 2), dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError):
        mx.moe_q8_store(4, 64, x.float(), q, s)
    with pytest.raises(TypeError):
        mx.moe_q8_store(4, 64, x, q.to(torch.int8), s)
    with pytest.raises(ValueError):
        mx.moe_q8_store(5, 64, x, q, s)
    with pytest.raises(ValueError):
        mx.moe_q8_store(4, 64, x, q, s[:, :1].contiguous())
    with pytest.raises(ValueError):
        mx.moe_q8_store(4, 64, x.t(), q, s)
    with pytest.raises(ValueError):
        mx.moe_q8_load(4, 64, q.cpu(), s, x)
