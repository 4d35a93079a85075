"""Product with bias, activation, dropout and residual, and its backward, against the oracle.

Tolerances: epilogue_checks.  dbias adds at most `rows` values in fp32, one step each, on top
of the errors of its terms.
"""
import numpy as np
import pytest
import torch

import moe_expert_load_amd as mx
import workloads as W
from epilogue_checks import close, dz_tol, h, product_tol, round_tol, z_tol
from gpu_helpers import announce, bits, cfgs, free, gpu_plan
from oracle import bf16
from oracle import epilogue as O

pytestmark = pytest.mark.gpu

SENT = 0x7E57


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    free()
    yield
    free()


def f64(t):
    """float64 values of a GPU tensor (bf16 or fp32)."""
    return t.detach().double().cpu().numpy()


class Out:
    """[rows, width] output with sentinels before, after and in it."""

    def __init__(self, rows, width, dtype):
        per = 2 if dtype == torch.float32 else 1
        self.raw = torch.full(((rows * width + 32) * per,), SENT, dtype=torch.int16, device="cuda")
        self.t = self.raw[16 * per:(16 + rows * width) * per].view(dtype).view(rows, width)
        self.per, self.n = per, rows * width
        self.start = self.t.clone()

    def check(self, untouched=None):
        assert torch.all(self.raw[:16 * self.per] == SENT)
        assert torch.all(self.raw[(16 + self.n) * self.per:] == SENT)
        if untouched is not None:
            i = torch.int32 if self.per == 2 else torch.int16
            assert torch.equal(self.t.view(i)[untouched], self.start.view(i)[untouched])


def normal(seed, f32, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(shape, generator=g, device="cuda") * scale
    return t if f32 else t.bfloat16()


def rng_of(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def workspace(c, ec):
    return torch.full((mx.moe_epilogue_workspace_size(c, ec),), 0xA5, dtype=torch.uint8, device="cuda")


def products(x, w, expert):
    """x @ w[expert] by rows in float64, and the sums of the terms' magnitudes (GPU tensors)."""
    z = torch.zeros((x.shape[0], w.shape[2]), dtype=torch.float64, device="cuda")
    t = torch.zeros_like(z)
    for e in np.unique(expert[expert >= 0]):
        at = torch.from_numpy(np.nonzero(expert == e)[0]).cuda()
        xe, we = x.index_select(0, at).double(), w[int(e)].double()
        z[at], t[at] = xe @ we, xe.abs() @ we.abs()
    return z.cpu().numpy(), t.cpu().numpy()


def some_rows(n, seed, most=700):
    """All of n rows, or those around the first and last tiles' ends and others at random."""
    if n <= most:
        return np.arange(n)
    near = [b + d for b in (0, 16, 32, 64, 128, 256, n // 2, n // 128 * 128, n) for d in range(-2, 3)]
    pick = np.random.default_rng(seed).integers(0, n, most - len(near))
    return np.unique(np.clip(np.concatenate([near, pick]), 0, n - 1))


class Case:
    """One product: inputs on the GPU, the call, and the comparison."""

    def __init__(self, c, plan, expert, kind, bias=True, residual=False, f32=False, p=0.0, pre=False, seed=1,
                 ranks=None):
        self.c, self.plan, self.expert, self.kind = c, plan, expert, kind
        self.f32, self.p, self.ranks = f32, p, ranks or (0, c.R)
        rows = c.R * c.S * c.K
        self.ec = mx.make_epilogue_cfg(kind, p, f32)
        self.x = normal(seed, False, rows, c.H)
        self.w = normal(seed + 1, False, c.E, c.H, c.Hp, scale=c.H ** -0.5)
        self.w_pref = None
        if plan is not None and c.B:
            self.w_pref = torch.full((c.R * c.B, c.H, c.Hp), float("nan"), dtype=torch.bfloat16, device="cuda")
            mx.moe_prefetch_weight(c, plan, self.w, self.w_pref)
        self.bias = normal(seed + 2, True, c.E, c.Hp) if bias else None
        self.residual = normal(seed + 3, f32, rows, c.Hp) if residual else None
        self.rng = rng_of(1234567890123456789, -3 - seed) if p else None
        self.y = Out(rows, c.Hp, torch.float32 if f32 else torch.bfloat16)
        self.pre = Out(rows, c.Hp, torch.bfloat16) if pre else None
        self.ws = workspace(c, self.ec)

    def __call__(self, **over):
        a = {"xperm": self.x, "residual": self.residual, "y": self.y.t, **over}
        mx.moe_grouped_gemm_epilogue(self.c, self.ec, self.plan, a["xperm"], self.w, self.w_pref, self.bias,
                                     a["residual"], self.rng, a["y"], None if self.pre is None else self.pre.t,
                                     *self.ranks, self.ws)
        torch.cuda.synchronize()
        return self

    def check(self):
        c, SK = self.c, self.c.S * self.c.K
        row = np.arange(c.R * SK)
        live = (self.expert >= 0) & (row >= self.ranks[0] * SK) & (row < self.ranks[1] * SK)
        dead = torch.from_numpy(np.nonzero(~live)[0]).cuda()
        self.y.check(dead)
        at = np.nonzero(live)[0]
        at = at[some_rows(len(at), c.H)]
        idx = torch.from_numpy(at).cuda()
        take = lambda t: f64(t.index_select(0, idx))
        e = self.expert[at]
        z, terms = products(self.x.index_select(0, idx), self.w, e)
        if self.bias is not None:
            z = z + f64(self.bias)[e]
            terms = terms + np.abs(f64(self.bias)[e])
        dz = z_tol(c.H, terms)
        f = O.row_factor(self.p, [0, 0] if self.rng is None else self.rng.tolist(), at, c.Hp)
        res = None if self.residual is None else take(self.residual)
        close(take(self.y.t), O.forward(z, self.kind, self.p, [0, 0] if self.rng is None else self.rng.tolist(),
                                           res, at), product_tol(z, dz, self.kind, f, res, self.f32), "y")
        if self.pre is not None:
            self.pre.check(dead)
            close(take(self.pre.t), z, (1 + 2.0 ** -8) * dz + round_tol(z, False), "pre")
        return self


def matrix(S, H, Hp, kind, **kw):
    """A product with one matrix."""
    announce("matrix", S, H, Hp, kind, kw)
    c = mx.make_cfg(1, S, 1, 1, H, Hp, 0, mx.MODE_INFER)
    return Case(c, None, np.zeros(S, np.int64), kind, **kw)


def experts(shape, kind, ids=None, **kw):
    announce("experts", shape, kind, kw)
    ids = W.routing_zipf(shape, 1.0)[0] if ids is None else ids
    c, _ = cfgs(shape)
    plan, v = gpu_plan(shape, ids)
    expert = O.segment_experts(v["cu_seqlens"], v["slot_expert"], shape.E, shape.SK)
    return Case(c, plan, expert, kind, **kw)


# one row to many, on both sides of every block height; k that ends inside a step of 32 and
# columns that end inside a strip of 128
@pytest.mark.parametrize("S,H,Hp", [(1, 8, 8), (1, 1000, 520), (2, 2056, 136), (15, 40, 128), (16, 256, 384),
                                    (17, 104, 120), (33, 1000, 264), (64, 520, 256), (65, 72, 1032),
                                    (130, 264, 392), (257, 128, 64), (700, 136, 264), (1021, 200, 1544),
                                    (1300, 264, 520), (2600, 72, 8), (3000, 1032, 72)])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_one_matrix(S, H, Hp, f32):
    kind = (S + H) % 6
    matrix(S, H, Hp, kind, residual=S % 2 == 1, f32=f32, p=0.25 if S % 3 else 0.0, pre=S % 4 != 2,
           bias=S != 16, seed=S).__call__().check()


@pytest.mark.parametrize("kind", range(6))
@pytest.mark.parametrize("S", [5, 1500])
def test_activations(kind, S):
    """Products of a wide range: the far tails on both sides."""
    k = matrix(S, 64, 72, kind, f32=True, pre=True, seed=kind)
    k.x.mul_(8.0)
    k().check()


@pytest.mark.parametrize("shape,ids,ranks", [
    (W.TINY, None, None), (W.TINY, None, (1, 3)), (W.TINY.with_(S=1), None, None),
    (W.TINY.with_(H=1000, Hp=520), None, None), (W.TINY.with_(S=200, H=264, Hp=136), None, None),
    (W.TINY.with_(S=200, H=264, Hp=136), None, (2, 4)), (W.TINY.with_(S=1200, H=72, Hp=264), None, None),
    (W.TINY, "hot", None), (W.TINY.with_(S=300), "hot", None),
    (W.TINY.with_(mode=1, B=1), "hot", None), (W.TINY.with_(mode=1, B=0, S=150), "hot", None),
    (W.TINY.with_(R=1, B=0, mode=1, S=23, E=48, K=8), None, None),
], ids=str)
def test_experts(shape, ids, ranks):
    """Home rows, prefetch slots and overflow; both sides of every kernel choice."""
    picked = W.routing_hot(shape) if ids == "hot" else W.routing_uniform(shape, 3)[0]
    for n, kw in enumerate(({"residual": True, "p": 0.1, "pre": True}, {"f32": True}, {"bias": False})):
        experts(shape, (shape.S + n) % 6, picked, ranks=ranks, seed=10 * n + shape.S, **kw)().check()


# Each tile height and width, with the k axis whole and in parts, by the count of segments that
# every wave does itself (at most 512 of them) and by a list: what the time model picks for these
# sizes, by a margin where it can, is noted beside them.
@pytest.mark.parametrize("R,S,E,K,H,Hp,B", [
    (1, 2, 1, 1, 728, 24, 0), (1, 1, 1, 1, 5136, 6072, 0), (1, 13, 1, 1, 7160, 392, 0),   # 16 rows; in 6 and 12 parts
    (1, 943, 1, 1, 360, 1080, 0), (1, 567, 1, 1, 3376, 536, 0),               # 32 rows; in 3
    (1, 2406, 1, 1, 432, 824, 0), (1, 1485, 1, 1, 3824, 1392, 0),             # 128 x 128; in 3
    (1, 6881, 1, 1, 360, 7016, 0), (1, 653, 1, 1, 7064, 5520, 0),             # 128 x 256; in 3
    (1, 1, 2, 2, 792, 360, 0), (1, 1, 2, 1, 3176, 24, 0),                     # 16 rows; in 16
    (1, 2, 24, 2, 1200, 4832, 0), (1, 1, 24, 8, 2648, 2160, 0),               # 16 rows past the caches; in 3
    (1, 1283, 2, 1, 440, 832, 0), (1, 664, 2, 1, 4072, 432, 0),               # 32 rows; in 4
    (1, 37, 16, 1, 2440, 3496, 0), (1, 18, 16, 2, 5072, 1680, 0),             # 32 rows past the caches; in 2
    (1, 944, 2, 2, 432, 1312, 0), (1, 562, 2, 2, 3064, 1808, 0),              # 128 x 128; in 3
    (1, 3570, 2, 2, 376, 6352, 0), (1, 905, 2, 1, 6424, 3248, 0),             # 128 x 256; in 3
    # 128 x 128 by two groups of waves: whole (one, three and 16 steps), in 8 parts; by two workgroups a unit
    (1, 5660, 4, 1, 32, 512, 0), (1, 2830, 4, 2, 176, 560, 0), (1, 2744, 1, 1, 160, 1144, 0),
    (1, 4100, 8, 1, 1000, 520, 0), (1, 3749, 1, 1, 2584, 24, 0), (1, 1713, 4, 2, 4152, 40, 0),
    (1, 2609, 1, 1, 264, 1920, 0), (1, 5285, 8, 1, 128, 1328, 0),
    (8, 1, 128, 2, 496, 32, 16), (4, 67, 128, 2, 2296, 16, 32),               # by a list: 16 rows; in 3
    (4, 31, 128, 2, 2120, 152, 32), (4, 5, 128, 2, 856, 1424, 32),            # 32 rows; past the caches
    (4, 5, 128, 2, 2608, 480, 32), (4, 293, 128, 2, 40, 176, 32),             # 32 rows in 3; 128 x 128
    (4, 39, 128, 2, 408, 6568, 32)])                                          # 128 x 256
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_every_tile(R, S, E, K, H, Hp, B, f32):
    kind, kw = (S + H // 8) % 6, {"residual": True, "f32": f32, "p": 0.1, "pre": True, "seed": S}
    if E == 1:
        matrix(S, H, Hp, kind, **kw)().check()
        return
    s = W.TINY.with_(R=R, S=S, E=E, K=K, H=H, Hp=Hp, B=B, mode=0 if B else 1)
    k = experts(s, kind, W.routing_uniform(s, 6)[0], **kw)()
    k.check()
    y = k.y.t.clone()
    k.ws.fill_(0x11)                                       # nothing in the workspace matters
    k()
    i = torch.int32 if f32 else torch.int16
    assert torch.equal(y.view(i), k.y.t.view(i))


def test_failed_plan_writes_nothing():
    for S in (16, 400):
        s = W.TINY.with_(S=S)
        ids = W.routing_uniform(s)[0].copy()
        ids[3, 1] = s.E
        k = experts(s, O.GELU, ids, pre=True)
        assert np.all(k.expert == -1)
        k().check()


@pytest.mark.parametrize("R,S,E,K,H,Hp,B", [
    (1, 1, 2, 1, 3176, 24, 0), (1, 664, 2, 1, 4072, 432, 0), (1, 562, 2, 2, 3064, 1808, 0),
    (1, 905, 2, 1, 6424, 3248, 0), (4, 67, 128, 2, 2296, 16, 32)])
def test_failed_plan_in_parts_writes_nothing(R, S, E, K, H, Hp, B):
    """The same where the k axis is cut and the parts are added by a kernel of their own."""
    s = W.TINY.with_(R=R, S=S, E=E, K=K, H=H, Hp=Hp, B=B, mode=0 if B else 1)
    ids = W.routing_uniform(s)[0].copy()
    ids[0, 0] = s.E
    k = experts(s, O.NONE, ids, pre=True, residual=True)
    assert np.all(k.expert == -1)
    k().check()


def test_no_rows():
    c = mx.make_cfg(1, 0, 1, 1, 64, 64, 0, mx.MODE_INFER)
    ec = mx.make_epilogue_cfg(O.GELU)
    t = torch.zeros(64 * 64, dtype=torch.bfloat16, device="cuda")
    mx.moe_grouped_gemm_epilogue(c, ec, None, t, t, None, None, None, None, t, None, 0, 1, workspace(c, ec))
    db = torch.full((1, 64), 3.0, device="cuda")
    mx.moe_epilogue_backward(c, ec, None, t, t, None, None, db, workspace(c, ec))
    torch.cuda.synchronize()
    assert torch.all(db == 0) and torch.all(t == 0)


@pytest.mark.parametrize("S", [7, 40, 1400])
def test_in_place_and_repeatable(S):
    k = matrix(S, 520, 264, O.SILU, residual=True, p=0.5, seed=4)().check()
    y = k.y.t.clone()
    k.ws.fill_(0x3C)
    k()
    assert torch.equal(y.view(torch.int16), k.y.t.view(torch.int16))
    buf = k.residual.clone()
    k(residual=buf, y=buf)
    assert torch.equal(y.view(torch.int16), buf.view(torch.int16))


# k ends inside a step, columns inside a strip; every tile shape, and parts of the k axis
@pytest.mark.parametrize("S,H,Hp", [(4, 136, 152), (100, 136, 152), (1400, 136, 152), (13, 7144, 392),
                                    (943, 360, 1080), (567, 3376, 536), (2406, 424, 824), (1485, 3832, 1392),
                                    (6881, 360, 7016), (653, 7064, 5520)])
def test_rows_and_columns_are_apart(S, H, Hp):
    """Infinities and NaN stay in the rows and columns whose definition has them."""
    k = matrix(S, H, Hp, O.NONE, residual=True, p=0.0, seed=6)()
    clean = k.y.t.clone()
    k.x[S // 2] = float("nan")
    k.w[0, :, 5] = float("inf")
    k.w[0, H - 1, Hp - 1] = float("nan")
    k.residual[0, 9] = float("-inf")
    k()
    ok = torch.ones((S, Hp), dtype=torch.bool, device="cuda")
    ok[S // 2] = ok[:, 5] = ok[:, Hp - 1] = False
    ok[0, 9] = False
    assert torch.equal(k.y.t[ok].view(torch.int16), clean[ok].view(torch.int16))
    assert torch.all(~torch.isfinite(k.y.t[~ok]))
    assert torch.isnan(k.y.t[:, Hp - 1]).all() and torch.isnan(k.y.t[S // 2]).all()


@pytest.mark.parametrize("shape", [W.TINY.with_(H=136, Hp=72), W.TINY.with_(S=300, H=136, Hp=72),
                                   W.TINY.with_(R=4, S=225, E=64, K=2, H=632, Hp=744, B=16),
                                   W.TINY.with_(R=4, S=293, E=128, K=2, H=40, Hp=176, B=32)], ids=str)
def test_neighbours_do_not_leak(shape):
    """Rows of other segments and weights of other experts are NaN; one segment is clean."""
    k = experts(shape, O.GELU, W.routing_uniform(shape, 5)[0], seed=7)()
    clean = k.y.t.clone()
    e = int(np.bincount(k.expert[k.expert >= 0]).argmax())
    keep = torch.from_numpy(k.expert == e).cuda()
    others = torch.arange(shape.E, device="cuda") != e
    k.x[~keep] = float("nan")
    k.bias[others] = float("nan")
    k.w[others] = float("nan")
    mx.moe_prefetch_weight(k.c, k.plan, k.w, k.w_pref)
    k()
    assert torch.equal(k.y.t[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert torch.isnan(k.y.t[~keep]).all()


def test_special_values_of_the_activations():
    """+-infinity, NaN and zeros as bias on zero products."""
    vals = [float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 1e30, -1e30, 3e38]
    for S in (3, 1300):
        for kind in range(6):
            k = matrix(S, 16, 8, kind, f32=True, pre=True, seed=1)
            k.x.zero_()
            k.bias[0] = torch.tensor(vals)
            k()
            got = k.y.t[0].tolist()
            big = float("inf") if kind == O.RELU2 else 1e30
            assert got[0] == float("inf") and np.isnan(got[2]) and got[3] == got[4] == 0
            assert got[5] == pytest.approx(big) and got[7] > 2e38
            if kind == O.NONE:
                assert got[1] == float("-inf") and got[6] == pytest.approx(-1e30)
            elif kind in (O.RELU, O.RELU2):
                assert got[1] == 0 and got[6] == 0
            else:
                assert np.isnan(got[1]) and got[6] == 0       # -inf * 0; the tail of -1e30 is 0
            assert torch.equal(k.y.t, k.y.t[:1].expand(S, 8)) or np.isnan(got[2])


def test_dropout_extremes():
    for S in (5, 1300):
        k = matrix(S, 64, 72, O.GELU, residual=True, p=1.0, seed=2)()
        assert torch.equal(k.y.t, k.residual)                # everything dropped
        k = matrix(S, 64, 72, O.GELU, residual=True, p=2.0 ** -18, seed=2)()
        plain = matrix(S, 64, 72, O.GELU, residual=True, seed=2)()
        assert torch.equal(k.y.t, plain.y.t)                 # rounds to nothing


@pytest.mark.parametrize("S", [3, 48, 1400])
def test_captured_with_new_numbers(S):
    """Replays read rng's new contents; each equals the eager call."""
    k = matrix(S, 264, 136, O.SILU, residual=True, p=0.3, pre=True, seed=8)()
    db, dz = torch.zeros((1, 136), device="cuda"), torch.zeros_like(k.y.t)
    ws2 = workspace(k.c, k.ec)

    def step():
        mx.moe_grouped_gemm_epilogue(k.c, k.ec, None, k.x, k.w, None, k.bias, k.residual, k.rng, k.y.t, k.pre.t, 0,
                                     1, k.ws)
        mx.moe_epilogue_backward(k.c, k.ec, None, k.y.t, k.pre.t, k.rng, dz, db, ws2)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in range(4):
        k.rng.copy_(rng_of(5, n))
        k.x.copy_(normal(100 + n, False, S, 264))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (k.y.t, k.pre.t, dz, db)]
        for t in (k.y.t, k.pre.t, dz, db):
            t.fill_(7)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (k.y.t, k.pre.t, dz, db)):
            assert torch.equal(a, b)
        k.check()


def test_two_streams():
    """Two calls in flight with workspaces of their own."""
    ks = [matrix(40, 1032, 520, O.GELU, p=0.1, residual=True, pre=True, seed=20 + i) for i in range(2)]
    ss = [torch.cuda.Stream() for _ in ks]
    torch.cuda.synchronize()
    for _ in range(10):
        for k, s in zip(ks, ss):
            mx.moe_grouped_gemm_epilogue(k.c, k.ec, None, k.x, k.w, None, k.bias, k.residual, k.rng, k.y.t, k.pre.t,
                                         0, 1, k.ws, s)
    torch.cuda.synchronize()
    for k in ks:
        k.check()


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------
def check_backward(c, plan, expert, kind, f32, p, seed, in_place=None, want_dz=True, want_db=True):
    announce("backward", c, kind, f32, p, seed, in_place)
    rows = c.R * c.S * c.K
    dy, pre = normal(seed, f32, rows, c.Hp), normal(seed + 1, False, rows, c.Hp, scale=2.0)
    rng = rng_of(-99, 1 << 40) if p else None
    ec = mx.make_epilogue_cfg(kind, p, f32)
    want = [f64(dy), f64(pre)]
    dz = Out(rows, c.Hp, torch.bfloat16) if want_dz else None
    db = Out(c.E, c.Hp, torch.float32) if want_db else None
    dzt = {None: dz.t if want_dz else None, "dy": dy, "pre": pre}[in_place]
    mx.moe_epilogue_backward(c, ec, plan, dy, None if kind == O.NONE else pre, rng, dzt,
                             db.t if want_db else None, workspace(c, ec))
    torch.cuda.synchronize()
    r = [0, 0] if rng is None else rng.tolist()
    f = O.row_factor(p, r, np.arange(rows), c.Hp)
    gz, gb = O.backward(want[0], want[1], kind, p, r, expert, c.E)
    err, tol = dz_tol(want[0], want[1], kind, f)
    if want_dz:
        close(f64(dzt), gz, tol, "dz")
        dz.check()
    if want_db:
        db.check()
        for e in range(c.E):
            at = expert == e
            bound = err[at].sum(0) + 2 * (at.sum() + 16) * h * (np.abs(gz[at]) + err[at]).sum(0)
            close(f64(db.t)[e], gb[e], bound, "dbias of %d" % e)


@pytest.mark.parametrize("S,Hp", [(1, 8), (3, 520), (63, 512), (64, 1032), (257, 264), (5000, 72), (70000, 16)])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_backward_one_matrix(S, Hp, f32):
    c = mx.make_cfg(1, S, 1, 1, 8, Hp, 0, mx.MODE_INFER)
    check_backward(c, None, np.zeros(S, np.int64), S % 6, f32, 0.25 if S % 2 else 0.0, S)


@pytest.mark.parametrize("kind", range(6))
@pytest.mark.parametrize("shape,ids", [
    (W.TINY, "uniform"), (W.TINY.with_(S=300, Hp=520), "uniform"), (W.TINY.with_(S=90), "hot"),
    (W.TINY.with_(mode=1, B=1, S=90), "hot"), (W.TINY.with_(mode=1, B=0), "hot"), (W.TINY, "failed"),
    (W.TINY.with_(R=2, E=96, B=48, S=20, K=3), "uniform")], ids=str)
def test_backward_experts(kind, shape, ids):
    picked = (W.routing_hot(shape) if ids == "hot" else W.routing_uniform(shape, 2)[0]).copy()
    if ids == "failed":
        picked[0, 0] = -1
    c, _ = cfgs(shape)
    plan, v = gpu_plan(shape, picked)
    expert = O.segment_experts(v["cu_seqlens"], v["slot_expert"], shape.E, shape.SK)
    check_backward(c, plan, expert, kind, kind % 2 == 0, 0.1 * (kind % 3), kind)


@pytest.mark.parametrize("in_place", ["dy", "pre"])
def test_backward_in_place(in_place):
    c = mx.make_cfg(1, 333, 1, 1, 8, 520, 0, mx.MODE_INFER)
    check_backward(c, None, np.zeros(333, np.int64), O.GELU, False, 0.1, 3, in_place)


def test_backward_each_part_alone():
    c = mx.make_cfg(1, 100, 1, 1, 8, 72, 0, mx.MODE_INFER)
    e = np.zeros(100, np.int64)
    check_backward(c, None, e, O.SILU, True, 0.1, 3, want_dz=False)
    check_backward(c, None, e, O.SILU, False, 0.1, 3, want_db=False)
    # dz alone needs neither plan nor workspace
    s = W.TINY
    cc, _ = cfgs(s)
    rows = s.R * s.SK
    dy, pre = normal(1, False, rows, s.Hp), normal(2, False, rows, s.Hp)
    dz = torch.empty_like(dy)
    mx.moe_epilogue_backward(cc, mx.make_epilogue_cfg(O.RELU2), None, dy, pre, None, dz, None)
    torch.cuda.synchronize()
    err, tol = dz_tol(f64(dy), f64(pre), O.RELU2, 1.0)
    close(f64(dz), f64(dy) * O.slope(f64(pre), O.RELU2), tol, "dz")


def test_backward_repeats_bit_for_bit():
    s = W.TINY.with_(S=700, Hp=264)
    c, _ = cfgs(s)
    plan, _ = gpu_plan(s, W.routing_uniform(s, 2)[0])
    ec = mx.make_epilogue_cfg(O.GELU, 0.1)
    rows = s.R * s.SK
    dy, pre, rng = normal(1, False, rows, s.Hp), normal(2, False, rows, s.Hp), rng_of(1, 2)
    dz, db, ws = torch.empty_like(dy), torch.empty((s.E, s.Hp), device="cuda"), workspace(c, ec)
    first = None
    for n in range(3):
        ws.fill_(n)
        mx.moe_epilogue_backward(c, ec, plan, dy, pre, rng, dz, db, ws)
        torch.cuda.synchronize()
        first = (dz.clone(), db.clone()) if first is None else first
        assert torch.equal(first[0], dz) and torch.equal(first[1], db)


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------
def test_many_rows():
    """More than 2^31 output values: rows at the start, around the border and at the end."""
    S, H, Hp = (1 << 31) // 2048 + 700, 8, 2048
    announce("many rows", S, H, Hp)
    c = mx.make_cfg(4, S // 4 + 1, 4, 1, H, Hp, 0, mx.MODE_INFER)     # S K max(H, Hp) 2 < 4 GiB a rank
    plan = mx.Plan(c)
    per = c.S
    cu = torch.zeros((4, 5), dtype=torch.int32)
    for r in range(4):
        cu[r, r + 1:] = per
    plan.cu_seqlens[:20].copy_(cu.reshape(-1))
    rows = 4 * per
    ec = mx.make_epilogue_cfg(O.SILU, 0.5)
    x, w, bias = normal(1, False, rows, H), normal(2, False, 4, H, Hp), normal(3, True, 4, Hp)
    y = torch.empty((rows, Hp), dtype=torch.bfloat16, device="cuda")
    pre, rng, ws = torch.empty_like(y), rng_of(9, 9), workspace(c, ec)
    mx.moe_grouped_gemm_epilogue(c, ec, plan, x, w, None, bias, None, rng, y, pre, 0, 4, ws)
    mid = (1 << 31) // Hp
    at = np.concatenate([np.arange(5), np.arange(per - 3, per + 3), np.arange(mid - 3, mid + 3),
                         np.arange(rows - 5, rows)])
    idx = torch.from_numpy(at).cuda()
    e = at // per
    z, t = products(x.index_select(0, idx), w, e)
    z, t = z + f64(bias)[e], t + np.abs(f64(bias)[e])
    dz = z_tol(H, t)
    f = O.row_factor(0.5, [9, 9], at, Hp)
    close(f64(y.index_select(0, idx)), O.forward(z, O.SILU, 0.5, [9, 9], None, at),
          product_tol(z, dz, O.SILU, f, None, False), "y")
    close(f64(pre.index_select(0, idx)), z, 1.01 * dz + round_tol(z, False), "pre")
    # and back, in place
    want_pre = f64(pre.index_select(0, idx))
    db = torch.empty((4, Hp), device="cuda")
    dy = y
    dy.fill_(0.5)
    mx.moe_epilogue_backward(c, ec, plan, dy, pre, rng, dy, db, ws)
    torch.cuda.synchronize()
    _, tol = dz_tol(np.full_like(want_pre, 0.5), want_pre, O.SILU, f)
    close(f64(dy.index_select(0, idx)), 0.5 * f * O.slope(want_pre, O.SILU), tol, "dz")
    for r in range(4):                                     # the sums of the rounded gradients
        part = dy[r * per:(r + 1) * per]
        want, mag = torch.zeros(Hp, dtype=torch.float64, device="cuda"), 0
        for lo in range(0, per, 1 << 15):
            d = part[lo:lo + (1 << 15)].double()
            want += d.sum(0)
            mag = mag + d.abs().sum(0)
        # each term off by its rounding, and one step of fp32 for each addition of a path: a
        # chunk's rows (64 and 3) and the chunks of a rank over 16 lanes (rows / 4096 and 15)
        bound = (2.0 ** -8 * 1.01 + 2 * (90 + per // 2048) * h) * mag
        close(db[r].double().cpu().numpy(), want.cpu().numpy(), bound.cpu().numpy(), "dbias")
