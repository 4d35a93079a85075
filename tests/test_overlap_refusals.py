"""Tensors that share memory with an output are refused before any launch (CPU).

Addresses are made up; a call that passed the checks would launch, so every call here is one
that must be refused: the output reaches one byte, or one aligned step, into its neighbour.
"""
import ctypes
import os

import pytest

import moe_expert_load_amd as mx

R, S, E, K, H, Hp, B = 4, 16, 8, 2, 128, 64, 2         # 64 tokens, 128 rows
T, ROWS = R * S, R * S * K
CFG = mx.make_cfg(R, S, E, K, H, Hp, B)
PLAN = mx.moe_plan(*[ctypes.c_void_p(1 << 24) for _ in mx.PLAN_FIELDS])
FAR = 1 << 32
GAP = 1 << 28


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        from moe_expert_load_amd import build
        build.build()
    return mx.load()


def refused(call, sizes, pairs, step=16):
    """call(addresses) is refused whenever a pair (written, other) of `sizes`' tensors shares
    its first or its last bytes; the other tensors lie far apart."""
    order = list(sizes)
    base = {n: FAR + i * GAP for i, n in enumerate(order)}
    for w, o in pairs:
        for at in (base[o], base[o] + sizes[o] - 1 & -step, base[o] - sizes[w] + step & -step):
            a = dict(base)
            a[w] = at
            assert at < base[o] + sizes[o] and base[o] < at + sizes[w]
            assert call(a) == mx.MOE_EINVAL, (w, o, at - base[o])


def pointer(a):
    return {k: ctypes.c_void_p(v) for k, v in a.items()}


def test_dispatch_q8(lib):
    sizes = {"xq": T * H, "xscale": T * H // 32, "xperm": ROWS * H * 2}

    def call(a):
        p = pointer(a)
        return lib.moe_dispatch_q8(ctypes.byref(CFG), ctypes.byref(PLAN), p["xq"], p["xscale"],
                                   p["xperm"], None)
    refused(call, sizes, [("xperm", "xq"), ("xperm", "xscale")])


def test_combine_backward_q8(lib):
    sizes = {"dout": T * Hp * 2, "yq": ROWS * Hp, "yscale": ROWS * Hp // 32, "gates": ROWS * 4,
             "dy": ROWS * Hp * 2, "dgates": ROWS * 4}

    def call(a):
        p = pointer(a)
        if p["dgates"].value == p["gates"].value:           # in place is allowed
            return mx.MOE_EINVAL
        return lib.moe_combine_backward_q8(ctypes.byref(CFG), ctypes.byref(PLAN), p["dout"],
                                           p["yq"], p["yscale"], p["gates"], p["dy"], p["dgates"],
                                           None)
    ins = ("dout", "yq", "yscale", "gates")
    refused(call, sizes, [(w, o) for w in ("dy", "dgates") for o in ins] + [("dy", "dgates")])


def swiglu_q8(lib, begin, end):
    def call(a):
        p = pointer(a)
        return lib.moe_grouped_gemm_swiglu_q8(
            ctypes.byref(CFG), *[p[n] for n in ("xperm", "home", "pref", "cu", "act", "q", "s")],
            begin, end, p["ws"], None)
    return call


def test_grouped_gemm_swiglu_q8(lib):
    sizes = {"xperm": ROWS * H * 2, "home": E * H * 2 * Hp * 2, "pref": R * B * H * 2 * Hp * 2,
             "cu": R * (E + B + 1) * 4, "act": ROWS * Hp * 2, "q": ROWS * 2 * Hp,
             "s": ROWS * 2 * (Hp // 32), "ws": mx.moe_gemm_workspace_size(CFG)}
    outs = ("act", "q", "s", "ws")
    pairs = [(w, o) for w in outs for o in ("xperm", "home", "pref", "cu")]
    pairs += [(w, o) for i, w in enumerate(outs) for o in outs[:i]]
    refused(swiglu_q8(lib, 0, R), sizes, pairs)


def test_grouped_gemm_swiglu_q8_of_one_rank(lib):
    """Only the listed rank's parts count: act may start where that rank's rows of xperm end,
    and not 16 bytes before."""
    n = ROWS // R
    a = {k: FAR + i * GAP for i, k in enumerate(("xperm", "home", "pref", "cu", "act", "q", "s", "ws"))}
    first = a["xperm"] + n * H * 2                          # rank 1's rows of xperm
    for at in (first - n * Hp * 2 + 16, first, first + n * H * 2 - 16):
        assert swiglu_q8(lib, 1, 2)({**a, "act": at - n * Hp * 2}) == mx.MOE_EINVAL


NSEQ = 3
LOSS = {"logits": T * E * 4, "bias": E * 4, "ids": T * K * 4, "gates": T * K * 4,
        "cu": (NSEQ + 1) * 4, "counts": NSEQ * E * 4, "prob": NSEQ * E * 4, "loss": NSEQ * 4}


def settings():
    return mx.make_router_cfg(mx.SCORE_SOFTMAX, 1, 1.0, False, NSEQ)


def pairs_of(outs, ins):
    return [(w, o) for w in outs for o in ins] + [(w, o) for i, w in enumerate(outs) for o in outs[:i]]


def test_router(lib):
    rc = settings()
    sizes = {**LOSS, "ws": mx.moe_router_workspace_size(CFG, rc)}

    def loss(a):
        p = pointer(a)
        return lib.moe_router(ctypes.byref(CFG), ctypes.byref(rc),
                              *[p[n] for n in ("logits", "bias", "ids", "gates", "cu", "counts",
                                               "prob", "loss", "ws")], None)

    def plain(a):
        p = pointer(a)
        return lib.moe_router(ctypes.byref(CFG), ctypes.byref(rc),
                              *[p[n] for n in ("logits", "bias", "ids", "gates")], *[None] * 6)

    outs = ("ids", "gates", "counts", "prob", "loss", "ws")
    refused(loss, sizes, pairs_of(outs, ("logits", "bias", "cu")))
    refused(plain, sizes, pairs_of(("ids", "gates"), ("logits", "bias")))


def test_balance_loss(lib):
    rc = settings()
    sizes = {**LOSS, "ws": mx.moe_router_workspace_size(CFG, rc)}

    def call(a):
        p = pointer(a)
        return lib.moe_balance_loss(ctypes.byref(CFG), ctypes.byref(rc),
                                    *[p[n] for n in ("logits", "ids", "cu", "counts", "prob", "loss",
                                                     "ws")], None)
    refused(call, sizes, pairs_of(("counts", "prob", "loss", "ws"), ("logits", "ids", "cu")))


def test_router_backward(lib):
    rc = settings()
    sizes = {**LOSS, "dgates": T * K * 4, "dloss": NSEQ * 4, "dlogits": T * E * 4}

    def call(names):
        def f(a):
            p = {**pointer(a), None: None}
            return lib.moe_router_backward(ctypes.byref(CFG), ctypes.byref(rc), p["logits"],
                                           *[p[n] for n in names], p["dlogits"], None)
        return f

    both = ("ids", "dgates", "cu", "counts", "dloss")
    refused(call(both), sizes, pairs_of(("dlogits",), both))
    refused(call(("ids", "dgates", None, None, None)), sizes,
            pairs_of(("dlogits",), ("ids", "dgates")))
    refused(call((None, None, "cu", "counts", "dloss")), sizes,
            pairs_of(("dlogits",), ("cu", "counts", "dloss")))
    # logits: shifted by a step either way (in place is allowed)
    base = {n: FAR + i * GAP for i, n in enumerate(sizes)}
    for off in (16, -16, sizes["logits"] - 16, 16 - sizes["logits"]):
        assert call(both)({**base, "dlogits": base["logits"] + off}) == mx.MOE_EINVAL
