"""Arguments that the epilogue and dropout entry points refuse before any launch (CPU)."""
import ctypes
import os

import pytest

import moe_expert_load_amd as mx

E, L, OK = mx.MOE_EINVAL, mx.MOE_ELIMIT, mx.MOE_OK


def at(n):
    return ctypes.c_void_p((1 << 40) + n)


def far(i):
    """Aligned addresses, 16 GiB apart."""
    return at(i << 34)


CFG = mx.make_cfg(4, 16, 8, 2, 128, 64, 2)             # 128 rows of 128 onto 64
ONE = mx.make_cfg(1, 33, 1, 1, 128, 64, 0, mx.MODE_INFER)
PLAN = mx.moe_plan(*[ctypes.c_void_p((1 << 24) + (i << 16)) for i in range(len(mx.PLAN_FIELDS))])


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        from moe_expert_load_amd import build
        build.build()
    return mx.load()


def ref(c):
    return ctypes.byref(c) if c is not None else None


BAD_EC = [mx.make_epilogue_cfg(-1), mx.make_epilogue_cfg(6), mx.make_epilogue_cfg(0, -0.1),
          mx.make_epilogue_cfg(0, 1.001), mx.make_epilogue_cfg(0, float("nan")),
          mx.moe_epilogue_cfg(0, 0.0, 2), mx.moe_epilogue_cfg(0, 0.0, -1)]
BAD_DC = [mx.make_dropout_cfg(-0.1), mx.make_dropout_cfg(1.5), mx.make_dropout_cfg(float("nan")),
          mx.moe_dropout_cfg(0.1, 2)]

# every tensor in a place of its own; by position: x, w, w_pref, bias, residual, rng, y, pre
NAMES = ["x", "w", "w_pref", "bias", "residual", "rng", "y", "pre"]


def product(lib, cfg=CFG, ec=None, plan=PLAN, rb=0, re=4, ws=far(20), **over):
    ec = mx.make_epilogue_cfg(mx.ACT_GELU, 0.1, False) if ec is None else ec
    a = [over.get(n, far(i + 1)) for i, n in enumerate(NAMES)]
    return lib.moe_grouped_gemm_epilogue(ref(cfg), ref(ec), ref(plan), *a, rb, re, ws, None)


def test_product_arguments(lib):
    assert product(lib, cfg=mx.make_cfg(4, 16, 8, 2, 100, 64, 2)) == E
    for ec in BAD_EC:
        assert product(lib, ec=ec) == E
    assert lib.moe_grouped_gemm_epilogue(ref(CFG), None, ref(PLAN), *[far(i + 1) for i in range(8)], 0, 4,
                                         far(20), None) == E
    assert product(lib, rb=-1) == E and product(lib, re=5) == E and product(lib, rb=3, re=2) == E
    assert product(lib, rb=2, re=2) == OK
    assert product(lib, plan=None) == E                                # E = 8 needs a plan
    for name in ("x", "w", "w_pref", "rng", "y"):
        assert product(lib, **{name: None}) == E, name
    assert product(lib, ws=None) == E
    no_cu = mx.moe_plan.from_buffer_copy(PLAN)
    no_cu.cu_seqlens = None
    no_slots = mx.moe_plan.from_buffer_copy(PLAN)
    no_slots.slot_expert = None
    assert product(lib, plan=no_cu) == E and product(lib, plan=no_slots) == E
    for i, name in enumerate(NAMES):
        if name != "rng":
            assert product(lib, **{name: at(((i + 1) << 34) + 8)}) == E, name
    assert product(lib, ws=at((20 << 34) + 8)) == E
    empty = mx.make_cfg(4, 0, 8, 2, 128, 64, 2)
    assert product(lib, cfg=empty, x=None, w=None, y=None) == OK


def test_product_overlaps(lib):
    y = 7 << 34
    rows, out = 128, 128 * 64 * 2
    ws = mx.moe_epilogue_workspace_size(CFG, mx.make_epilogue_cfg())
    for name in ("x", "w", "w_pref", "bias", "pre"):
        assert product(lib, **{name: at(y + out - 16)}) == E, name
    assert product(lib, residual=at(y + 16)) == E                      # in place only exactly
    assert product(lib, residual=at(y - 16)) == E
    assert product(lib, rng=at(y + 8)) == E
    assert product(lib, pre=far(5)) == E                               # pre over the residual
    assert product(lib, pre=far(1)) == E
    for i in range(1, 9):
        assert product(lib, ws=far(i)) == E, i
    assert product(lib, ws=at(y - ws + 16)) == E
    f32 = mx.make_epilogue_cfg(mx.ACT_NONE, 0.0, True)                 # y is twice as long
    assert product(lib, ec=f32, x=at(y + out)) == E
    plan = mx.moe_plan.from_buffer_copy(PLAN)
    plan.cu_seqlens = (1 << 40) + y
    assert product(lib, plan=plan) == E
    plan = mx.moe_plan.from_buffer_copy(PLAN)
    plan.slot_expert = (1 << 40) + y
    assert product(lib, plan=plan) == E


def test_rng_boundary(lib):
    """Two int64 on their own boundary, wherever something is dropped."""
    odd = at((40 << 34) + 4)
    dc, c, p = ref(mx.make_dropout_cfg(0.1)), ref(CFG), ref(PLAN)
    assert product(lib, rng=odd) == E and backward(lib, rng=odd) == E
    assert lib.moe_dropout(dc, 4, 64, far(1), far(2), odd, far(4), None) == E
    assert lib.moe_combine_dropout(c, dc, p, far(1), far(2), far(3), odd, far(5), None) == E
    assert lib.moe_combine_dropout_backward(c, dc, p, far(1), far(2), far(3), odd, far(5), far(6), None) == E


def test_too_many_tiles(lib):
    big = mx.make_cfg(1024, 16383, 2048, 64, 8, 2040, 0, mx.MODE_INFER)   # 2^30 rows, 8 tiles wide
    wide = {n: ctypes.c_void_p((i + 1) << 46) for i, n in enumerate(NAMES)}
    assert product(lib, cfg=big, re=1024, ws=ctypes.c_void_p(20 << 46), **wide) == L


def test_one_matrix_arguments(lib):
    assert product(lib, cfg=ONE, plan=None, re=1, y=None) == E
    assert product(lib, cfg=ONE, plan=None, re=1, x=at((1 << 34) + 4)) == E
    assert product(lib, cfg=ONE, plan=None, re=2) == E


def test_workspace_size(lib):
    size = ctypes.c_size_t()
    ec = mx.make_epilogue_cfg()
    assert lib.moe_epilogue_workspace_size(ref(CFG), None, ctypes.byref(size)) == E
    assert lib.moe_epilogue_workspace_size(ref(CFG), ref(ec), None) == E
    assert lib.moe_epilogue_workspace_size(ref(mx.make_cfg(4, 16, 8, 2, 128, 60, 2)), ref(ec),
                                           ctypes.byref(size)) == E
    for c in (CFG, ONE, mx.make_cfg(8, 8192, 384, 8, 7168, 2048, 48), mx.make_cfg(4, 0, 8, 2, 128, 64, 2)):
        assert mx.moe_epilogue_workspace_size(c, ec) >= mx.moe_gemm_workspace_size(c) // 2 > 0


def backward(lib, cfg=CFG, ec=None, plan=PLAN, dy=far(1), pre=far(2), rng=far(3), dz=far(4), dbias=far(5),
             ws=far(6)):
    ec = mx.make_epilogue_cfg(mx.ACT_GELU, 0.1, False) if ec is None else ec
    return lib.moe_epilogue_backward(ref(cfg), ref(ec), ref(plan), dy, pre, rng, dz, dbias, ws, None)


def test_backward_arguments(lib):
    for ec in BAD_EC:
        assert backward(lib, ec=ec) == E
    assert backward(lib, dz=None, dbias=None) == E
    for name in ("dy", "pre", "rng", "ws", "plan"):
        assert backward(lib, **{name: None}) == E, name
    for i, name in enumerate(("dy", "pre", "rng", "dz", "dbias", "ws")):
        if name != "rng":
            assert backward(lib, **{name: at(((i + 1) << 34) + 8)}) == E, name
    n = 128 * 64 * 2
    # in place on dy or pre only exactly, and on dy only in bf16
    assert backward(lib, dz=at((1 << 34) + 16)) == E and backward(lib, dz=at((2 << 34) + 16)) == E
    assert backward(lib, ec=mx.make_epilogue_cfg(mx.ACT_GELU, 0.1, True), dz=far(1)) == E
    assert backward(lib, dbias=at((4 << 34) + n - 16)) == E
    assert backward(lib, dbias=far(1)) == E and backward(lib, dbias=far(2)) == E
    # an output in place does not allow a third tensor there
    assert backward(lib, dz=far(1), dbias=far(1)) == E and backward(lib, dz=far(1), ws=far(1)) == E
    for i in range(1, 6):
        assert backward(lib, ws=far(i)) == E, i
    assert backward(lib, rng=at((4 << 34) + 8)) == E


def test_dropout_arguments(lib):
    dc = mx.make_dropout_cfg(0.1)
    f = lib.moe_dropout
    ok = [far(1), far(2), far(3), far(4)]                              # src, residual, rng, dst
    for bad in BAD_DC + [None]:
        assert f(ref(bad), 4, 64, *ok, None) == E
    for rows, width, code in ((-1, 64, E), (4, 0, E), (4, 12, E), (4, -8, E), (1 << 34, 64, L),
                              (1 << 60, 8, L), (0, 8, OK)):
        assert f(ref(dc), rows, width, *ok, None) == code, (rows, width)
    for i in (0, 2, 3):
        assert f(ref(dc), 4, 64, *[None if q == i else v for q, v in enumerate(ok)], None) == E
    for i in (0, 1, 3):
        assert f(ref(dc), 4, 64, *[at(((q + 1) << 34) + 8) if q == i else v for q, v in enumerate(ok)],
                 None) == E
    assert f(ref(dc), 4, 64, far(1), far(2), far(3), at((1 << 34) + 496), None) == E
    assert f(ref(dc), 4, 64, far(1), far(2), far(3), at((2 << 34) - 496), None) == E
    assert f(ref(dc), 4, 64, far(1), far(2), at((4 << 34) + 8), far(4), None) == E


def test_combine_arguments(lib):
    dc = mx.make_dropout_cfg(0.1)
    p = ref(PLAN)
    fwd = [far(1), far(2), far(3), far(4), far(5)]                     # y, gates, residual, rng, out
    f = lambda a, d=dc, pl=p, c=CFG: lib.moe_combine_dropout(ref(c), ref(d), pl, *a, None)
    put = lambda a, i, v: [v if q == i else w for q, w in enumerate(a)]
    for bad in BAD_DC + [None]:
        assert f(fwd, bad) == E
    assert f(fwd, pl=None) == E and f(fwd, c=mx.make_cfg(4, 16, 8, 2, 128, 60, 2)) == E
    assert f(fwd, c=mx.make_cfg(4, 0, 8, 2, 128, 64, 2)) == OK
    for i in (0, 1, 3, 4):
        assert f(put(fwd, i, None)) == E, i
    for i in (0, 2, 4):
        assert f(put(fwd, i, at(((i + 1) << 34) + 8))) == E, i
    for i in (0, 1):
        assert f(put(fwd, 4, far(i + 1))) == E
    assert f(put(fwd, 4, at((3 << 34) + 16))) == E                     # over the residual, not in place
    assert f(put(fwd, 3, at((5 << 34) + 8))) == E
    route = mx.moe_plan.from_buffer_copy(PLAN)
    route.route = (1 << 40) + (5 << 34)
    assert f(fwd, pl=ref(route)) == E
    bwd = [far(1), far(2), far(3), far(4), far(5), far(6)]             # dout, y, gates, rng, dy, dgates
    g = lambda a, d=dc, pl=p: lib.moe_combine_dropout_backward(ref(CFG), ref(d), pl, *a, None)
    for bad in BAD_DC + [None]:
        assert g(bwd, bad) == E
    for i in range(6):
        assert g(put(bwd, i, None)) == E, i
    for i in (0, 1, 4):
        assert g(put(bwd, i, at(((i + 1) << 34) + 8))) == E, i
    for i in (0, 1, 2, 3):
        assert g(put(bwd, 4, far(i + 1))) == E, i
    for i in (0, 1, 3, 4):
        assert g(put(bwd, 5, far(i + 1))) == E, i
    assert g(put(bwd, 5, at((3 << 34) + 4))) == E                      # over the gates, not in place
