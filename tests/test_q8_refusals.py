"""Arguments that the 8-bit checkpoint entry points refuse before any launch (CPU)."""
import ctypes
import os

import pytest

import moe_expert_load_amd as mx


def at(n):
    return ctypes.c_void_p((1 << 32) + n)


A, M = at(0), at(8)
CFG = mx.make_cfg(4, 16, 8, 2, 128, 64, 2)             # 128 rows of 64
PLAN = mx.moe_plan(*[ctypes.c_void_p(1 << 24) for _ in mx.PLAN_FIELDS])
E, L = mx.MOE_EINVAL, mx.MOE_ELIMIT


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        from moe_expert_load_amd import build
        build.build()
    return mx.load()


@pytest.mark.parametrize("name", ["moe_q8_store", "moe_q8_load"])
def test_rows_and_widths(lib, name):
    f = getattr(lib, name)
    for rows, width, code in ((-1, 64, E), (4, 0, E), (4, 7, E), (4, 12, E), (4, -8, E),
                              (1 << 60, 64, L), (1 << 32, 1024, L), (0, 8, mx.MOE_OK)):
        assert f(rows, width, A, A, A, None) == code, (rows, width)
    for i in range(3):
        args = [A, A, A]
        args[i] = None
        assert f(4, 64, *args, None) == E
    # bf16 rows and codes on 16-byte boundaries; scale bytes anywhere
    order = (lambda x, q, s: (x, q, s)) if name == "moe_q8_store" else (lambda x, q, s: (q, s, x))
    B, C = at(1 << 16), at(1 << 17)
    assert f(4, 64, *order(M, B, C), None) == E
    assert f(4, 64, *order(A, at((1 << 16) + 8), C), None) == E
    # 512 bytes of rows, 256 of codes, 8 of scales: no two may share memory
    assert f(4, 64, *order(A, at(496), C), None) == E
    assert f(4, 64, *order(at(240), A, C), None) == E
    assert f(4, 64, *order(A, B, at(511)), None) == E
    assert f(4, 64, *order(A, B, at((1 << 16) + 255)), None) == E


def test_dispatch_and_combine(lib):
    c, p = ctypes.byref(CFG), ctypes.byref(PLAN)
    bad = mx.make_cfg(4, 16, 8, 2, 100, 64, 2)
    assert lib.moe_dispatch_q8(ctypes.byref(bad), p, A, A, A, None) == E
    assert lib.moe_dispatch_q8(c, None, A, A, A, None) == E
    for i in range(3):
        args = [A, A, A]
        args[i] = None
        assert lib.moe_dispatch_q8(c, p, *args, None) == E
    assert lib.moe_dispatch_q8(c, p, M, A, A, None) == E
    assert lib.moe_dispatch_q8(c, p, A, A, M, None) == E
    assert lib.moe_combine_backward_q8(c, None, A, A, A, A, A, A, None) == E
    for i in range(6):
        args = [A] * 6                                 # dout yq yscale gates dy dgates
        args[i] = None
        assert lib.moe_combine_backward_q8(c, p, *args, None) == E
        if i != 2:
            args[i] = M
            assert lib.moe_combine_backward_q8(c, p, *args, None) == E


def test_swiglu(lib):
    c = ctypes.byref(CFG)
    n = 128 * 64                                       # codes of one half
    hq, hs, da, dh, ac = at(0), at(4 * n), at(8 * n), at(16 * n), at(32 * n)
    f = lib.moe_swiglu_backward_q8
    for i in range(4):
        args = [hq, hs, da, dh, ac]
        args[i] = None
        assert f(c, *args, None) == E
    assert f(c, M, hs, da, dh, ac, None) == E
    assert f(c, hq, hs, at(8 * n + 8), dh, ac, None) == E
    assert f(c, hq, hs, da, at(16 * n + 8), ac, None) == E
    assert f(c, hq, hs, da, dh, at(32 * n + 8), None) == E
    # overlaps: dh13 with each input and with act; act with the codes, partly with dact
    assert f(c, hq, hs, da, at(2 * n - 16), ac, None) == E
    assert f(c, hq, hs, da, at(4 * n + 16), ac, None) == E
    assert f(c, hq, hs, da, at(10 * n - 16), ac, None) == E
    assert f(c, hq, hs, da, dh, at(20 * n - 16), None) == E
    assert f(c, hq, hs, da, dh, at(2 * n - 16), None) == E
    assert f(c, hq, hs, da, dh, at(8 * n + 16), None) == E
    g = lib.moe_grouped_gemm_swiglu_q8
    big = mx.make_cfg(8, 16, 8, 2, 65536, 16384, 1)
    assert g(ctypes.byref(big), *[None] * 7, 0, 8, None, None) == L
    assert g(c, *[None] * 7, 2, 2, None, None) == mx.MOE_OK
    assert g(c, *[A] * 7, 0, 5, A, None) == E
    for i in (0, 1, 2, 3, 4, 5, 6):
        args = [A] * 7                                 # xperm w13 pref cu act q scale
        args[i] = None
        assert g(c, *args, 0, 4, A, None) == E, i
    assert g(c, *[A] * 7, 0, 4, None, None) == E
    for i in (0, 1, 2, 4, 5):
        args = [A] * 7
        args[i] = M
        assert g(c, *args, 0, 4, A, None) == E, i
