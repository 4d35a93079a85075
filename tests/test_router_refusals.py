"""Arguments that the router's entry points refuse before any launch (CPU)."""
import ctypes
import os

import pytest

import moe_expert_load_amd as mx

A, M = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
CFG = (1, 4, 8, 2, 8, 8, 0, mx.MODE_INFER)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        from moe_expert_load_amd import build
        build.build()
    return mx.load()


def refs(cfg=CFG, **kw):
    r = mx.make_router_cfg(kw.get("score", 0), kw.get("renorm", 1), 1.0, kw.get("bf16", 0),
                           kw.get("nseq", 1))
    return ctypes.byref(mx.make_cfg(*cfg)), ctypes.byref(r)


@pytest.mark.parametrize("kw,code", [({"score": 2}, mx.MOE_EINVAL), ({"score": -1}, mx.MOE_EINVAL),
                                     ({"renorm": 2}, mx.MOE_EINVAL), ({"bf16": -1}, mx.MOE_EINVAL),
                                     ({"nseq": 0}, mx.MOE_EINVAL),
                                     ({"nseq": (1 << 20) + 1}, mx.MOE_ELIMIT)])
def test_settings(lib, kw, code):
    c, r = refs(**kw)
    n = ctypes.c_size_t()
    assert lib.moe_router_workspace_size(c, r, ctypes.byref(n)) == code
    assert lib.moe_router(c, r, A, None, A, A, None, None, None, None, None, None) == code
    assert lib.moe_balance_loss(c, r, A, A, A, A, A, A, A, None) == code
    assert lib.moe_router_backward(c, r, A, A, A, A, A, A, A, None) == code


def test_cfg_limits_apply(lib):
    n = ctypes.c_size_t()
    for cfg, code in [((1, 4, 8, 9, 8, 8, 0, 1), mx.MOE_EINVAL),
                      ((1, 4, 4096, 2, 8, 8, 0, 1), mx.MOE_ELIMIT),
                      ((1, 4, 2048, 65, 8, 8, 0, 1), mx.MOE_ELIMIT),
                      ((1, -1, 8, 2, 8, 8, 0, 1), mx.MOE_EINVAL)]:
        c, r = refs(cfg)
        assert lib.moe_router_workspace_size(c, r, ctypes.byref(n)) == code
        assert lib.moe_router(c, r, A, None, A, A, None, None, None, None, None, None) == code
    assert lib.moe_router_workspace_size(None, r, ctypes.byref(n)) == mx.MOE_EINVAL
    assert lib.moe_router_workspace_size(refs()[0], None, ctypes.byref(n)) == mx.MOE_EINVAL
    assert lib.moe_router_workspace_size(*refs(), None) == mx.MOE_EINVAL


def test_missing_and_misaligned(lib):
    c, r = refs()
    r2 = refs(nseq=2)[1]
    E = mx.MOE_EINVAL
    # logits, ids or gates missing
    for args in ((None, None, A, A), (A, None, None, A), (A, None, A, None)):
        assert lib.moe_router(c, r, *args, None, None, None, None, None, None) == E
    # the loss's outputs in part, without a workspace, two sequences without their ends
    for rest in ((None, A, None, None, A), (None, A, A, None, A), (None, None, A, A, A),
                 (None, A, A, A, None)):
        assert lib.moe_router(c, r, A, None, A, A, *rest, None) == E
    assert lib.moe_router(c, r2, A, None, A, A, None, A, A, A, A, None) == E
    assert lib.moe_balance_loss(c, r2, A, A, None, A, A, A, A, None) == E
    for i in range(7):
        args = [A, A, A, A, A, A, A]                        # logits ids cu counts prob loss ws
        args[i] = None
        if i != 2:                                          # one sequence needs no cu_tokens
            assert lib.moe_balance_loss(c, r, *args, None) == E, i
    # backward: neither gradient, one without what it needs
    assert lib.moe_router_backward(c, r, A, A, None, A, A, None, A, None) == E
    assert lib.moe_router_backward(c, r, A, None, A, A, A, None, A, None) == E
    assert lib.moe_router_backward(c, r, A, A, None, A, None, A, A, None) == E
    assert lib.moe_router_backward(c, r2, A, A, None, None, A, A, A, None) == E
    assert lib.moe_router_backward(c, r, None, A, A, A, A, A, A, None) == E
    assert lib.moe_router_backward(c, r, A, A, A, A, A, A, None, None) == E
    # floating tensors and the workspace off a 16-byte boundary
    assert lib.moe_router(c, r, M, None, A, A, None, None, None, None, None, None) == E
    assert lib.moe_router(c, r, A, M, A, A, None, None, None, None, None, None) == E
    assert lib.moe_router(c, r, A, None, A, M, None, None, None, None, None, None) == E
    assert lib.moe_router(c, r, A, None, A, A, None, A, M, A, A, None) == E
    assert lib.moe_router(c, r, A, None, A, A, None, A, A, M, A, None) == E
    assert lib.moe_router(c, r, A, None, A, A, None, A, A, A, M, None) == E
    assert lib.moe_balance_loss(c, r, M, A, None, A, A, A, A, None) == E
    assert lib.moe_router_backward(c, r, A, A, A, None, A, A, M, None) == E
    assert lib.moe_router_backward(c, r, A, A, M, None, A, A, A, None) == E
    # dlogits over a part of logits (4 x 8 fp32 = 128 bytes)
    for off in (16, 112, -112):
        part = ctypes.c_void_p((1 << 20) + off)
        assert lib.moe_router_backward(c, r, A, A, A, None, A, A, part, None) == E


def test_workspace_size_covers_every_piece():
    # chunks + sequences rows of E sums and E counts, and the joined double sums and counts
    for T, E, n in ((1, 8, 1), (1024, 384, 5), (1025, 384, 1), (65536, 896, 64), (65536, 384, 1)):
        c = mx.make_cfg(1, T, E, 1, 8, 8, 0, mx.MODE_INFER)
        chunk = 8 * max(1, -(-T // 8192))
        chunks = -(-T // chunk)
        parts = 8 if chunks >= 256 * n else 1
        need = (chunks + n) * E * 8 + n * parts * E * 12
        assert need <= mx.moe_router_workspace_size(c, mx.make_router_cfg(0, 1, 1.0, 0, n)) < need + 256
