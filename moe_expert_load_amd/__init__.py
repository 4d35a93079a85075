"""Thin Python binding of libmoonep_hip.so (the MoonEP hot path on gfx950).

Argument marshalling only: every step runs in the HIP library.  Functions
carry the C entry points' names and take torch tensors that live on the GPU
(torch is used for device memory and the current stream).  The library must
have been built (``python -m moe_expert_load_amd.build``); without it every
call raises -- there is no CPU fallback.
"""
import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoonep_hip.so")

MOE_OK, MOE_EINVAL, MOE_EHIP, MOE_ELIMIT = 0, -1, -2, -3
MODE_TRAIN, MODE_INFER = 0, 1
STATUS_BAD_ID, STATUS_UNBALANCED, STATUS_CAPACITY, STATUS_INTERNAL = 1, 2, 4, 8
PLAN_ASCENDING, PLAN_LARGEST_FIRST = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU, ACT_RELU2 = range(6)
PLAN_FIELDS = ("counts", "load0", "route", "cu_seqlens", "slot_expert",
               "n_redundant", "src_rank", "moves", "status", "workspace")
ENTRY_POINTS = ("moe_plan_sizes", "moe_plan_run", "moe_plan_run_policy", "moe_prefetch_weight",
                "moe_dispatch", "moe_gemm_workspace_size", "moe_grouped_gemm",
                "moe_grouped_gemm_noalloc",
                "moe_combine", "moe_grouped_gemm_wgrad", "moe_reduce_grad",
                "moe_combine_backward", "moe_grouped_gemm_dgrad",
                "moe_dispatch_backward", "moe_route_encode", "moe_dispatch_dedup",
                "moe_grouped_gemm_swiglu", "moe_swiglu_backward",
                "moe_router_workspace_size", "moe_router", "moe_balance_loss",
                "moe_router_backward", "moe_q8_store", "moe_q8_load", "moe_dispatch_q8",
                "moe_grouped_gemm_swiglu_q8", "moe_swiglu_backward_q8",
                "moe_combine_backward_q8", "moe_epilogue_workspace_size",
                "moe_grouped_gemm_epilogue", "moe_epilogue_backward", "moe_dropout",
                "moe_combine_dropout", "moe_combine_dropout_backward", "moe_strerror")


class MoeError(RuntimeError):
    def __init__(self, code, where):
        super().__init__("%s failed: %s (%d)" % (where, moe_strerror(code), code))
        self.code = code


class moe_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "S", "E", "K", "H", "Hp", "B", "mode")]

    def __repr__(self):
        return "moe_cfg(%s)" % ", ".join("%s=%d" % (n, getattr(self, n)) for n, _ in self._fields_)


class moe_router_cfg(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("logits_bf16", ctypes.c_int32),
                ("nseq", ctypes.c_int32)]


class moe_epilogue_cfg(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("p", ctypes.c_float), ("f32", ctypes.c_int32)]


class moe_dropout_cfg(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("f32", ctypes.c_int32)]


class moe_plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in PLAN_FIELDS]


_lib = None


def load(path=None):
    """Load (once) and return the library; raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("MoonEP HIP library not built: %s is missing "
                           "(run python -m moe_expert_load_amd.build)" % p)
    lib = ctypes.CDLL(p)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    C = ctypes.POINTER(moe_cfg)
    PL = ctypes.POINTER(moe_plan)
    RC = ctypes.POINTER(moe_router_cfg)
    EC = ctypes.POINTER(moe_epilogue_cfg)
    DC = ctypes.POINTER(moe_dropout_cfg)
    sig = {
        "moe_plan_sizes": [C, ctypes.POINTER(SZ)],
        "moe_plan_run": [C, P, PL, P],
        "moe_plan_run_policy": [C, P, PL, I32, P],
        "moe_prefetch_weight": [C, PL, P, P, P],
        "moe_dispatch": [C, PL, P, P, P],
        "moe_gemm_workspace_size": [C, ctypes.POINTER(SZ)],
        "moe_grouped_gemm": [C, P, P, P, P, P, I32, I32, P, P],
        "moe_grouped_gemm_noalloc": [C, P, P, P, P, P, I32, I32, P],
        "moe_combine": [C, PL, P, P, P, P],
        "moe_grouped_gemm_wgrad": [C, PL, P, P, P, P, P, P],
        "moe_reduce_grad": [C, PL, P, P, P],
        "moe_combine_backward": [C, PL, P, P, P, P, P, P],
        "moe_grouped_gemm_dgrad": [C, P, P, P, P, P, I32, I32, P, P],
        "moe_dispatch_backward": [C, PL, P, P, P],
        "moe_route_encode": [C, PL, P, P],
        "moe_dispatch_dedup": [C, P, P, P, P],
        "moe_grouped_gemm_swiglu": [C, P, P, P, P, P, P, I32, I32, P, P],
        "moe_swiglu_backward": [C, P, P, P, P],
        "moe_router_workspace_size": [C, RC, ctypes.POINTER(SZ)],
        "moe_router": [C, RC, P, P, P, P, P, P, P, P, P, P],
        "moe_balance_loss": [C, RC, P, P, P, P, P, P, P, P],
        "moe_router_backward": [C, RC, P, P, P, P, P, P, P, P],
        "moe_q8_store": [I64, I32, P, P, P, P],
        "moe_q8_load": [I64, I32, P, P, P, P],
        "moe_dispatch_q8": [C, PL, P, P, P, P],
        "moe_grouped_gemm_swiglu_q8": [C, P, P, P, P, P, P, P, I32, I32, P, P],
        "moe_swiglu_backward_q8": [C, P, P, P, P, P, P],
        "moe_combine_backward_q8": [C, PL, P, P, P, P, P, P, P],
        "moe_epilogue_workspace_size": [C, EC, ctypes.POINTER(SZ)],
        "moe_grouped_gemm_epilogue": [C, EC, PL, P, P, P, P, P, P, P, P, I32, I32, P, P],
        "moe_epilogue_backward": [C, EC, PL, P, P, P, P, P, P, P],
        "moe_dropout": [DC, I64, I32, P, P, P, P, P],
        "moe_combine_dropout": [C, DC, PL, P, P, P, P, P, P],
        "moe_combine_dropout_backward": [C, DC, PL, P, P, P, P, P, P, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.moe_strerror.argtypes = [ctypes.c_int]
    lib.moe_strerror.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def make_cfg(R, S, E, K, H, Hp, B, mode=MODE_TRAIN):
    return moe_cfg(R, S, E, K, H, Hp, B, mode)


def _check(code, where):
    if code != MOE_OK:
        raise MoeError(code, where)


def _ptr(t, dtype, numel=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if numel is not None and t.numel() < numel:
        raise ValueError("%s holds %d elements, needs %d" % (name, t.numel(), numel))
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _arg(t, dtype, numel, name, device):
    """Address of a tensor that a kernel on `device` (the current one) may use.

    The checks and errors of _ptr, in one pass over cheap attributes: a
    decode-size call lasts only a few microseconds on the GPU.
    """
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device
            or t.numel() < numel or not t.is_contiguous()):
        _ptr(t, dtype, numel, name)
        raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, device))
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(stream, device):
    """_stream; the current stream's handle without making a Stream object (3 us)."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream(stream)


def moe_strerror(code):
    return load().moe_strerror(int(code)).decode()


def moe_plan_sizes(cfg):
    out = (ctypes.c_size_t * 10)()
    _check(load().moe_plan_sizes(ctypes.byref(cfg), out), "moe_plan_sizes")
    return [int(v) for v in out]


def moe_gemm_workspace_size(cfg):
    out = ctypes.c_size_t()
    _check(load().moe_gemm_workspace_size(ctypes.byref(cfg), ctypes.byref(out)),
           "moe_gemm_workspace_size")
    return int(out.value)


class Plan:
    """Device arrays of one moe_plan, allocated with torch (int32 + bytes)."""

    def __init__(self, cfg, device="cuda"):
        sizes = moe_plan_sizes(cfg)
        self.cfg = cfg
        self.arrays = {}
        for name, nbytes in zip(PLAN_FIELDS, sizes):
            if name == "workspace":
                self.arrays[name] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
            else:
                self.arrays[name] = torch.empty(max(nbytes // 4, 1), dtype=torch.int32, device=device)
        self._c = moe_plan(*[ctypes.c_void_p(self.arrays[n].data_ptr()) for n in PLAN_FIELDS])

    def __getattr__(self, name):
        arrays = self.__dict__.get("arrays")
        if arrays is not None and name in arrays:
            return arrays[name]
        raise AttributeError(name)

    @property
    def c(self):
        return ctypes.byref(self._c)

    # shaped views of the outputs
    def views(self):
        c = self.cfg
        a = self.arrays
        st = a["status"][:4]
        return {
            "counts": a["counts"][:c.E],
            "load0": a["load0"][:c.R],
            "route": a["route"][:c.R * c.S * c.K],
            "cu_seqlens": a["cu_seqlens"][:c.R * (c.E + c.B + 1)].view(c.R, c.E + c.B + 1),
            "slot_expert": a["slot_expert"][:c.R * c.B].view(c.R, c.B),
            "n_redundant": a["n_redundant"][:c.R],
            "src_rank": a["src_rank"][:c.R],
            "moves": a["moves"][:4 * (c.E + c.R - 1)].view(-1, 4),
            "status": st,
        }


def moe_plan_run(cfg, topk_ids, plan, stream=None):
    n = cfg.R * cfg.S * cfg.K
    ids = _ptr(topk_ids, torch.int32, n, "topk_ids") if n else None
    _check(load().moe_plan_run(ctypes.byref(cfg), ids, plan.c, _stream(stream)), "moe_plan_run")


def moe_plan_run_policy(cfg, topk_ids, plan, policy, stream=None):
    n = cfg.R * cfg.S * cfg.K
    ids = _ptr(topk_ids, torch.int32, n, "topk_ids") if n else None
    _check(load().moe_plan_run_policy(ctypes.byref(cfg), ids, plan.c, int(policy),
                                      _stream(stream)), "moe_plan_run_policy")


def moe_prefetch_weight(cfg, plan, w_home, w_pref, stream=None):
    hh = cfg.H * cfg.Hp
    a = _ptr(w_home, torch.bfloat16, cfg.E * hh, "w_home")
    b = _ptr(w_pref, torch.bfloat16, cfg.R * cfg.B * hh, "w_pref") if cfg.B else None
    _check(load().moe_prefetch_weight(ctypes.byref(cfg), plan.c, a, b, _stream(stream)),
           "moe_prefetch_weight")


def moe_dispatch(cfg, plan, x, xperm, stream=None):
    a = _ptr(x, torch.bfloat16, cfg.R * cfg.S * cfg.H, "x")
    b = _ptr(xperm, torch.bfloat16, cfg.R * cfg.S * cfg.K * cfg.H, "xperm")
    _check(load().moe_dispatch(ctypes.byref(cfg), plan.c, a, b, _stream(stream)), "moe_dispatch")


def moe_grouped_gemm(cfg, xperm, w_home, w_pref, cu_seqlens, y, rank_begin, rank_end,
                     workspace, stream=None):
    SK = cfg.S * cfg.K
    hh = cfg.H * cfg.Hp
    args = (ctypes.byref(cfg),
            _ptr(xperm, torch.bfloat16, cfg.R * SK * cfg.H, "xperm"),
            _ptr(w_home, torch.bfloat16, cfg.E * hh, "w_home"),
            _ptr(w_pref, torch.bfloat16, cfg.R * cfg.B * hh, "w_pref") if cfg.B else None,
            _ptr(cu_seqlens, torch.int32, cfg.R * (cfg.E + cfg.B + 1), "cu_seqlens"),
            _ptr(y, torch.bfloat16, cfg.R * SK * cfg.Hp, "y"),
            int(rank_begin), int(rank_end),
            _ptr(workspace, torch.uint8, moe_gemm_workspace_size(cfg), "workspace"),
            _stream(stream))
    _check(load().moe_grouped_gemm(*args), "moe_grouped_gemm")


def moe_grouped_gemm_noalloc(cfg, xperm, w_home, w_pref, cu_seqlens, y, rank_begin, rank_end,
                             stream=None):
    SK = cfg.S * cfg.K
    hh = cfg.H * cfg.Hp
    args = (ctypes.byref(cfg),
            _ptr(xperm, torch.bfloat16, cfg.R * SK * cfg.H, "xperm"),
            _ptr(w_home, torch.bfloat16, cfg.E * hh, "w_home"),
            _ptr(w_pref, torch.bfloat16, cfg.R * cfg.B * hh, "w_pref") if cfg.B else None,
            _ptr(cu_seqlens, torch.int32, cfg.R * (cfg.E + cfg.B + 1), "cu_seqlens"),
            _ptr(y, torch.bfloat16, cfg.R * SK * cfg.Hp, "y"),
            int(rank_begin), int(rank_end), _stream(stream))
    _check(load().moe_grouped_gemm_noalloc(*args), "moe_grouped_gemm_noalloc")


def moe_combine(cfg, plan, y, gates, out, stream=None):
    ntok = cfg.R * cfg.S
    a = _ptr(y, torch.bfloat16, ntok * cfg.K * cfg.Hp, "y")
    g = _ptr(gates, torch.float32, ntok * cfg.K, "gates")
    o = _ptr(out, torch.bfloat16, ntok * cfg.Hp, "out")
    _check(load().moe_combine(ctypes.byref(cfg), plan.c, a, g, o, _stream(stream)), "moe_combine")


def moe_grouped_gemm_wgrad(cfg, plan, xperm, dy, grad_home, grad_pref, workspace, stream=None):
    SK = cfg.S * cfg.K
    hh = cfg.H * cfg.Hp
    args = (ctypes.byref(cfg), plan.c,
            _ptr(xperm, torch.bfloat16, cfg.R * SK * cfg.H, "xperm"),
            _ptr(dy, torch.bfloat16, cfg.R * SK * cfg.Hp, "dy"),
            _ptr(grad_home, torch.float32, cfg.E * hh, "grad_home"),
            _ptr(grad_pref, torch.float32, cfg.R * cfg.B * hh, "grad_pref") if cfg.B else None,
            _ptr(workspace, torch.uint8, moe_gemm_workspace_size(cfg), "workspace"),
            _stream(stream))
    _check(load().moe_grouped_gemm_wgrad(*args), "moe_grouped_gemm_wgrad")


def moe_combine_backward(cfg, plan, dout, y, gates, dy, dgates, stream=None):
    ntok = cfg.R * cfg.S
    args = (ctypes.byref(cfg), plan.c,
            _ptr(dout, torch.bfloat16, ntok * cfg.Hp, "dout"),
            _ptr(y, torch.bfloat16, ntok * cfg.K * cfg.Hp, "y"),
            _ptr(gates, torch.float32, ntok * cfg.K, "gates"),
            _ptr(dy, torch.bfloat16, ntok * cfg.K * cfg.Hp, "dy"),
            _ptr(dgates, torch.float32, ntok * cfg.K, "dgates"),
            _stream(stream))
    _check(load().moe_combine_backward(*args), "moe_combine_backward")


def moe_grouped_gemm_dgrad(cfg, dy, w_home, w_pref, cu_seqlens, dxperm, rank_begin, rank_end,
                           workspace, stream=None):
    SK = cfg.S * cfg.K
    hh = cfg.H * cfg.Hp
    args = (ctypes.byref(cfg),
            _ptr(dy, torch.bfloat16, cfg.R * SK * cfg.Hp, "dy"),
            _ptr(w_home, torch.bfloat16, cfg.E * hh, "w_home"),
            _ptr(w_pref, torch.bfloat16, cfg.R * cfg.B * hh, "w_pref") if cfg.B else None,
            _ptr(cu_seqlens, torch.int32, cfg.R * (cfg.E + cfg.B + 1), "cu_seqlens"),
            _ptr(dxperm, torch.bfloat16, cfg.R * SK * cfg.H, "dxperm"),
            int(rank_begin), int(rank_end),
            _ptr(workspace, torch.uint8, moe_gemm_workspace_size(cfg), "workspace"),
            _stream(stream))
    _check(load().moe_grouped_gemm_dgrad(*args), "moe_grouped_gemm_dgrad")


def moe_grouped_gemm_swiglu(cfg, xperm, w13_home, w13_pref, cu_seqlens, act, h13, rank_begin,
                            rank_end, workspace, stream=None):
    """cfg.Hp is the intermediate size H'; W13 rows are [H][2H'] (gate | up)."""
    SK = cfg.S * cfg.K
    hh = cfg.H * 2 * cfg.Hp
    args = (ctypes.byref(cfg),
            _ptr(xperm, torch.bfloat16, cfg.R * SK * cfg.H, "xperm"),
            _ptr(w13_home, torch.bfloat16, cfg.E * hh, "w13_home"),
            _ptr(w13_pref, torch.bfloat16, cfg.R * cfg.B * hh, "w13_pref") if cfg.B else None,
            _ptr(cu_seqlens, torch.int32, cfg.R * (cfg.E + cfg.B + 1), "cu_seqlens"),
            _ptr(act, torch.bfloat16, cfg.R * SK * cfg.Hp, "act"),
            _ptr(h13, torch.bfloat16, cfg.R * SK * 2 * cfg.Hp, "h13"),
            int(rank_begin), int(rank_end),
            _ptr(workspace, torch.uint8, moe_gemm_workspace_size(cfg), "workspace"),
            _stream(stream))
    _check(load().moe_grouped_gemm_swiglu(*args), "moe_grouped_gemm_swiglu")


def moe_swiglu_backward(cfg, h13, dact, dh13, stream=None):
    rows = cfg.R * cfg.S * cfg.K
    args = (ctypes.byref(cfg),
            _ptr(h13, torch.bfloat16, rows * 2 * cfg.Hp, "h13"),
            _ptr(dact, torch.bfloat16, rows * cfg.Hp, "dact"),
            _ptr(dh13, torch.bfloat16, rows * 2 * cfg.Hp, "dh13"),
            _stream(stream))
    _check(load().moe_swiglu_backward(*args), "moe_swiglu_backward")


def moe_dispatch_backward(cfg, plan, dxperm, dx, stream=None):
    ntok = cfg.R * cfg.S
    a = _ptr(dxperm, torch.bfloat16, ntok * cfg.K * cfg.H, "dxperm")
    o = _ptr(dx, torch.bfloat16, ntok * cfg.H, "dx")
    _check(load().moe_dispatch_backward(ctypes.byref(cfg), plan.c, a, o, _stream(stream)),
           "moe_dispatch_backward")


def moe_route_encode(cfg, plan, route_enc, stream=None):
    e = _ptr(route_enc, torch.int32, cfg.R * cfg.S * cfg.K, "route_enc")
    _check(load().moe_route_encode(ctypes.byref(cfg), plan.c, e, _stream(stream)),
           "moe_route_encode")


def moe_dispatch_dedup(cfg, route_enc, x, xperm, stream=None):
    ntok = cfg.R * cfg.S
    args = (ctypes.byref(cfg),
            _ptr(route_enc, torch.int32, ntok * cfg.K, "route_enc"),
            _ptr(x, torch.bfloat16, ntok * cfg.H, "x"),
            _ptr(xperm, torch.bfloat16, ntok * cfg.K * cfg.H, "xperm"),
            _stream(stream))
    _check(load().moe_dispatch_dedup(*args), "moe_dispatch_dedup")


def moe_reduce_grad(cfg, plan, grad_home, grad_pref, stream=None):
    hh = cfg.H * cfg.Hp
    a = _ptr(grad_home, torch.float32, cfg.E * hh, "grad_home")
    b = _ptr(grad_pref, torch.float32, cfg.R * cfg.B * hh, "grad_pref") if cfg.B else None
    _check(load().moe_reduce_grad(ctypes.byref(cfg), plan.c, a, b, _stream(stream)),
           "moe_reduce_grad")


def make_router_cfg(score, renormalize, scale=1.0, logits_bf16=False, nseq=1):
    return moe_router_cfg(int(score), int(renormalize), float(scale), int(logits_bf16), int(nseq))


def moe_router_workspace_size(cfg, rcfg):
    out = ctypes.c_size_t()
    _check(load().moe_router_workspace_size(ctypes.byref(cfg), ctypes.byref(rcfg),
                                            ctypes.byref(out)), "moe_router_workspace_size")
    return int(out.value)


def _loss_args(cfg, rcfg, cu_tokens, counts, prob, loss, workspace, dev):
    n, m = rcfg.nseq, rcfg.nseq * cfg.E
    return (_arg(cu_tokens, torch.int32, n + 1, "cu_tokens", dev),
            _arg(counts, torch.int32, m, "counts", dev),
            _arg(prob, torch.float32, m, "prob", dev),
            _arg(loss, torch.float32, n, "loss", dev),
            _arg(workspace, torch.uint8, moe_router_workspace_size(cfg, rcfg), "workspace", dev))


def moe_router(cfg, rcfg, logits, bias, topk_ids, gates, cu_tokens=None, counts=None, prob=None,
               loss=None, workspace=None, stream=None):
    """Ids and gates; with counts, prob, loss and workspace the balance loss too."""
    dev = torch.cuda.current_device()
    T = cfg.R * cfg.S
    rest = (None,) * 5
    if loss is not None or counts is not None or prob is not None:
        rest = _loss_args(cfg, rcfg, cu_tokens, counts, prob, loss, workspace, dev)
    _check(load().moe_router(
        ctypes.byref(cfg), ctypes.byref(rcfg),
        _arg(logits, torch.bfloat16 if rcfg.logits_bf16 else torch.float32, T * cfg.E, "logits",
             dev),
        _arg(bias, torch.float32, cfg.E, "bias", dev),
        _arg(topk_ids, torch.int32, T * cfg.K, "topk_ids", dev),
        _arg(gates, torch.float32, T * cfg.K, "gates", dev),
        *rest, _on(stream, dev)), "moe_router")


def moe_balance_loss(cfg, rcfg, logits, topk_ids, cu_tokens, counts, prob, loss, workspace,
                     stream=None):
    dev = torch.cuda.current_device()
    T = cfg.R * cfg.S
    _check(load().moe_balance_loss(
        ctypes.byref(cfg), ctypes.byref(rcfg),
        _arg(logits, torch.bfloat16 if rcfg.logits_bf16 else torch.float32, T * cfg.E, "logits",
             dev),
        _arg(topk_ids, torch.int32, T * cfg.K, "topk_ids", dev),
        *_loss_args(cfg, rcfg, cu_tokens, counts, prob, loss, workspace, dev),
        _on(stream, dev)), "moe_balance_loss")


def moe_router_backward(cfg, rcfg, logits, topk_ids, dgates, cu_tokens, counts, dloss, dlogits,
                        stream=None):
    """dgates or dloss (with counts and cu_tokens) may be None."""
    dev = torch.cuda.current_device()
    T, n = cfg.R * cfg.S, rcfg.nseq
    dtype = torch.bfloat16 if rcfg.logits_bf16 else torch.float32
    _check(load().moe_router_backward(
        ctypes.byref(cfg), ctypes.byref(rcfg),
        _arg(logits, dtype, T * cfg.E, "logits", dev),
        _arg(topk_ids, torch.int32, T * cfg.K, "topk_ids", dev),
        _arg(dgates, torch.float32, T * cfg.K, "dgates", dev),
        _arg(cu_tokens, torch.int32, n + 1, "cu_tokens", dev),
        _arg(counts, torch.int32, n * cfg.E, "counts", dev),
        _arg(dloss, torch.float32, n, "dloss", dev),
        _arg(dlogits, dtype, T * cfg.E, "dlogits", dev), _on(stream, dev)), "moe_router_backward")


def _fits(rows, width, where):
    """Refuses what the library's int64 and int32 would cut to its low bits."""
    if not (-(1 << 63) <= rows < 1 << 63 and -(1 << 31) <= width < 1 << 31):
        raise MoeError(MOE_ELIMIT, where)


def _kept(rows, width, q, scale, what, dev):
    """Codes and scale bytes of `rows` rows of `width` values."""
    return (_arg(q, torch.uint8, rows * width, what + " codes", dev),
            _arg(scale, torch.uint8, rows * ((width + 31) // 32), what + " scales", dev))


def moe_q8_store(rows, width, src, q, scale, stream=None):
    """Codes q [rows, width] and scale bytes [rows, ceil(width / 32)] of bf16 rows."""
    _fits(rows, width, "moe_q8_store")
    dev = torch.cuda.current_device()
    _check(load().moe_q8_store(rows, width,
                               _arg(src, torch.bfloat16, rows * width, "src", dev),
                               *_kept(rows, width, q, scale, "q8", dev), _on(stream, dev)),
           "moe_q8_store")


def moe_q8_load(rows, width, q, scale, dst, stream=None):
    _fits(rows, width, "moe_q8_load")
    dev = torch.cuda.current_device()
    _check(load().moe_q8_load(rows, width, *_kept(rows, width, q, scale, "q8", dev),
                              _arg(dst, torch.bfloat16, rows * width, "dst", dev),
                              _on(stream, dev)), "moe_q8_load")


def moe_dispatch_q8(cfg, plan, xq, xscale, xperm, stream=None):
    dev = torch.cuda.current_device()
    ntok = cfg.R * cfg.S
    _arg(plan.route, torch.int32, ntok * cfg.K, "plan", dev)
    _check(load().moe_dispatch_q8(ctypes.byref(cfg), plan.c,
                                  *_kept(ntok, cfg.H, xq, xscale, "x", dev),
                                  _arg(xperm, torch.bfloat16, ntok * cfg.K * cfg.H, "xperm", dev),
                                  _on(stream, dev)), "moe_dispatch_q8")


def moe_grouped_gemm_swiglu_q8(cfg, xperm, w13_home, w13_pref, cu_seqlens, act, h13q, h13scale,
                               rank_begin, rank_end, workspace, stream=None):
    """cfg.Hp is the intermediate size H'; W13 rows are [H][2H'] (gate | up)."""
    dev = torch.cuda.current_device()
    rows = cfg.R * cfg.S * cfg.K
    hh = cfg.H * 2 * cfg.Hp
    bf = torch.bfloat16
    _check(load().moe_grouped_gemm_swiglu_q8(
        ctypes.byref(cfg), _arg(xperm, bf, rows * cfg.H, "xperm", dev),
        _arg(w13_home, bf, cfg.E * hh, "w13_home", dev),
        _arg(w13_pref, bf, cfg.R * cfg.B * hh, "w13_pref", dev) if cfg.B else None,
        _arg(cu_seqlens, torch.int32, cfg.R * (cfg.E + cfg.B + 1), "cu_seqlens", dev),
        _arg(act, bf, rows * cfg.Hp, "act", dev),
        *_kept(2 * rows, cfg.Hp, h13q, h13scale, "h13", dev), int(rank_begin), int(rank_end),
        _arg(workspace, torch.uint8, moe_gemm_workspace_size(cfg), "workspace", dev),
        _on(stream, dev)), "moe_grouped_gemm_swiglu_q8")


def moe_swiglu_backward_q8(cfg, h13q, h13scale, dact, dh13, act=None, stream=None):
    """dh13, and act again for the second projection's weight gradient if given."""
    dev = torch.cuda.current_device()
    rows = cfg.R * cfg.S * cfg.K
    bf = torch.bfloat16
    _check(load().moe_swiglu_backward_q8(
        ctypes.byref(cfg), *_kept(2 * rows, cfg.Hp, h13q, h13scale, "h13", dev),
        _arg(dact, bf, rows * cfg.Hp, "dact", dev),
        _arg(dh13, bf, rows * 2 * cfg.Hp, "dh13", dev),
        _arg(act, bf, rows * cfg.Hp, "act", dev), _on(stream, dev)), "moe_swiglu_backward_q8")


def moe_combine_backward_q8(cfg, plan, dout, yq, yscale, gates, dy, dgates, stream=None):
    dev = torch.cuda.current_device()
    ntok = cfg.R * cfg.S
    rows = ntok * cfg.K
    _arg(plan.route, torch.int32, rows, "plan", dev)
    _check(load().moe_combine_backward_q8(
        ctypes.byref(cfg), plan.c, _arg(dout, torch.bfloat16, ntok * cfg.Hp, "dout", dev),
        *_kept(rows, cfg.Hp, yq, yscale, "y", dev),
        _arg(gates, torch.float32, rows, "gates", dev),
        _arg(dy, torch.bfloat16, rows * cfg.Hp, "dy", dev),
        _arg(dgates, torch.float32, rows, "dgates", dev), _on(stream, dev)),
        "moe_combine_backward_q8")


def make_epilogue_cfg(act=ACT_NONE, p=0.0, f32=False):
    return moe_epilogue_cfg(int(act), float(p), int(f32))


def make_dropout_cfg(p=0.0, f32=False):
    return moe_dropout_cfg(float(p), int(f32))


def moe_epilogue_workspace_size(cfg, ecfg):
    out = ctypes.c_size_t()
    _check(load().moe_epilogue_workspace_size(ctypes.byref(cfg), ctypes.byref(ecfg),
                                              ctypes.byref(out)), "moe_epilogue_workspace_size")
    return int(out.value)


def _row_type(f32):
    return torch.float32 if f32 else torch.bfloat16


def _rng(rng, dev):
    """Seed and step of dropout: two int64 on the device."""
    return _arg(rng, torch.int64, 2, "rng", dev)


def _plan_or_none(cfg, plan, dev):
    if plan is None:
        return None
    _arg(plan.cu_seqlens, torch.int32, cfg.R * (cfg.E + cfg.B + 1), "plan", dev)
    if cfg.B:
        _arg(plan.slot_expert, torch.int32, cfg.R * cfg.B, "the plan's slots", dev)
    return plan.c


def moe_grouped_gemm_epilogue(cfg, ecfg, plan, xperm, w_home, w_pref, bias, residual, rng, y,
                              pre, rank_begin, rank_end, workspace, stream=None):
    """plan None: one matrix for all rows (cfg.R = cfg.E = 1); w_pref is then not read."""
    dev = torch.cuda.current_device()
    rows = cfg.R * cfg.S * cfg.K
    hh = cfg.H * cfg.Hp
    bf, out = torch.bfloat16, _row_type(ecfg.f32)
    slots = plan is not None and cfg.B
    _check(load().moe_grouped_gemm_epilogue(
        ctypes.byref(cfg), ctypes.byref(ecfg), _plan_or_none(cfg, plan, dev),
        _arg(xperm, bf, rows * cfg.H, "xperm", dev),
        _arg(w_home, bf, cfg.E * hh, "w_home", dev),
        _arg(w_pref, bf, cfg.R * cfg.B * hh, "w_pref", dev) if slots else None,
        _arg(bias, torch.float32, cfg.E * cfg.Hp, "bias", dev),
        _arg(residual, out, rows * cfg.Hp, "residual", dev), _rng(rng, dev),
        _arg(y, out, rows * cfg.Hp, "y", dev), _arg(pre, bf, rows * cfg.Hp, "pre", dev),
        int(rank_begin), int(rank_end),
        _arg(workspace, torch.uint8, moe_epilogue_workspace_size(cfg, ecfg), "workspace", dev),
        _on(stream, dev)), "moe_grouped_gemm_epilogue")


def moe_epilogue_backward(cfg, ecfg, plan, dy, pre, rng, dz, dbias, workspace=None, stream=None):
    """dz or dbias may be None; plan and workspace are needed for dbias only."""
    dev = torch.cuda.current_device()
    rows = cfg.R * cfg.S * cfg.K
    bf = torch.bfloat16
    need = moe_epilogue_workspace_size(cfg, ecfg) if dbias is not None else 0
    _check(load().moe_epilogue_backward(
        ctypes.byref(cfg), ctypes.byref(ecfg), _plan_or_none(cfg, plan, dev),
        _arg(dy, _row_type(ecfg.f32), rows * cfg.Hp, "dy", dev),
        _arg(pre, bf, rows * cfg.Hp, "pre", dev), _rng(rng, dev),
        _arg(dz, bf, rows * cfg.Hp, "dz", dev),
        _arg(dbias, torch.float32, cfg.E * cfg.Hp, "dbias", dev),
        _arg(workspace, torch.uint8, need, "workspace", dev), _on(stream, dev)),
        "moe_epilogue_backward")


def moe_dropout(dcfg, rows, width, src, residual, rng, dst, stream=None):
    """dst = residual + dropout(src); residual may be None."""
    _fits(rows, width, "moe_dropout")
    dev = torch.cuda.current_device()
    n, to = rows * width, _row_type(dcfg.f32)
    _check(load().moe_dropout(
        ctypes.byref(dcfg), rows, width, _arg(src, to, n, "src", dev),
        _arg(residual, to, n, "residual", dev), _rng(rng, dev), _arg(dst, to, n, "dst", dev),
        _on(stream, dev)), "moe_dropout")


def moe_combine_dropout(cfg, dcfg, plan, y, gates, residual, rng, out, stream=None):
    """residual may be None, rng with p = 0."""
    dev = torch.cuda.current_device()
    ntok = cfg.R * cfg.S
    to = _row_type(dcfg.f32)
    _arg(plan.route, torch.int32, ntok * cfg.K, "plan", dev)
    _check(load().moe_combine_dropout(
        ctypes.byref(cfg), ctypes.byref(dcfg), plan.c,
        _arg(y, torch.bfloat16, ntok * cfg.K * cfg.Hp, "y", dev),
        _arg(gates, torch.float32, ntok * cfg.K, "gates", dev),
        _arg(residual, to, ntok * cfg.Hp, "residual", dev), _rng(rng, dev),
        _arg(out, to, ntok * cfg.Hp, "out", dev), _on(stream, dev)), "moe_combine_dropout")


def moe_combine_dropout_backward(cfg, dcfg, plan, dout, y, gates, rng, dy, dgates, stream=None):
    dev = torch.cuda.current_device()
    ntok = cfg.R * cfg.S
    rows = ntok * cfg.K
    bf = torch.bfloat16
    _arg(plan.route, torch.int32, rows, "plan", dev)
    _check(load().moe_combine_dropout_backward(
        ctypes.byref(cfg), ctypes.byref(dcfg), plan.c,
        _arg(dout, _row_type(dcfg.f32), ntok * cfg.Hp, "dout", dev),
        _arg(y, bf, rows * cfg.Hp, "y", dev), _arg(gates, torch.float32, rows, "gates", dev),
        _rng(rng, dev), _arg(dy, bf, rows * cfg.Hp, "dy", dev),
        _arg(dgates, torch.float32, rows, "dgates", dev), _on(stream, dev)),
        "moe_combine_dropout_backward")
