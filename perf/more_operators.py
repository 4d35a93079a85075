"""Cases, plain forms and float64 values of the product with an epilogue and of dropout.

The operators, each as a user's program calls it:

* ``product``  -- rows times weights with bias, activation, dropout and residual in the
  epilogue: one matrix (a shared expert, the router's projection) or one per expert;
* ``backward`` -- the gradient of that epilogue: of the product itself, and of the bias of
  every expert;
* ``dropout``  -- dropout with a residual; the generator counts, so no mask is kept;
* ``combine``  -- the gate-weighted sum of the expert outputs with dropout and residual, and
  its backward pass, which draws the same numbers again.

``own`` chooses between the plain form (elementary torch operations) and the package's calls.
"""
import math

import torch

own = False

NONE, RELU, GELU, GELU_TANH, SILU, RELU2 = range(6)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _product(name, S, E, K, H, Hp, act, bias=True, residual=False, f32=False, p=0.0, pre=False):
    """S tokens of K routes to E experts; E = 1: one matrix for all rows."""
    return {"name": name, "op": "product", "S": S, "E": E, "K": K, "H": H, "Hp": Hp, "act": act,
            "bias": bias, "residual": residual, "f32": f32, "p": p, "pre": pre}


def _backward(name, S, E, K, Hp, act, f32, p):
    return {"name": name, "op": "backward", "S": S, "E": E, "K": K, "Hp": Hp, "act": act, "f32": f32, "p": p}


def _combine(name, R, S, E, K, Hp, f32, p):
    return {"name": name, "op": "combine", "R": R, "S": S, "E": E, "K": K, "Hp": Hp, "f32": f32, "p": p}


def listed():
    return [
        # first projection of a shared expert for the one token being decoded: all latency
        _product("matrix 1 token 7168x2048", 1, 1, 1, 7168, 2048, GELU),
        # router logits of a serving batch, in fp32 as the router takes them
        _product("router 2048 tokens 7168x384", 2048, 1, 1, 7168, 384, NONE, f32=True),
        # second projection of a shared expert in training: dropout, then the residual stream
        _product("matrix 8192 rows 2048x7168", 8192, 1, 1, 2048, 7168, NONE, residual=True, p=0.1),
        # one token per rank being decoded: every route meets its own expert
        _product("experts 8 tokens E384", 8, 384, 8, 7168, 2048, GELU_TANH),
        # one rank of the training step: 65,536 rows over its 48 experts, products kept for the backward
        _product("experts 65536 rows E48", 8192, 48, 8, 7168, 2048, GELU, pre=True),
        # odd sizes: 4,100 rows of 1,000 onto 520 columns with everything in the epilogue
        _product("experts 4100 rows E8 1000x520", 1025, 8, 4, 1000, 520, RELU2, residual=True, f32=True, p=0.25,
                 pre=True),
        # the epilogue's backward over all ranks of the training step
        _backward("backward 524288 rows E384", 65536, 384, 8, 2048, GELU, False, 0.1),
        # a small layer with an fp32 residual stream and an odd width
        _backward("backward 4100 rows E8 520", 1025, 8, 4, 520, SILU, True, 0.0),
        # a few rows of the residual stream: latency
        {"name": "dropout 8x7168", "op": "dropout", "rows": 8, "width": 7168, "residual": True, "f32": False, "p": 0.1},
        # the step's residual stream
        {"name": "dropout 65536x7168", "op": "dropout", "rows": 65536, "width": 7168, "residual": True, "f32": False,
         "p": 0.1},
        # forward and backward of the step's combine
        _combine("combine 8x8192 H7168", 8, 8192, 384, 8, 7168, False, 0.1),
        # a small layer, odd token count and width, fp32 residual stream
        _combine("combine 8x125 H1000", 8, 125, 64, 4, 1000, True, 0.25),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "product", "backward", "dropout", "combine"])
    f32, p = rng.random() < 0.4, rng.choice([0.0, 0.1, 0.25, 0.5])
    act = rng.randint(NONE, RELU2)
    if op == "product":
        wide = 8 * _log(rng, 4, 896)
        case = _product("", 1, 1, 1, wide, 8 * _log(rng, 1, 896 if wide <= 2048 else 256), act, rng.random() < 0.8,
                        rng.random() < 0.4, f32, p, rng.random() < 0.4)
        del case["name"]
        if rng.random() < 0.5:
            return {**case, "S": _log(rng, 1, 16384)}
        E = _log(rng, 2, 96)
        K = rng.choice([k for k in (1, 2, 4, 8) if k <= E])
        return {**case, "E": E, "K": K, "S": max(1, _log(rng, 1, 16384) // K)}
    if op == "backward":
        E = _log(rng, 1, 384)
        K = rng.choice([k for k in (1, 2, 4, 8) if k <= E])
        return {"op": op, "S": max(1, _log(rng, 1, 131072) // K), "E": E, "K": K, "Hp": 8 * _log(rng, 1, 512),
                "act": act, "f32": f32, "p": p}
    if op == "dropout":
        return {"op": op, "rows": _log(rng, 1, 32768), "width": 8 * _log(rng, 1, 1024), "residual": rng.random() < 0.6,
                "f32": f32, "p": rng.choice([0.1, 0.25, 0.5])}
    R, n, K = rng.choice([1, 2, 4, 8]), rng.randint(2, 24), rng.randint(1, 8)
    return {"op": op, "R": R, "S": _log(rng, 1, 16384 // R), "E": R * n, "K": min(K, R * n), "Hp": 8 * _log(rng, 4, 512),
            "f32": f32, "p": p}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, f32, *shape):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x if f32 else x.to(torch.bfloat16)


def _cuts(gen, tokens, E, K):
    """Where each expert's rows begin among tokens * K rows; some experts are far more popular."""
    if E == 1:
        return torch.tensor([0, tokens * K], dtype=torch.int32, device="cuda")
    z = torch.randn((tokens, E), generator=gen, device="cuda")
    z += torch.randn((E,), generator=gen, device="cuda")
    n = torch.bincount(z.topk(K, dim=1).indices.reshape(-1), minlength=E)
    return torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1) + 29)
    st = {"case": case, "kept": {}}
    # the generator's seed and the program's step, on the device as a captured step reads them
    st["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda", dtype=torch.int64)
    op = case["op"]
    if op == "dropout":
        st["src"] = _randn(gen, case["f32"], case["rows"], case["width"])
        st["residual"] = _randn(gen, case["f32"], case["rows"], case["width"]) if case["residual"] else None
        return st
    if op == "combine":
        T, K, Hp = case["R"] * case["S"], case["K"], case["Hp"]
        st["route"] = torch.randperm(T * K, generator=gen, device="cuda").to(torch.int32)
        st["y"] = _randn(gen, False, T * K, Hp)
        st["residual"], st["dout"] = _randn(gen, case["f32"], T, Hp), _randn(gen, case["f32"], T, Hp)
        g = torch.rand((T, K), generator=gen, device="cuda") + 0.01
        st["gates"] = g / g.sum(1, keepdim=True)
        return st
    rows, E, Hp = case["S"] * case["K"], case["E"], case["Hp"]
    st["cu_seqlens"] = _cuts(gen, case["S"], E, case["K"])
    st["cuts"] = st["cu_seqlens"].tolist()
    if op == "backward":
        st["dy"], st["pre"] = _randn(gen, case["f32"], rows, Hp), _randn(gen, False, rows, Hp)
        return st
    H = case["H"]
    st["x"] = _randn(gen, False, rows, H)
    st["w"] = torch.empty((E, H, Hp), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        st["w"][e] = torch.randn((H, Hp), generator=gen, device="cuda") / math.sqrt(H)
    st["bias"] = 0.5 * _randn(gen, True, E, Hp) if case["bias"] else None
    st["residual"] = _randn(gen, case["f32"], rows, Hp) if case["residual"] else None
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _keep(rng, p, rows, width):
    """Which values stay: 16 random bits each, eight from one Philox4x32-10 block of the counter
    (block index, step) under the seed, against p in steps of 2^-16; and the factor on them."""
    cut = int(p * 65536 + 0.5)
    word = 0xFFFFFFFF
    at = torch.arange(rows * width // 8, dtype=torch.int64, device=rng.device)
    seed, step = rng[0], rng[1]
    a, b = at & word, at >> 32
    c, d = (step & word).expand_as(at), ((step >> 32) & word).expand_as(at)
    k0, k1 = seed & word, (seed >> 32) & word
    for _ in range(10):
        x, z = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((z >> 32) & word) ^ b ^ k0, z & word, ((x >> 32) & word) ^ d ^ k1, x & word
        k0, k1 = (k0 + 0x9E3779B9) & word, (k1 + 0xBB67AE85) & word
    halves = [h for v in (a, b, c, d) for h in (v & 0xFFFF, v >> 16)]
    bits = torch.stack(halves, 1).to(torch.int32).view(rows, width)
    return bits >= cut, 65536.0 / (65536 - cut) if cut < 65536 else 0.0


def _drop(st, v):
    """v with some of its values zero and the others scaled."""
    p = st["case"]["p"]
    if p == 0.0:
        return v
    keep, scale = _keep(st["rng"], p, *v.shape)
    return torch.where(keep, v * scale, torch.zeros_like(v))


def _act(z, act):
    if act == RELU:
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == RELU2:
        return torch.where(z > 0, z * z, torch.zeros_like(z))
    if act == GELU:
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if act == GELU_TANH:
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == SILU:
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == RELU:
        return (z > 0).to(z.dtype)
    if act == RELU2:
        return torch.where(z > 0, 2.0 * z, torch.zeros_like(z))
    if act == GELU:
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == GELU_TANH:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1.0 - s) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == SILU:
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _plain(st):
    c = st["case"]
    to = torch.float32 if c["f32"] else torch.bfloat16
    if c["op"] == "dropout":
        v = _drop(st, st["src"].float())
        return {"dst": (v if st["residual"] is None else v + st["residual"].float()).to(to)}
    if c["op"] == "combine":
        T, K, Hp = c["R"] * c["S"], c["K"], c["Hp"]
        at = st["route"].long()
        y = st["y"][at].float().view(T, K, Hp)
        g = st["gates"].view(T, K, 1)
        out = (_drop(st, (g * y).sum(1)) + st["residual"].float()).to(to)
        d = _drop(st, st["dout"].float()).view(T, 1, Hp)
        dgates = (d * y).sum(2)
        dy = torch.empty_like(st["y"])
        dy[at] = (g * d).to(torch.bfloat16).view(T * K, Hp)
        return {"out": out, "dy": dy, "dgates": dgates}
    cuts = st["cuts"]
    if c["op"] == "backward":
        v = _drop(st, st["dy"].float()) * _act_slope(st["pre"].float(), c["act"])
        dbias = torch.stack([v[lo:hi].double().sum(0).float() for lo, hi in zip(cuts, cuts[1:])])
        return {"dz": v.to(torch.bfloat16), "dbias": dbias}
    z = torch.empty((cuts[-1], c["Hp"]), dtype=torch.float32, device=st["x"].device)
    for e in range(c["E"]):
        lo, hi = cuts[e], cuts[e + 1]
        if lo < hi:
            z[lo:hi] = st["x"][lo:hi].float() @ st["w"][e].float()
            if c["bias"]:
                z[lo:hi] += st["bias"][e]
    v = _drop(st, _act(z, c["act"]))
    if c["residual"]:
        v = v + st["residual"].float()
    out = {"y": v.to(to)}
    if c["pre"]:
        out["pre"] = z.to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _kept(st, mx):
    """Configurations, plan and buffers that a program makes once and keeps."""
    k, c = st["kept"], st["case"]
    if k:
        return k
    to = torch.float32 if c["f32"] else torch.bfloat16
    if c["op"] == "dropout":
        k["dc"] = mx.make_dropout_cfg(c["p"], c["f32"])
        k["dst"] = _empty(c["rows"], c["width"], dtype=to)
    elif c["op"] == "combine":
        k["dc"] = mx.make_dropout_cfg(c["p"], c["f32"])
        k["cfg"] = mx.make_cfg(c["R"], c["S"], c["E"], c["K"], 8, c["Hp"], 0, mx.MODE_INFER)
        k["plan"] = mx.Plan(k["cfg"])
        k["plan"].route.copy_(st["route"])
        k["out"] = torch.empty_like(st["residual"])
        k["dy"], k["dgates"] = torch.empty_like(st["y"]), torch.empty_like(st["gates"])
    else:
        rows, E, Hp = c["S"] * c["K"], c["E"], c["Hp"]
        k["cfg"] = mx.make_cfg(1, c["S"], E, c["K"], c.get("H", 8), Hp, 0, mx.MODE_INFER)
        k["ec"] = mx.make_epilogue_cfg(c["act"], c["p"], c["f32"])
        k["plan"] = None                                  # one matrix: every row is its own
        if E > 1:
            k["plan"] = mx.Plan(k["cfg"])
            k["plan"].cu_seqlens.copy_(st["cu_seqlens"])
        k["ws"] = _empty(mx.moe_epilogue_workspace_size(k["cfg"], k["ec"]), dtype=torch.uint8)
        if c["op"] == "backward":
            k["dz"], k["dbias"] = torch.empty_like(st["pre"]), _empty(E, Hp)
        else:
            k["y"] = _empty(rows, Hp, dtype=to)
            k["pre"] = _empty(rows, Hp, dtype=torch.bfloat16) if c["pre"] else None
    return k


def _own(st):
    import moe_expert_load_amd as mx
    c, k = st["case"], _kept(st, mx)
    rng = st["rng"] if c["p"] > 0.0 else None
    if c["op"] == "dropout":
        mx.moe_dropout(k["dc"], c["rows"], c["width"], st["src"], st["residual"], rng, k["dst"])
        return {"dst": k["dst"]}
    if c["op"] == "combine":
        mx.moe_combine_dropout(k["cfg"], k["dc"], k["plan"], st["y"], st["gates"], st["residual"], rng, k["out"])
        mx.moe_combine_dropout_backward(k["cfg"], k["dc"], k["plan"], st["dout"], st["y"], st["gates"], rng, k["dy"],
                                        k["dgates"])
        return {"out": k["out"], "dy": k["dy"], "dgates": k["dgates"]}
    if c["op"] == "backward":
        mx.moe_epilogue_backward(k["cfg"], k["ec"], k["plan"], st["dy"], st["pre"], rng, k["dz"], k["dbias"], k["ws"])
        return {"dz": k["dz"], "dbias": k["dbias"]}
    mx.moe_grouped_gemm_epilogue(k["cfg"], k["ec"], k["plan"], st["x"], st["w"], None, st["bias"], st["residual"], rng,
                                 k["y"], k["pre"], 0, 1, k["ws"])
    return {"y": k["y"], "pre": k["pre"]} if c["pre"] else {"y": k["y"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    wide = 4 if case["f32"] else 2
    if case["op"] == "dropout":
        n = case["rows"] * case["width"]
        return {"bytes": n * wide * (3 if case["residual"] else 2), "flops": 2 * n}
    if case["op"] == "combine":
        T, K, Hp = case["R"] * case["S"], case["K"], case["Hp"]
        # y, gates, route, residual and dout in; out, dy and dgates out
        return {"bytes": 2 * 2 * T * K * Hp + 3 * wide * T * Hp + 12 * T * K, "flops": 5 * T * K * Hp}
    rows, E, Hp = case["S"] * case["K"], case["E"], case["Hp"]
    if case["op"] == "backward":
        return {"bytes": rows * Hp * (wide + 4) + 4 * E * Hp, "flops": 4 * rows * Hp}
    H = case["H"]
    met = E if E == 1 else E * (1.0 - (1.0 - case["K"] / E) ** case["S"])     # experts that get a row
    moved = 2 * rows * H + met * (2 * H * Hp + (4 * Hp if case["bias"] else 0))
    moved += rows * Hp * (wide * (2 if case["residual"] else 1) + (2 if case["pre"] else 0))
    return {"bytes": int(moved), "flops": 2 * rows * H * Hp}


# ---------------------------------------------------------------------------
# the same values in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _wide_product(m, v):
    """High and low word of the 64-bit product of the constant m and the words v, from 16-bit parts."""
    m0, m1, v0, v1 = m % 65536, m // 65536, v % 65536, v // 65536
    low, mid = m0 * v0, m0 * v1 + m1 * v0                  # below 2^32 and 2^33
    part = low // 65536 + mid % 65536
    return m1 * v1 + mid // 65536 + part // 65536, part % 65536 * 65536 + low % 65536


def _factor(st, rows, width):
    """What dropout multiplies each value with: 0, or one over the share that stays."""
    cut = math.floor(st["case"]["p"] * 65536 + 0.5)
    if cut == 0:
        return 1.0
    two32 = 1 << 32
    seed, step = [int(v) for v in st["rng"].tolist()]
    out = torch.empty((rows * width // 8, 8), dtype=torch.float64, device="cuda")
    piece = 1 << 22
    for lo in range(0, out.shape[0], piece):
        n = torch.arange(lo, min(lo + piece, out.shape[0]), device="cuda")
        ctr = [n % two32, n // two32, torch.full_like(n, step % two32), torch.full_like(n, step // two32)]
        key = [seed % two32, seed // two32]
        for r in range(10):
            h0, l0 = _wide_product(3528531795, ctr[0])
            h1, l1 = _wide_product(3449720151, ctr[2])
            ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
            key = [(key[0] + 2654435769) % two32, (key[1] + 3144134277) % two32]
        for i in range(8):
            bits = ctr[i // 2] // 65536 if i % 2 else ctr[i // 2] % 65536
            out[lo:lo + piece, i] = (bits >= cut).double() * (65536.0 / max(1, 65536 - cut))
    return out.view(rows, width)


def _exact_act(z, act):
    """The activation and its slope."""
    if act == NONE:
        return z, torch.ones_like(z)
    if act in (RELU, RELU2):
        n = z.clamp(min=0.0)
        return (n, (z > 0).double()) if act == RELU else (n * n, 2 * n)
    if act == GELU:
        below = torch.special.ndtr(z)
        return z * below, below + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == SILU:
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    r = math.sqrt(8 / math.pi)
    u = r * z + r * 0.044715 * z ** 3
    s = torch.sigmoid(u)
    return z * s, s + z * s * torch.sigmoid(-u) * (r + 3 * r * 0.044715 * z ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "dropout":
        v = st["src"].double() * _factor(st, case["rows"], case["width"])
        return {"dst": v + st["residual"].double() if case["residual"] else v}
    if case["op"] == "combine":
        T, K, Hp = case["R"] * case["S"], case["K"], case["Hp"]
        f = _factor(st, T, Hp)
        back = st["route"].long()
        gates, d = st["gates"].double(), st["dout"].double() * f
        out = torch.zeros((T, Hp), dtype=torch.float64, device="cuda")
        dy = torch.empty((T * K, Hp), dtype=torch.float64, device="cuda")
        dgates = torch.empty_like(gates)
        for k in range(K):
            rows = back.view(T, K)[:, k]
            y = st["y"].index_select(0, rows).double()
            out += gates[:, k:k + 1] * y
            dgates[:, k] = (d * y).sum(1)
            dy.index_copy_(0, rows, gates[:, k:k + 1] * d)
        return {"out": out * f + st["residual"].double(), "dy": dy, "dgates": dgates}
    rows, E, Hp, cuts = case["S"] * case["K"], case["E"], case["Hp"], st["cuts"]
    f = _factor(st, rows, Hp)
    if case["op"] == "backward":
        dz = st["dy"].double() * f * _exact_act(st["pre"].double(), case["act"])[1]
        dbias = torch.zeros((E, Hp), dtype=torch.float64, device="cuda")
        owner = torch.repeat_interleave(torch.arange(E, device="cuda"), st["cu_seqlens"].long().diff())
        return {"dz": dz, "dbias": dbias.index_add_(0, owner, dz)}
    parts = []
    for e in range(E):
        if cuts[e] < cuts[e + 1]:
            z = st["x"][cuts[e]:cuts[e + 1]].double() @ st["w"][e].double()
            parts.append(z + st["bias"][e].double() if case["bias"] else z)
    z = torch.cat(parts, 0)
    y = _exact_act(z, case["act"])[0] * f
    if case["residual"]:
        y = y + st["residual"].double()
    return {"y": y, "pre": z} if case["pre"] else {"y": y}
