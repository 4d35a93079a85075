"""Oracle for the product's epilogue and for dropout (test infrastructure only).

``z = product + bias``, ``y = residual + dropout(act(z))`` and its gradients; the
gate-weighted combine with dropout and residual and its gradients; all in float64 from the
definitions in ``include/moonep.h``.  The generator is Philox4x32-10 (Salmon, Moraes, Dror
and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) on Python-sized words.

Pinned by tests/test_oracle_epilogue.py: the published known answers of the generator, the
share of dropped values, closed forms of the activations, and differences for every slope.
"""
import numpy as np
from scipy.special import expit, ndtr

NONE, RELU, GELU, GELU_TANH, SILU, RELU2 = range(6)
WORD = np.uint64(0xFFFFFFFF)


def philox(counter, key):
    """Four output words of four counter words (arrays or numbers) under two key words."""
    a, b, c, d = (np.asarray(v, np.uint64) for v in counter)
    k0, k1 = (int(v) for v in key)
    s = np.uint64(32)
    for _ in range(10):
        x, z = np.uint64(0xD2511F53) * a, np.uint64(0xCD9E8D57) * c     # below 2^64
        a, b, c, d = (z >> s) ^ b ^ np.uint64(k0), z & WORD, (x >> s) ^ d ^ np.uint64(k1), x & WORD
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    return a, b, c, d


def steps(p):
    """Dropout probability in steps of 2^-16; p as the float32 that the entry points take."""
    return int(np.floor(65536 * float(np.float32(p)) + 0.5))


def numbers(rng, index):
    """The 16-bit numbers of the values at these flat indices; rng = (seed, step)."""
    index = np.asarray(index, np.uint64)
    block, i = index // np.uint64(8), (index % np.uint64(8)).astype(np.int64)
    seed, step = (int(v) % 2 ** 64 for v in rng)
    n = np.broadcast_to
    words = np.stack(philox((block & WORD, block >> np.uint64(32), n(np.uint64(step % 2 ** 32), block.shape),
                             n(np.uint64(step >> 32), block.shape)), (seed % 2 ** 32, seed >> 32)))
    w = np.take_along_axis(words, (i // 2)[None], 0)[0]
    return np.where(i % 2 == 1, w >> np.uint64(16), w & np.uint64(0xFFFF)).astype(np.int64)


def factor(p, rng, index):
    """What dropout multiplies the values at these flat indices with."""
    d = steps(p)
    if d == 0:
        return np.ones(np.shape(index))
    keep = numbers(rng, index) >= d
    return keep * (65536.0 / (65536 - d) if d < 65536 else 0.0)


def row_factor(p, rng, rows, width):
    """factor for whole rows (row numbers) of a tensor of this width."""
    return factor(p, rng, np.asarray(rows, np.int64)[:, None] * width + np.arange(width)[None])


def _tanh_parts(z):
    u2 = 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    return expit(u2), 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * z ** 2)


def act(z, kind):
    if kind == RELU:
        return np.maximum(z, 0)
    if kind == RELU2:
        return np.maximum(z, 0) ** 2
    if kind == GELU:
        return z * ndtr(z)
    if kind == GELU_TANH:
        return z * _tanh_parts(z)[0]
    if kind == SILU:
        return z * expit(z)
    return z


def slope_terms(z, kind):
    """Two terms whose sum is the slope of act."""
    o = np.zeros_like(z)
    if kind == RELU:
        return (z > 0) * 1.0, o
    if kind == RELU2:
        return 2 * np.maximum(z, 0), o
    if kind == GELU:
        return ndtr(z), z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if kind == GELU_TANH:
        s, du = _tanh_parts(z)
        return s, z * s * (1 - s) * du
    if kind == SILU:
        return expit(z), z * expit(z) * expit(-z)
    return o + 1, o


def slope(z, kind):
    a, b = slope_terms(z, kind)
    return a + b


def segment_experts(cu_seqlens, slot_expert, E, SK):
    """Expert of every row of every rank's buffer; -1 where no segment is, -2 where a slot
    names no expert."""
    R = cu_seqlens.shape[0]
    out = np.full(R * SK, -1, np.int64)
    for r in range(R):
        for j in range(cu_seqlens.shape[1] - 1):
            e = j if j < E else int(slot_expert[r, j - E])
            out[r * SK + cu_seqlens[r, j]:r * SK + cu_seqlens[r, j + 1]] = e if 0 <= e < E else -2
    return out


def forward(z, kind, p, rng, residual=None, rows=None):
    """y of the products-plus-bias z of these rows (all rows if None)."""
    rows = np.arange(z.shape[0]) if rows is None else rows
    y = act(z, kind) * row_factor(p, rng, rows, z.shape[1])
    return y if residual is None else y + residual


def backward(dy, pre, kind, p, rng, expert=None, E=1):
    """(dz, dbias) before rounding; expert of every row, negative ones own no bias."""
    dz = dy * row_factor(p, rng, np.arange(dy.shape[0]), dy.shape[1]) * slope(pre, kind)
    expert = np.zeros(dy.shape[0], np.int64) if expert is None else expert
    dbias = np.stack([dz[expert == e].sum(0) for e in range(E)])
    return dz, dbias


def combine(y, gates, route, p, rng, residual=None):
    """residual + dropout(sum_k gates * y[route]); y, route over R*S*K rows, -1: no route."""
    T, K = gates.shape
    route = route.reshape(T, K)
    rows = np.where((route >= 0)[..., None], y[np.maximum(route, 0)], 0.0)
    out = (gates[..., None] * rows).sum(1) * row_factor(p, rng, np.arange(T), y.shape[1])
    return out if residual is None else out + residual


def combine_backward(dout, y, gates, route, p, rng):
    """(dy rows in route order [T, K, width], dgates)."""
    T, K = gates.shape
    route = route.reshape(T, K)
    d = dout * row_factor(p, rng, np.arange(T), y.shape[1])
    rows = np.where((route >= 0)[..., None], y[np.maximum(route, 0)], 0.0)
    return gates[..., None] * d[:, None], (d[:, None] * rows).sum(2)
