"""Oracle for the router, its balance loss and their gradients (test infrastructure only).

[TSR] §6.1: a token's router weights pick its K experts and sum their outputs.
The pages name neither the score function nor an auxiliary loss; the readings
taken here are the two scores in use (softmax over the experts, or a sigmoid
per expert, with an optional bias that takes part in the choice only) and the
per-sequence loss sum_e f_e P_e with f_e = E c_e / (K L) and P_e the mean
share of expert e over the sequence's L tokens.

Everything is float64.  Pinned by tests/test_oracle_router.py: closed forms,
ties and masks by hand, and the gradients against central differences.
"""
import numpy as np

SOFTMAX, SIGMOID = 0, 1


def scores(z, score):
    """(s, shares) of logits z [T, E]: the router scores and what the loss averages."""
    z = np.asarray(z, np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        m = np.max(z, axis=1, keepdims=True)
        empty = m == -np.inf
        e = np.where(empty, 0.0, np.exp(z - np.where(empty, 0.0, m)))
        total = e.sum(axis=1, keepdims=True)
        soft = np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))
        if score == SOFTMAX:
            return soft, soft
        s = 1.0 / (1.0 + np.exp(-z))
        # log s = -log(1 + e^-z) keeps ratios of scores that underflow
        ls = -np.logaddexp(0.0, -z)
        m = np.max(ls, axis=1, keepdims=True)
        e = np.where(m == -np.inf, 0.0, np.exp(ls - np.where(m == -np.inf, 0.0, m)))
        total = e.sum(axis=1, keepdims=True)
        return s, np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def complement(z):
    """1 - sigmoid(z), not as a difference: from z = 37 on the sigmoid is 1 in float64."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(np.asarray(z, np.float64)))


def choose(z, bias, K, score):
    """The K largest of z, or of s + bias; equal ones in ascending id.  Sums that are NaN come
    after numbers, masked experts (-inf) after those, NaN logits last, each in ascending id."""
    z = np.asarray(z, np.float64)
    key = z
    if bias is not None:
        key = scores(z, score)[0] + np.asarray(bias, np.float64)
    kind = np.where(np.isnan(z), 3, np.where(z == -np.inf, 2, np.where(np.isnan(key), 1, 0)))
    order = np.lexsort((np.broadcast_to(np.arange(z.shape[1]), z.shape),
                        np.where(kind == 0, -key, 0.0), kind), axis=1)
    return order[:, :K].astype(np.int32)


def gate_shares(z, ids, score, renorm):
    """gates / scale of the chosen experts."""
    z = np.asarray(z, np.float64)
    zk = np.take_along_axis(z, ids, 1)
    if renorm:
        return scores(zk, score)[1]                    # shares among the chosen alone
    return np.take_along_axis(scores(z, score)[0], ids, 1)


def balance(z, ids, cu, score):
    """(counts, prob, loss) of every sequence cu[q] .. cu[q + 1]."""
    E, K = z.shape[1], ids.shape[1]
    share = scores(z, score)[1]
    n = len(cu) - 1
    counts = np.zeros((n, E), np.int64)
    prob, loss = np.zeros((n, E)), np.zeros(n)
    for q in range(n):
        rows = slice(cu[q], cu[q + 1])
        L = cu[q + 1] - cu[q]
        if L == 0:
            continue
        got = ids[rows].reshape(-1)
        got = got[(got >= 0) & (got < E)]
        counts[q] = np.bincount(got, minlength=E)
        prob[q] = share[rows].sum(0) / L
        loss[q] = (E * counts[q] / (K * L) * prob[q]).sum()
    return counts, prob, loss


def backward(z, ids, score, renorm, scale, dgates=None, cu=None, counts=None, dloss=None):
    """(dlogits, size): the gradient, and the sum of the magnitudes it is made of."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    K = ids.shape[1] if ids is not None else 0
    s, p = scores(z, score)
    dz, size = np.zeros_like(z), np.zeros_like(z)
    if dloss is not None:
        for q in range(len(cu) - 1):
            L = cu[q + 1] - cu[q]
            if L == 0:
                continue
            r = slice(cu[q], cu[q + 1])
            u = dloss[q] * E * counts[q] / (K * L * float(L))
            mean = p[r] @ u
            f = p[r] * (complement(z[r]) if score == SIGMOID else 1.0)
            dz[r] += f * (u - mean[:, None])
            size[r] += f * (np.abs(u) + (p[r] @ np.abs(u))[:, None])
    if dgates is not None:
        dg = scale * np.asarray(dgates, np.float64)
        ok = (ids >= 0) & (ids < E)
        at = np.where(ok, ids, 0)
        zk = np.where(ok, np.take_along_axis(z, at, 1), -np.inf)
        dg = np.where(ok, dg, 0.0)
        t = np.broadcast_to(np.arange(T)[:, None], ids.shape)
        if renorm:
            w = scores(zk, score)[1]
            d = w * (dg - (dg * w).sum(1, keepdims=True))
            a = w * (np.abs(dg) + (np.abs(dg) * w).sum(1, keepdims=True))
            if score == SIGMOID:
                co = complement(zk)
                d, a = d * co, a * co
            np.add.at(dz, (t, at), np.where(ok, d, 0.0))
            np.add.at(size, (t, at), np.where(ok, a, 0.0))
        else:
            full, mag = np.zeros_like(z), np.zeros_like(z)
            np.add.at(full, (t, at), dg)
            np.add.at(mag, (t, at), np.abs(dg))
            if score == SOFTMAX:
                dz += s * (full - (full * s).sum(1, keepdims=True))
                size += s * (mag + (mag * s).sum(1, keepdims=True))
            else:
                co = complement(z)
                dz += full * s * co
                size += mag * s * co
    return dz, size
