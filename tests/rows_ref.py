"""Definitions of the row operators in 64 bits (numpy), and the bounds on a
32-bit computation's error that the GPU tests hold the kernels to.

Bounds are the standard ones: a sum of n terms held in 32 bits is off by at
most n * 2^-24 times the sum of the terms' magnitudes, whatever its order; a
result rounded to a type of unit roundoff u by u times its magnitude, or half
the type's smallest number."""
import numpy as np
import torch

U32 = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound):
    """got is finite where want is and within bound of it there, and equal (NaN included) elsewhere."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    off = np.abs(got[fine] - want[fine]) - np.broadcast_to(bound, want.shape)[fine]
    assert off.size == 0 or off.max() <= 0, "off by %g more than the bound" % off.max()


def rounded(dtype, size):
    """The last rounding's part of a bound."""
    return 1.01 * UNIT[dtype] * size + TINY[dtype]


# ---- routing ---------------------------------------------------------------------------------------------------

def choose(keys, k):
    """The k best columns of each row: larger first, NaN above all, ties to the lower column, -inf never (-1)."""
    rank = np.where(np.isnan(keys), np.inf, keys)
    ids = np.empty((len(keys), k), dtype=np.int64)
    for t in range(len(keys)):
        order = sorted(range(keys.shape[1]), key=lambda e: (not np.isnan(keys[t, e]), -rank[t, e], e))[:k]
        ids[t] = [e if not (rank[t, e] == -np.inf) else -1 for e in order]
    return ids


def scores(l, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-l))
    with np.errstate(invalid="ignore"):
        e = np.exp(l - l.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)


def log_scores(l, score):
    """Logarithms of the scores up to a summand of the row (for ratios of scores that vanish)."""
    if score == "sigmoid":
        return -np.logaddexp(0, -l)
    return l


def weights_of(l, ids, score, renormalize, scale):
    """Weights of the chosen experts, differentiable in l (ids are held fixed)."""
    some = ids >= 0
    at = np.where(some, ids, 0)
    if renormalize:
        x = np.where(some, np.take_along_axis(log_scores(l, score), at, 1), -np.inf)
        high = x.max(1, keepdims=True)
        with np.errstate(invalid="ignore"):
            e = np.where(some, np.exp(x - np.where(high == -np.inf, 0, high)), 0)
            total = e.sum(1, keepdims=True)
            return scale * e / np.where(total == 0, 1, total)
    with np.errstate(invalid="ignore"):
        return scale * np.where(some, np.take_along_axis(scores(l, score), at, 1), 0)


def logits_gradient(l, ids, g, score, renormalize, scale):
    """Through the Jacobians of the weights and of the scores; also the magnitudes of what is added up."""
    some = ids >= 0
    at = np.where(some, ids, 0)
    h = np.where(some, scale * g, 0)
    s = scores(l, score)
    u = weights_of(l, ids, score, renormalize, 1.0)
    out, size = np.zeros_like(l), np.zeros_like(l)
    dot = (u * h).sum(1, keepdims=True)
    mag = (u * np.abs(h)).sum(1, keepdims=True)
    # 1 - sigmoid(x) = sigmoid(-x), which does not cancel
    slope = np.take_along_axis(scores(-l, score), at, 1) if score == "sigmoid" else np.ones_like(u)
    for j in range(ids.shape[1]):
        rows = np.flatnonzero(some[:, j])
        e = ids[rows, j]
        if renormalize:
            out[rows, e] += (u * (h - dot) * slope)[rows, j]
            size[rows, e] += (u * (np.abs(h) + mag) * slope)[rows, j]
        else:
            out[rows, e] += (u * h * slope)[rows, j]
            size[rows, e] += (u * np.abs(h) * slope)[rows, j]
    if score == "softmax" and not renormalize:
        rows = some.any(1)
        out[rows] -= s[rows] * dot[rows]
        size[rows] += s[rows] * mag[rows]
    return out, size


def exp_bound(l, experts):
    """Relative error of a weight: exp of a rounded difference d is off by |d| + 2 units, each of the sums by its
    longest chain of additions (a lane's share, five steps over the warp), and a division and a scale follow."""
    with np.errstate(invalid="ignore"):
        spread = np.where(np.isfinite(l), np.abs(l), 0).max(initial=0) * 2
    return 2 * U32 * (2 * spread + experts / 32 + 5 + 12)


# ---- tokens and experts ----------------------------------------------------------------------------------------

def group(ids, experts):
    flat = ids.reshape(-1)
    kept = [i for i in range(len(flat)) if 0 <= flat[i] < experts]
    order = sorted(kept, key=lambda i: (flat[i], i))
    rows = np.full(len(flat), -1)
    rows[order] = np.arange(len(order))
    slots = np.full(len(flat), -1)
    slots[:len(order)] = order
    counts = np.bincount(flat[kept], minlength=experts) if kept else np.zeros(experts, dtype=np.int64)
    return np.concatenate([[0], np.cumsum(counts)]), rows.reshape(ids.shape), slots


def dispatch(x, slots, k):
    out = np.zeros((len(slots), x.shape[1]))
    some = slots >= 0
    out[some] = x[slots[some] // k]
    return out


def combine(y, rows, w):
    """Result and the sum of the terms' magnitudes."""
    out, size = np.zeros((rows.shape[0], y.shape[1])), np.zeros((rows.shape[0], y.shape[1]))
    for j in range(rows.shape[1]):
        some = rows[:, j] >= 0
        term = w[some, j:j + 1] * y[rows[some, j]]
        out[some] += term
        size[some] += np.abs(term)
    return out, size


def combine_backward(g, y, rows, w):
    n = rows.size
    grad_y = np.zeros((n, y.shape[1]))
    grad_w, size = np.zeros(rows.shape), np.zeros(rows.shape)
    for j in range(rows.shape[1]):
        some = rows[:, j] >= 0
        grad_y[rows[some, j]] = w[some, j:j + 1] * g[some]
        grad_w[some, j] = (y[rows[some, j]] * g[some]).sum(1)
        size[some, j] = np.abs(y[rows[some, j]] * g[some]).sum(1)
    return grad_y, grad_w, size


# ---- embedding -------------------------------------------------------------------------------------------------

def embedding(table, tokens, scale):
    flat = tokens.reshape(-1)
    out = np.zeros((len(flat), table.shape[1]))
    some = (flat >= 0) & (flat < len(table))
    out[some] = scale * table[flat[some]]
    return out.reshape(*tokens.shape, table.shape[1])


def embedding_backward(g, tokens, vocab, scale, padding=-1):
    """Result, sums of magnitudes, and terms per row."""
    flat = tokens.reshape(-1)
    g = g.reshape(len(flat), -1)
    out, size = np.zeros((vocab, g.shape[1])), np.zeros((vocab, g.shape[1]))
    some = (flat >= 0) & (flat < vocab) & (flat != padding)
    np.add.at(out, flat[some], scale * g[some])
    np.add.at(size, flat[some], abs(scale) * np.abs(g[some]))
    return out, size, np.bincount(flat[some], minlength=vocab)[:vocab, None]
