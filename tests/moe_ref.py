"""The calls of include/gmm_moe.h in 64 bits, with numpy, from their formulas."""
import math

import numpy as np

NONE = -1
F32_MAX = float(np.finfo(np.float32).max)


def clean(logits):
    """float64 logits, -inf where the expert is off."""
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, F32_MAX)


def scores(l, score):
    """Scores of every expert, 0 where it is off."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.where(l > -np.inf, 1 / (1 + np.exp(-l)), 0.0)
        top = l.max(axis=1, keepdims=True)
        e = np.where(l > -np.inf, np.exp(l - np.where(top > -np.inf, top, 0.0)), 0.0)
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def share(l, ids, score):
    """score / sum of the chosen scores, from logarithms so that nothing vanishes; l in float64."""
    T, k = ids.shape
    out = np.zeros((T, k))
    for t in range(T):
        at = [j for j in range(k) if ids[t, j] >= 0 and l[t, ids[t, j]] > -np.inf]
        if not at:
            continue
        z = l[t, ids[t, at]]
        logs = z if score == "softmax" else -np.logaddexp(0.0, -z)
        e = np.exp(logs - logs.max())
        out[t, at] = e / e.sum()
    return out


def route(logits, k, bias=None, score="softmax", normalize=True, scale=1.0):
    l = clean(logits)
    s = scores(l, score)
    key = l.copy()
    if bias is not None:
        with np.errstate(invalid="ignore"):
            key = np.where(l > -np.inf, s + np.asarray(bias, dtype=np.float64), -np.inf)
        key[np.isnan(key)] = -np.inf
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ids = np.where(np.take_along_axis(key, order, 1) > -np.inf, order, NONE)
    if normalize:
        w = share(l, ids, score)
    else:
        w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    return ids.astype(np.int32), scale * w


def route_bwd(dweights, logits, ids, score="softmax", normalize=True, scale=1.0):
    """(gradient, the sum of the magnitudes of the terms each value is made of)."""
    l = clean(logits)
    T, E = l.shape
    s = scores(l, score)
    dw = np.asarray(dweights, dtype=np.float64)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    q = share(l, ids, score) if normalize else None
    for t in range(T):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and l[t, ids[t, j]] > -np.inf]
        e = ids[t, at]
        if normalize:
            dot, adot = (q[t, at] * dw[t, at]).sum(), (q[t, at] * abs(dw[t, at])).sum()
            slope = 1 / (1 + np.exp(np.minimum(l[t, e], 700))) if score == "sigmoid" else 1.0
            np.add.at(out[t], e, scale * q[t, at] * (dw[t, at] - dot) * slope)
            np.add.at(mag[t], e, abs(scale) * q[t, at] * (abs(dw[t, at]) + adot) * slope)
        elif score == "sigmoid":
            g = s[t, e] * (1 / (1 + np.exp(np.minimum(l[t, e], 700))))
            np.add.at(out[t], e, scale * dw[t, at] * g)
            np.add.at(mag[t], e, abs(scale * dw[t, at]) * g)
        else:
            d, a = np.zeros(E), np.zeros(E)
            np.add.at(d, e, dw[t, at])
            np.add.at(a, e, abs(dw[t, at]))
            out[t] = scale * s[t] * (d - (s[t, e] * dw[t, at]).sum())
            mag[t] = abs(scale) * s[t] * (a + (s[t, e] * abs(dw[t, at])).sum())
    return out, mag


def order(ids, G, first=0, rows=None):
    """(group_sizes, row_of, slot_of)."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64)
    M = flat.size if rows is None else rows
    slots = np.concatenate([np.flatnonzero(flat == first + g) for g in range(G)] + [np.zeros(0, np.int64)])
    kept = slots[:M]
    row_of, slot_of = np.full(flat.size, NONE), np.full(M, NONE)
    row_of[kept] = np.arange(kept.size)
    slot_of[:kept.size] = kept
    gs = np.bincount(flat[kept] - first, minlength=G)
    return gs.astype(np.int32), row_of.reshape(np.shape(ids)).astype(np.int32), slot_of.astype(np.int32)


def dispatch(x, slot_of, k):
    out = np.zeros((slot_of.size, x.shape[1]))
    out[slot_of >= 0] = x[slot_of[slot_of >= 0] // k]
    return out


def combine(y, row_of, weights=None, residual=None):
    """(tokens, the sum of the magnitudes of what is added)."""
    T, k = row_of.shape
    out = np.zeros((T, y.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    mag = np.abs(out)
    for j in range(k):
        t = np.flatnonzero(row_of[:, j] >= 0)
        w = 1.0 if weights is None else np.asarray(weights, dtype=np.float64)[t, j][:, None]
        v = w * y[row_of[t, j]]
        out[t] += v
        mag[t] += np.abs(v)
    return out, mag


def combine_bwd(dout, y, row_of, weights, M):
    """(dy, dweights, the sums of the magnitudes that dweights adds)."""
    T, k = row_of.shape
    dy, dw, mag = np.zeros((M, dout.shape[1])), np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        t = np.flatnonzero(row_of[:, j] >= 0)
        r = row_of[t, j]
        dy[r] = np.asarray(weights, dtype=np.float64)[t, j][:, None] * dout[t]
        dw[t, j] = (dout[t] * y[r]).sum(1)
        mag[t, j] = np.abs(dout[t] * y[r]).sum(1)
    return dy, dw, mag


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(name, z):
    """(value, slope)."""
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore"):
        if name == "relu":
            return np.maximum(z, 0), (z > 0).astype(np.float64)
        if name == "gelu":
            cdf = 0.5 * _erfc(-z / math.sqrt(2))
            return z * cdf, cdf + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if name == "silu":
            u, du = z, 1.0
        elif name == "gelu_tanh":
            r = math.sqrt(2 / math.pi)
            u, du = 2 * r * (z + 0.044715 * z ** 3), 2 * r * (1 + 3 * 0.044715 * z * z)
        else:
            return z, np.ones_like(z)
        s = 1 / (1 + np.exp(-u))
    return z * s, s + z * s * (1 - s) * du
