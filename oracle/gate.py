"""Router gate, load-balance loss and their backward, in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

  * A logit that is NaN or -inf makes its expert ineligible (score 0); +inf
    counts as the largest finite fp32 value.
  * scores: softmax over the eligible experts, or sigmoid.
  * choice: the topk largest keys (the logit, or score + bias), decreasing,
    equal keys to the lower index; -1 where nothing eligible is left or the
    token is masked.
  * weights: route_scale * score, divided by the chosen scores' sum when asked.
  * loss: coef / S * sum over s, i of f * P with f = c E / (topk n), P the mean
    of the scores divided by their sum, over the unmasked tokens of sequence s
    (group-offset rule; tokens behind the last sequence do not count).
"""
from __future__ import annotations

import numpy as np

from .quant import group_bounds

FLT_MAX = float(np.finfo(np.float32).max)


def eligible_logits(logits: np.ndarray) -> np.ndarray:
    z = np.asarray(logits, np.float64)
    return np.minimum(np.where(np.isnan(z), -np.inf, z), FLT_MAX)


def scores(z: np.ndarray, sigmoid: bool) -> np.ndarray:
    out = np.zeros_like(z)
    for t in range(z.shape[0]):
        ok = z[t] > -np.inf
        if not ok.any():
            continue
        if sigmoid:
            with np.errstate(over="ignore"):
                out[t, ok] = 1.0 / (1.0 + np.exp(-z[t, ok]))
        else:
            e = np.exp(z[t, ok] - z[t, ok].max())
            out[t, ok] = e / e.sum()
    return out


def gate(logits, topk: int, sigmoid: bool, bias=None, mask=None, renorm: bool = False, route_scale: float = 1.0):
    """-> (ids int32 [T, topk], weights fp64 [T, topk])."""
    z = eligible_logits(logits)
    s = scores(z, sigmoid)
    T = z.shape[0]
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        key = z[t] if bias is None else np.where(z[t] > -np.inf, s[t] + np.asarray(bias, np.float64), -np.inf)
        key = np.where(np.isnan(key), -np.inf, key)
        order = np.argsort(-key, kind="stable")[:topk]
        order = order[key[order] > -np.inf]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[t, order]
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * route_scale


def sequences(seq_offs, T: int):
    return [(0, T)] if seq_offs is None else list(zip(*group_bounds(seq_offs, T)))


def shares(z: np.ndarray, sigmoid: bool) -> np.ndarray:
    s = scores(z, sigmoid)
    tot = s.sum(axis=1, keepdims=True)
    return np.divide(s, tot, out=np.zeros_like(s), where=tot > 0)


def balance(logits, ids, coef: float, seq_offs, sigmoid: bool, mask=None):
    """-> (loss, counts int64 [S, E], dprob fp64 [S, E])."""
    z = eligible_logits(logits)
    T, E = z.shape
    p = shares(z, sigmoid)
    seqs = sequences(seq_offs, T)
    S, k = len(seqs), ids.shape[1]
    counts, dprob, loss = np.zeros((S, E), np.int64), np.zeros((S, E)), 0.0
    for s, (lo, hi) in enumerate(seqs):
        rows = [t for t in range(lo, hi) if mask is None or mask[t]]
        if not rows:
            continue
        n = len(rows)
        chosen = ids[rows].ravel()
        counts[s] = np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
        f = counts[s] * E / (k * n)
        loss += coef / S * (f * p[rows].mean(axis=0)).sum()
        dprob[s] = coef / S * f / n
    return loss, counts, dprob


def backward(logits, ids, dweights, sigmoid: bool, mask=None, renorm: bool = False, route_scale: float = 1.0, dprob=None,
             dloss: float = 1.0, seq_offs=None):
    """-> (dlogits fp64 [T, E], size fp64 [T, E]): the gradient, and the sum of the magnitudes of the terms it is a sum of
    (what its rounding errors scale with)."""
    z = eligible_logits(logits)
    T, E = z.shape
    s = scores(z, sigmoid)
    ds, mag = np.zeros((T, E)), np.zeros((T, E))
    on = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    if dprob is not None:
        for i, (lo, hi) in enumerate(sequences(seq_offs, T)):
            ds[lo:hi] = dloss * dprob[i]
            mag[lo:hi] = np.abs(ds[lo:hi])
        if sigmoid:
            tot = s.sum(axis=1, keepdims=True)
            inv = np.divide(1.0, tot, out=np.zeros_like(tot), where=tot > 0)
            mag = (mag + (mag * s * inv).sum(axis=1, keepdims=True)) * inv
            ds = (ds - (ds * s * inv).sum(axis=1, keepdims=True)) * inv
    if dweights is not None:
        for t in range(T):
            j = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
            i = ids[t, j]
            dw = np.asarray(dweights, np.float64)[t, j] * route_scale
            size = np.abs(dw)
            if renorm:
                tot = s[t, i].sum()
                if not tot > 0:
                    continue
                u = s[t, i] / tot
                dw, size = (dw - (dw * u).sum()) / tot, (size + (size * u).sum()) / tot
            np.add.at(ds[t], i, dw)
            np.add.at(mag[t], i, size)
    if sigmoid:
        dz, mag = ds * s * (1 - s), mag * s
    else:
        dz = s * (ds - (ds * s).sum(axis=1, keepdims=True))
        mag = s * (mag + (mag * s).sum(axis=1, keepdims=True))
    return np.where(on[:, None], dz, 0.0), np.where(on[:, None], mag, 0.0)


# ---------------------------------------------------------------- the same gradient by differences
#
# A softmax's (or a quotient's) gradient is u_i (x_i - sum u x) with sum u = 1, which is u_i times the sum over the others
# j of u_j (x_i - x_j): no digits are lost where one u is close to 1.  Scores are kept on the scale of the largest one, and
# a sigmoid's complement is sigmoid(-z).


def sigmoid_parts(z: np.ndarray):
    """(s exp(-min(row maximum, 0)), 1 - s) of logits z [T, N]; (0, 1) for -inf."""
    with np.errstate(over="ignore", invalid="ignore"):
        c = np.minimum(np.max(z, axis=1, keepdims=True, initial=-FLT_MAX), 0.0)
        e = np.exp(-np.abs(z))
        return np.exp(np.minimum(z, 0.0) - c) / (1 + e), np.where(z >= 0, e, 1.0) / (1 + e)


def parts_of_one(z: np.ndarray, sigmoid: bool) -> np.ndarray:
    """Scores over their sum along the rows [T, N], on the scale of the largest (rows of -inf: zeros)."""
    w = sigmoid_parts(z)[0] if sigmoid else np.exp(z - np.max(z, axis=1, keepdims=True, initial=-FLT_MAX))
    tot = w.sum(axis=1, keepdims=True)
    return np.divide(w, tot, out=np.zeros_like(w), where=tot > 0)


LEAST_SIGMOID = -709.78   # 1 / (1 + exp(-z)) is 0 in 64 bits below


def loss_shares(z: np.ndarray, sigmoid: bool) -> np.ndarray:
    """What the loss averages: none for a token whose sigmoids are 0 in 64 bits."""
    p = parts_of_one(z, sigmoid)
    if sigmoid:
        p[np.max(z, axis=1, initial=-FLT_MAX) < LEAST_SIGMOID] = 0.0
    return p


def quotient_gradient(u: np.ndarray, x: np.ndarray, size: np.ndarray):
    """u_i sum over the others j of u_j (x_i - x_j), and the same sum of magnitudes, size standing for |x|."""
    n = u.shape[1]
    rest = np.ones((n, n)) - np.eye(n)
    g = u * ((u @ rest) * x - (u * x) @ rest)
    return g, u * ((u @ rest) * size + (u * size) @ rest)


def backward_by_differences(logits, ids, dweights, sigmoid: bool, mask=None, renorm: bool = False, route_scale: float = 1.0,
                            dprob=None, dloss: float = 1.0, seq_offs=None):
    """backward() for eligible choices, with every term to its own digits -> (dlogits, size), size the sum of the magnitudes
    of the terms that remain (after a sigmoid's complement, and the others' share of a quotient)."""
    z = eligible_logits(logits)
    T, E = z.shape
    on = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    p = loss_shares(z, sigmoid)
    comp = sigmoid_parts(z)[1] if sigmoid else np.ones((T, E))
    ds, mag = np.zeros((T, E)), np.zeros((T, E))     # through the scores' own quotient
    dz, size = np.zeros((T, E)), np.zeros((T, E))    # past it
    if dprob is not None:
        for i, (lo, hi) in enumerate(sequences(seq_offs, T)):
            ds[lo:hi] = dloss * np.asarray(dprob, np.float64)[i]
    mag += np.abs(ds)
    if dweights is not None:
        for t in range(T):
            j = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
            if not j:
                continue
            i = ids[t, j]
            dw = np.asarray(dweights, np.float64)[t, j] * route_scale
            if renorm:
                u = parts_of_one(z[t, i][None], sigmoid)
                g, m = quotient_gradient(u, dw[None], np.abs(dw)[None])
                np.add.at(dz[t], i, g[0])
                np.add.at(size[t], i, m[0])
            elif sigmoid:
                with np.errstate(over="ignore"):
                    s = 1.0 / (1.0 + np.exp(-z[t, i]))
                np.add.at(dz[t], i, s * dw)
                np.add.at(size[t], i, s * np.abs(dw))
            else:
                np.add.at(ds[t], i, dw)
                np.add.at(mag[t], i, np.abs(dw))
    g, m = quotient_gradient(p, ds, mag)
    ok = on[:, None] & (z > -np.inf)
    return np.where(ok, (dz + g) * comp, 0.0), np.where(ok, (size + m) * comp, 0.0)
