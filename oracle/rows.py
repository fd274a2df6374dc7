"""The plain CPU definition, in fp64 numpy, of the calls around the linears:
router, rows sorted by group, weighted sum of rows, low-rank adapters, and the
two gradients.  It shares no code with the library and takes and returns
numpy arrays (bf16 inputs as their exact float values).
"""
from __future__ import annotations

import numpy as np


def _scores(z, scoring):
    """(score, share) of one row's logits, in fp64; -inf gives 0."""
    if scoring == "softmax":
        e = np.exp(z - z.max())
        p = e / e.sum()
        return p, p
    with np.errstate(over="ignore"):  # exp(-z) of a far z: a score of 0
        s = 1 / (1 + np.exp(-z))
    # shares from scores times exp(-m), m = min(max z, 0), so that a row of
    # very small scores still has them
    m = min(z.max(), 0.0)
    t = np.exp(z - m) / (1 + np.exp(z)) if m < 0 else s
    return s, t / t.sum()


def choose(z, k):
    """Indices of the k largest logits above -inf, ties to the lowest index."""
    key = np.where(np.isnan(z), -np.inf, z)
    at = np.argsort(-key, kind="stable")[:k]
    return [int(i) for i in at if key[i] > -np.inf]


def route(logits, k, scoring="softmax", renormalize=True, scale=1.0, balance=0.0, mask=None):
    """(ids, weights, counts, loss, loss_grad)."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    counts = np.zeros(E, np.int64)
    shares = np.zeros(E)
    n = 0
    with np.errstate(all="ignore"):
        for t in range(T):
            if mask is not None and not mask[t]:
                continue
            at = choose(z[t], k)
            if not at:
                continue
            n += 1
            score, share = _scores(z[t], scoring)
            shares += share
            ids[t, :len(at)] = at
            # the chosen shares are the chosen scores times a factor of the row
            w = share[at] / share[at].sum() if renormalize else score[at]
            weights[t, :len(at)] = scale * w
            counts[at] += 1
    slope = balance * E * counts / (k * max(n, 1) ** 2)
    return ids, weights, counts, float((slope * shares).sum()), slope


def route_backward(logits, ids, d_weights=None, loss_grad=None, d_loss=1.0, scoring="softmax",
                   renormalize=True, scale=1.0):
    """Gradient of sum(d_weights * weights) + d_loss * loss by the chain rule."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    d = np.zeros((T, E))
    for t in range(T):
        at = [int(i) for i in ids[t] if 0 <= i < E]
        if not at:
            continue
        slots = [j for j, i in enumerate(ids[t]) if 0 <= i < E]
        score, share = _scores(z[t], scoring)
        # d share / d z: diag(share f) - share (share f)^T, f = dlog(score)/dz
        f = np.ones(E) if scoring == "softmax" else 1 - score
        g = np.zeros(E)
        if loss_grad is not None:
            up = np.asarray(loss_grad, np.float64) * d_loss
            g += share * f * (up - (share * up).sum())
        if d_weights is not None:
            dw = scale * np.asarray(d_weights[t], np.float64)[slots]
            if renormalize:
                r = share[at] / share[at].sum()
                g[at] += r * f[at] * (dw - (r * dw).sum())
            elif scoring == "sigmoid":
                g[at] += score[at] * f[at] * dw
            else:
                g[at] += score[at] * dw
                g -= score * (score[at] * dw).sum()
        d[t] = g
    return d


def group_rows(ids, groups):
    """(offsets, order, slot)."""
    flat = np.asarray(ids).reshape(-1)
    lists = [[] for _ in range(groups + 1)]
    for i, g in enumerate(flat):
        lists[g if 0 <= g < groups else groups].append(i)
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists[:groups]])]).astype(np.int32)
    order = np.array([i for v in lists for i in v], np.int32)
    slot = np.full(flat.size, -1, np.int32)
    for r, i in enumerate(order[:offsets[-1]]):
        slot[i] = r
    return offsets, order, slot.reshape(np.shape(ids))


def combine_rows(y, weights, slot, base=None):
    y = np.asarray(y, np.float64)
    T, k = slot.shape
    out = np.zeros((T, y.shape[1])) if base is None else np.array(base, np.float64)
    for t in range(T):
        for j in range(k):
            if 0 <= slot[t, j] < y.shape[0]:
                out[t] += float(weights[t, j]) * y[slot[t, j]]
    return out


def combine_rows_backward(d_out, y, weights, slot):
    y, d_out = np.asarray(y, np.float64), np.asarray(d_out, np.float64)
    d_y, d_w = np.zeros_like(y), np.zeros(slot.shape)
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            r = slot[t, j]
            if 0 <= r < y.shape[0]:
                d_y[r] = float(weights[t, j]) * d_out[t]
                d_w[t, j] = d_out[t] @ y[r]
    return d_y, d_w


def lora_add(y, x, a, b, ids, scales=None):
    """out = y + scales[l] (x A_l^T) B_l^T for the rows with ids == l."""
    out = np.array(y, np.float64)
    for l in range(a.shape[0]):
        at = np.nonzero(np.asarray(ids) == l)[0]
        if at.size:
            u = np.asarray(x[at], np.float64) @ np.asarray(a[l], np.float64).T
            out[at] += (1.0 if scales is None else float(scales[l])) * (u @ np.asarray(b[l], np.float64).T)
    return out
