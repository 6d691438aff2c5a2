"""Routing of tokens to experts in float64 (CPU oracle).

Pins: a row-by-row restatement with Python's sort, closed cases, and central differences for
the gradient.
"""

import numpy as np


def sigmoid(x):
    """(s, 1 - s), both to a few units of rounding wherever s lies."""
    t = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, t) / (1.0 + t), np.where(x >= 0, t, 1.0) / (1.0 + t)


def scores(x, scoring):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        if scoring == "sigmoid":
            return sigmoid(x)[0]
        top = x.max(1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        total = e.sum(1, keepdims=True)
        return e / np.where(total > 0, total, 1.0)


def shares(c, scoring):
    """Scores of the chosen logits c (minus infinity: none) over their sum, taken relative to the
    largest, so that small scores do not vanish: softmax exp(c), sigmoid exp(min(c, 0)) / (1 +
    exp(-|c|)), each divided by the largest exp."""
    low = c if scoring == "softmax" else np.minimum(c, 0.0)
    top = low.max(1, keepdims=True)
    u = np.exp(low - np.where(np.isfinite(top), top, 0.0))
    if scoring == "sigmoid":
        u = u / (1.0 + np.exp(-np.abs(c)))
    total = u.sum(1, keepdims=True)
    return u / np.where(total > 0, total, 1.0)


def route(x, k, scoring, bias=None, n_group=1, topk_group=1, group_rule="max", renorm=True, scale=1.0):
    """(indices, weights): best first, ties to the lower index, -1 and 0 where no expert is left."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    s = scores(x, scoring)
    # without a bias and with groups ranked by their best, scores order like logits
    by_logit = bias is None and (n_group == 1 or group_rule == "max")
    key = x.copy() if by_logit else s + (0.0 if bias is None else np.asarray(bias, np.float64))
    key[x == -np.inf] = -np.inf
    if n_group > 1:
        per = np.sort(key.reshape(T, n_group, -1), axis=2)
        g = per[:, :, -1].copy()
        if group_rule == "top2" and per.shape[2] > 1:
            second = per[:, :, -2]
            g = np.where(second > -np.inf, g + np.where(second > -np.inf, second, 0.0), g)
        order = np.argsort(-g, axis=1, kind="stable")
        lose = np.ones((T, n_group), bool)
        np.put_along_axis(lose, order[:, :topk_group], False, axis=1)
        key = np.where(np.repeat(lose, E // n_group, axis=1), -np.inf, key)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    left = np.take_along_axis(key, idx, 1) > -np.inf
    u = np.where(left, np.take_along_axis(s, idx, 1), 0.0)
    if renorm:
        u = shares(np.where(left, np.take_along_axis(x, idx, 1), -np.inf), scoring)
    return np.where(left, idx, -1).astype(np.int32), u * scale


def weights_of(x, idx, scoring, renorm, scale):
    """The weights as a function of the logits for fixed indices."""
    s = scores(x, scoring)
    ok = (idx >= 0) & (idx < x.shape[1])
    u = np.where(ok, np.take_along_axis(s, np.where(ok, idx, 0), 1), 0.0)
    if renorm:
        total = u.sum(1, keepdims=True)
        u = u / np.where(total > 0, total, 1.0)
    return u * scale


def backward(x, idx, dw, scoring, renorm, scale):
    """(d logits, magnitude of the terms it is summed from) in float64."""
    x, dw = np.asarray(x, np.float64), np.asarray(dw, np.float64)
    T, E = x.shape
    s = scores(x, scoring)
    ok = (idx >= 0) & (idx < E)
    at = np.where(ok, idx, 0)
    u = np.where(ok, np.take_along_axis(s, at, 1), 0.0)
    rest = sigmoid(x)[1]                  # 1 - s without its cancellation
    g = np.where(ok, dw * scale, 0.0)
    ds, mag = np.zeros((T, E)), np.zeros((T, E))
    rows = np.broadcast_to(np.arange(T)[:, None], idx.shape)
    if renorm:
        p = shares(np.where(ok, np.take_along_axis(x, at, 1), -np.inf), scoring)
        mean, mmean = (g * p).sum(1, keepdims=True), (np.abs(g) * p).sum(1, keepdims=True)
        f = p if scoring == "softmax" else p * np.take_along_axis(rest, at, 1)
        np.add.at(ds, (rows, at), np.where(ok, f * (g - mean), 0.0))
        np.add.at(mag, (rows, at), np.where(ok, f * (np.abs(g) + mmean), 0.0))
        return ds, mag
    np.add.at(ds, (rows, at), g)
    np.add.at(mag, (rows, at), np.abs(g))
    if scoring == "sigmoid":
        return ds * s * rest, mag * s * rest
    return (s * (ds - (ds * s).sum(1, keepdims=True)), s * (mag + (mag * s).sum(1, keepdims=True)))
