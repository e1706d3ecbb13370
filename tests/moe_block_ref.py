"""64-bit references of the norm, the router and the gated activation, in numpy
and from their definitions alone."""

import numpy as np


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


# ------------------------------------------------------------------- norm


def norm(h, w, eps):
    """(y, rstd) of rows h."""
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    return h * r[:, None] * w, r


def norm_grad(g, h, w, r, g_h=None):
    """(d_h, d_w, size of the terms that d_h is summed from)."""
    n, gw = h * r[:, None], g * w
    c = (gw * n).mean(1, keepdims=True)
    d = r[:, None] * (gw - n * c)
    size = r[:, None] * (np.abs(gw) + np.abs(n) * np.abs(gw * n).mean(1, keepdims=True))
    if g_h is not None:
        d, size = d + g_h, size + np.abs(g_h)
    return d, (g * n).sum(0), size


# ------------------------------------------------------------------- gate


def gate(x):
    H = x.shape[1] // 2
    return x[:, :H] * sigmoid(x[:, :H]) * x[:, H:]


def gate_grad(g, x):
    """(d_x, size of the terms that it is summed from)."""
    H = x.shape[1] // 2
    a, u, s, rest = x[:, :H], x[:, H:], sigmoid(x[:, :H]), sigmoid(-x[:, :H])
    d_gate, size = g * u * (s + a * s * rest), np.abs(g * u) * (s + np.abs(a) * s * rest)
    return np.concatenate([d_gate, g * a * s], 1), np.concatenate([size, np.abs(g * a * s)], 1)


# ------------------------------------------------------------------ router


def scores(logits, score):
    if score == "sigmoid":
        return sigmoid(logits)
    with np.errstate(invalid="ignore"):
        e = np.exp(logits - logits.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)


def first(v, k):
    """The places of the k largest of each row, ties to the lowest index."""
    return np.argsort(-v, axis=1, kind="stable")[:, :k]


def route(logits, topk, bias=None, score="softmax", groups=1, topk_groups=1, group_top=1, renormalize=True, scale=1.0):
    """(ids, weights).  Without a bias, and with groups scored by one expert,
    the logits give the order of the scores, also of those that 64 bits round
    to one value."""
    T, E = logits.shape
    bad = np.isnan(logits).any(1) | ((score == "softmax") & np.isposinf(logits.max(1)))
    if bias is not None:
        bad |= np.isnan(bias).any()
    logits = np.where(bad[:, None], 0.0, logits)
    there = logits > -np.inf
    s = np.where(there, scores(np.where(there.any(1, keepdims=True), logits, 0.0), score), 0.0)
    if bias is None and (groups == 1 or group_top == 1):
        c = logits.copy()
    else:
        c = np.where(there, s + (0.0 if bias is None else np.nan_to_num(bias, nan=0.0, posinf=np.inf, neginf=-np.inf)), -np.inf)
    if groups > 1:
        best = -np.sort(-c.reshape(T, groups, -1), axis=2)[:, :, :group_top]
        total = np.where(np.isneginf(best).all(2), -np.inf, np.where(np.isneginf(best), 0.0, best).sum(2))
        kept = np.zeros((T, groups), bool)
        np.put_along_axis(kept, first(total, topk_groups), True, 1)
        c = np.where(np.repeat(kept, E // groups, 1), c, -np.inf)
    ids = first(c, topk)
    ok = np.take_along_axis(c, ids, 1) > -np.inf
    x = np.take_along_axis(logits, ids, 1)
    w = chosen_weights(x, ok, np.take_along_axis(s, ids, 1), score, renormalize) * scale
    ids, w = np.where(ok, ids, -1), np.where(ok, w, 0.0)
    return np.where(bad[:, None], np.arange(topk), ids), np.where(bad[:, None], np.nan, w)


def log_score(x, score):
    """log s up to a constant of the row."""
    return x if score == "softmax" else np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))


def chosen_weights(x, ok, s, score, renormalize):
    if not renormalize:
        return np.where(ok, s, 0.0)
    v = np.where(ok, log_score(np.where(ok, x, 0.0), score), -np.inf)
    m = np.where(ok.any(1, keepdims=True), v.max(1, keepdims=True), 0.0)
    u = np.exp(v - m)
    return u / np.maximum(u.sum(1, keepdims=True), 1e-300)


def route_grad(g, logits, ids, score="softmax", renormalize=True, scale=1.0):
    """(d_logits, size of the terms that it is summed from); ids outside the experts are left out."""
    T, E = logits.shape
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, 0)
    s = scores(logits, score)
    x = np.take_along_axis(logits, at, 1)
    w = chosen_weights(x, ok, np.take_along_axis(s, at, 1), score, renormalize)
    t, size = g * w * scale * ok, np.abs(g * w * scale * ok)
    if renormalize:  # d log w_j / d log s_i = [i = j] - w_i
        t, size = t - w * t.sum(1, keepdims=True), size + w * size.sum(1, keepdims=True)
    rest = sigmoid(-x) if score == "sigmoid" else np.ones_like(x)
    d, S = np.zeros((T, E)), np.zeros((T, E))
    rows = np.repeat(np.arange(T)[:, None], ids.shape[1], 1)
    np.add.at(d, (rows, at), t * rest * ok)
    np.add.at(S, (rows, at), size * rest * ok)
    if score == "softmax" and not renormalize:
        d, S = d - s * t.sum(1, keepdims=True), S + s * size.sum(1, keepdims=True)
    return d, S
