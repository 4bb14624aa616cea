"""Plain 64-bit implementations of the routing and int8 operators, for their tests."""

import numpy as np


def clean(x):
    """Logits as the scores take them: +Inf is the largest finite fp32 value, -0 is +0."""
    x = np.asarray(x, np.float64)
    return np.where(x > 3.402823466385288598e38, 3.402823466385288598e38, x) + 0.0


def scores(x, score):
    """Scores of all experts; a NaN logit has no part in the others' softmax."""
    x = clean(x)
    x = np.where(np.isnan(x), -np.inf, x)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-x))
    top = np.max(x, 1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0)
    e = np.exp(x - top)
    total = e.sum(1, keepdims=True)
    return e / np.where(total > 0, total, 1)


def route(rc, logits, bias=None, mask=None):
    """(idx int64 [T, K], weights float64 [T, K]) by the definition in the header."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    x = clean(logits)
    s = scores(logits, rc.score)
    by_logit = bias is None and (rc.num_groups == 1 or rc.group_score == "max")
    key = x.copy() if by_logit else s.copy()
    if bias is not None:
        key = key + np.asarray(bias, np.float64)
    key = np.where(np.isnan(logits) | (logits == -np.inf) | np.isnan(key), -np.inf, key)
    size = E // rc.num_groups
    if rc.num_groups > 1:
        per = -np.sort(-key.reshape(T, rc.num_groups, size), axis=2)
        gs = per[:, :, 0]
        if rc.group_score == "top2" and size > 1:
            gs = np.where(per[:, :, 1] > -np.inf, per[:, :, 0] + per[:, :, 1], per[:, :, 0])
        order = np.argsort(-gs, axis=1, kind="stable")[:, :rc.topk_groups]
        keep = np.zeros((T, rc.num_groups), bool)
        np.put_along_axis(keep, order, True, 1)
        key = np.where(np.repeat(keep, size, 1), key, -np.inf)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :rc.K]
    valid = np.take_along_axis(key, idx, 1) > -np.inf
    w = weights(rc, logits, np.where(valid, idx, -1))
    w[np.isnan(logits).any(1)] = np.nan
    if mask is not None:
        valid &= np.asarray(mask)[:, None]
    return np.where(valid, idx, -1).astype(np.int64), np.where(valid, w, 0.0)


def log_scores(x, score):
    """log of the scores, which does not underflow."""
    x = clean(x)
    if score == "sigmoid":
        return np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
    top = np.max(x, 1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0)
    with np.errstate(divide="ignore", invalid="ignore"):
        return x - top - np.log(np.exp(x - top).sum(1, keepdims=True))


def weights(rc, logits, idx):
    """Weights of given choices (-1: none), float64."""
    logits = np.asarray(logits, np.float64)
    valid = idx >= 0
    ls = log_scores(np.where(np.isnan(logits), -np.inf, logits), rc.score)
    ls = np.where(valid, np.take_along_axis(ls, np.maximum(idx, 0), 1), -np.inf)
    if rc.renormalize:
        top = ls.max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0)
        e = np.exp(ls - top)
        total = e.sum(1, keepdims=True)
        return rc.scale * e / np.where(total > 0, total, 1)
    return rc.scale * np.exp(ls)


def route_backward(rc, logits, idx, g):
    """Gradient of sum(weights * g) with respect to the logits, from the formulas."""
    x = clean(logits)
    T, E = x.shape
    valid = (idx >= 0) & (idx < E)
    at = np.where(valid, idx, 0)
    g = np.where(valid, np.asarray(g, np.float64), 0.0)
    w = np.where(valid, weights(rc, logits, np.where(valid, idx, -1)), 0.0)
    s = scores(logits, rc.score)
    out = np.zeros((T, E))
    rows = np.arange(T)[:, None]
    if rc.renormalize:
        d = w * (g - (g * w).sum(1, keepdims=True) / rc.scale)
        if rc.score == "sigmoid":
            d = d * (1 - s[rows, at])
    elif rc.score == "sigmoid":
        d = g * w * (1 - s[rows, at])
    else:
        d = g * w
        out -= (g * w).sum(1, keepdims=True) * s
    np.add.at(out, (np.broadcast_to(rows, at.shape), at), np.where(valid, d, 0.0))
    return out


def quantize(x):
    """(codes int8, scales float32) of rows given as float64 values of an fp32 or 16-bit type."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(1)
    x = np.where(bad[:, None], 0, x)
    scale = np.abs(x).max(1).astype(np.float32) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(x / scale.astype(np.float64)[:, None])
    codes = np.where(scale[:, None] > 0, np.clip(q, -127, 127), 0).astype(np.int8)
    return codes, np.where(bad, np.float32(np.nan), scale).astype(np.float32)


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1 + np.exp(-x))


def product(a, a_scale, w, w_scale, gated):
    """One group's product in float64, and the gate values (None without a gate)."""
    acc = a.astype(np.int64) @ w.astype(np.int64).T
    y = acc.astype(np.float64) * a_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)[None, :]
    if not gated:
        return y, None
    half = y.shape[1] // 2
    return silu(y[:, :half]) * y[:, half:], y[:, :half]
