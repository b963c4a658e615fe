"""Plain fp64 CPU oracle of routing by scores and of the blockwise 8-bit quantiser and product.

TEST INFRASTRUCTURE ONLY (as ``moe_ref``).  Plain numpy, loops over tokens and blocks.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_encode_rne, e4m3_to_f64

INF = np.inf


# ------------------------------------------------------------------ routing by scores
def scores(x, sigmoid):
    """Scores of one token's logits in fp64; a logit of -inf scores 0."""
    x = np.asarray(x, np.float64)
    if sigmoid:
        with np.errstate(over="ignore"):
            return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    top = x.max()
    if top == -INF:
        return np.zeros_like(x)
    with np.errstate(invalid="ignore"):
        e = np.exp(x - top)
        return e / e.sum()


def choose(x, k, sigmoid, bias=None, groups=1, group_topk=1, group_best=1):
    """The experts of one token, in order, as a list of at most k ids; None for a token that has a NaN."""
    s = scores(x, sigmoid)
    E = len(x)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    if np.isnan(x).any() or np.isnan(b).any() or np.isnan(s).any():
        return None
    c = {e: s[e] + b[e] for e in range(E) if x[e] != -INF and b[e] != -INF}
    each = E // groups
    value = {}
    for e in c:
        value.setdefault(e // each, []).append(c[e])
    value = {g: sum(sorted(v, reverse=True)[:group_best]) for g, v in value.items()}
    stay = sorted(value, key=lambda g: (-value[g], g))[:group_topk]
    return sorted((e for e in c if e // each in stay), key=lambda e: (-c[e], e))[:k]


def route(logits, k, sigmoid, renormalise, scale=1.0, bias=None, mask=None, groups=1, group_topk=1, group_best=1):
    """ids [T, k] (-1: none) and weights [T, k] in fp64."""
    T, E = logits.shape
    ids, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        x = logits[t].astype(np.float64)
        got = choose(x, k, sigmoid, bias, groups, group_topk, group_best)
        if got is None:
            w[t] = np.nan
            continue
        ids[t, :len(got)] = got
        w[t, :len(got)] = weights(x, got, sigmoid, renormalise, scale)
    return ids, w


def weights(x, ids, sigmoid, renormalise, scale=1.0):
    """Weights of one token's chosen experts, from logarithms of the scores, so that none underflows."""
    x = np.asarray(x, np.float64)
    if not len(ids):
        return np.zeros(0)
    l = x[ids]
    if sigmoid:
        log_s = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
    else:
        top = x.max()
        log_s = l - top - np.log(np.exp(x - top).sum())
    if renormalise:
        log_s = log_s - log_s.max()
        s = np.exp(log_s)
        return scale * s / s.sum()
    return scale * np.exp(log_s)


def backward(logits, ids, d_w, sigmoid, renormalise, scale=1.0):
    """d_logits [T, E], by the chain rule through the scores."""
    T, E = logits.shape
    d = np.zeros((T, E))
    size = np.zeros((T, E))   # the sum of the terms' magnitudes
    for t in range(T):
        at = [j for j, e in enumerate(ids[t]) if 0 <= e < E]
        if not at:
            continue
        e = ids[t][at]
        x = logits[t].astype(np.float64)
        g = scale * np.asarray(d_w[t], np.float64)[at]
        q = weights(x, e, sigmoid, renormalise)       # normalised scores, or the scores
        s = scores(x, sigmoid)
        if renormalise:
            # dq_i / dlog s_j = q_i (1{i = j} - q_j)
            dlog, slog = q * (g - (g * q).sum()), q * (np.abs(g) + np.abs(g * q).sum())
        else:
            dlog, slog = g * q, np.abs(g * q)
        if sigmoid:                                    # dlog s_j / dl_j = 1 - s_j
            f = scores(-x, True)[e]
            np.add.at(d[t], e, dlog * f)
            np.add.at(size[t], e, slog * f)
        elif renormalise:                              # the sum over all experts drops out
            np.add.at(d[t], e, dlog)
            np.add.at(size[t], e, slog)
        else:                                          # dlog s_j / dl_e = 1{e = j} - s_e
            d[t] -= s * dlog.sum()
            size[t] += s * slog.sum()
            np.add.at(d[t], e, dlog)
            np.add.at(size[t], e, slog)
    return d, size


def bias_update(counts, rate, bias):
    counts = np.asarray(counts, object)                # whole numbers of any size
    over = counts * len(counts) - counts.sum()
    return np.asarray(bias, np.float64) + rate * np.array([float((o < 0) - (o > 0)) for o in over])


# ------------------------------------------------------------------ blockwise e4m3
def blocks_of(n):
    return (n + 127) // 128


def quantize(x, form):
    """codes (uint8) and scales (fp32) of fp32 values, in the format's own fp32 arithmetic: scale = m / 448,
    factor = 448 / m, code = e4m3(value * factor), every quotient and product rounded to fp32."""
    x = np.asarray(x, np.float32)
    if form == "tokens":
        x = np.ascontiguousarray(x.T)
    R, C = x.shape
    step = 128 if form == "tiles" else 1
    scales = np.ones((blocks_of(R) if form == "tiles" else R, blocks_of(C)), np.float32)
    codes = np.zeros((R, (C + 15) // 16 * 16), np.uint8)
    least, top = np.float32(448 * 2.0 ** -126), np.float32(448)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            b = x[i * step:(i + 1) * step, j * 128:(j + 1) * 128]
            m = np.abs(b).max()
            if m > 0:
                m = max(m, least)
                scales[i, j] = m / top
                b = b * (top / m)
            codes[i * step:(i + 1) * step, j * 128:j * 128 + b.shape[1]] = e4m3_encode_rne(b)
    return codes, scales


def values(codes, scales):
    """What codes [R, C] with scales [R or ceil(R / 128), ceil(C / 128)] stand for, exactly, in fp64."""
    v = e4m3_to_f64(codes)
    R, C = v.shape
    s = np.repeat(np.asarray(scales, np.float64), 128, 1)[:, :C]
    if s.shape[0] != R:
        s = np.repeat(s, 128, 0)[:R]
    with np.errstate(invalid="ignore"):   # 0 times an infinite scale
        return v * s
