"""The router of a mixture of experts in float64, token by token."""
import math

import numpy as np

LOW = -math.inf


def scores(x, score):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-x))
        m = x.max(axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(m), m, 0))
        return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)


def _rank(c):
    return -1e308 if math.isnan(c) else c


def choose(x, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1):
    """ids [T][k]: by c = score + bias (the logits themselves without a bias), ties to the lower index."""
    s = scores(x, score)
    T, E = s.shape
    size = E // groups
    ids = np.full((T, k), -1, np.int32)
    for t in range(T):
        can = [e for e in range(E) if x[t, e] != LOW and (bias is None or bias[e] != LOW)]
        c = [float(x[t, e]) if bias is None else float(s[t, e]) + float(bias[e]) for e in range(E)]
        if groups > 1:
            by = [float(s[t, e]) for e in range(E)] if bias is None and group_top == 2 else c
            total = {}
            for g in range(groups):
                members = sorted((_rank(by[e]) for e in can if e // size == g), reverse=True)
                if members:
                    total[g] = sum(members[:group_top])
            kept = sorted(total, key=lambda g: (-total[g], g))[:top_groups]
            can = [e for e in can if e // size in kept]
        best = sorted(can, key=lambda e: (-_rank(c[e]), e))[:k]
        ids[t, :len(best)] = best
    return ids


def weights(x, ids, score="softmax", renormalize=True, scale=1.0):
    s = scores(x, score)
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0).astype(np.int64), axis=1), 0.0)
    if renormalize:
        w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    return w * scale


def grad(x, ids, dw, score="softmax", renormalize=True, scale=1.0):
    """dlogits, and for each the magnitude of what was added up."""
    s = scores(x, score)
    T, E = s.shape
    dx, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        at = [int(ids[t, j]) for j in on]
        d = [float(dw[t, j]) * scale for j in on]
        if renormalize:
            total = sum(s[t, e] for e in at)
            w = [s[t, e] / total if total > 0 else 0.0 for e in at]
            mean, size = sum(a * b for a, b in zip(w, d)), sum(a * abs(b) for a, b in zip(w, d))
            for e, a, b in zip(at, w, d):
                f = 1 - s[t, e] if score == "sigmoid" else 1.0
                dx[t, e] += a * (b - mean) * f
                mag[t, e] += a * (abs(b) + size) * f
            continue
        ds, size = np.zeros(E), np.zeros(E)
        for e, b in zip(at, d):
            ds[e] += b
            size[e] += abs(b)
        if score == "sigmoid":
            dx[t], mag[t] = ds * s[t] * (1 - s[t]), size * s[t] * (1 - s[t])
        else:
            dx[t], mag[t] = s[t] * (ds - (s[t] * ds).sum()), s[t] * (size + (s[t] * size).sum())
    return dx, mag
