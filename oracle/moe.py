"""Oracle for expert routing (test infrastructure only; NumPy, float64): the stable sort of routes by expert, rows
carried there and back with weights, and the gradients, each from its definition route by route."""
from __future__ import annotations

import numpy as np


def sort(ids: np.ndarray, experts: int):
    """(order [R], pos [T][k], offsets [experts + 1]); routes with an id outside [0, experts) are dropped."""
    flat = ids.reshape(-1)
    kept = [(int(e), i) for i, e in enumerate(flat) if 0 <= e < experts]
    kept.sort()
    order = np.full(flat.size, -1, dtype=np.int32)
    pos = np.full(flat.size, -1, dtype=np.int32)
    for r, (_, i) in enumerate(kept):
        order[r], pos[i] = i, r
    count = np.zeros(experts, dtype=np.int64)
    for e, _ in kept:
        count[e] += 1
    return order, pos.reshape(ids.shape), np.concatenate([[0], np.cumsum(count)]).astype(np.int32)


def gather(x: np.ndarray, pos: np.ndarray) -> np.ndarray:
    xs = np.zeros((pos.size, x.shape[1]))
    for t, j in zip(*np.nonzero(pos >= 0)):
        xs[pos[t, j]] = x[t]
    return xs


def combine(ys: np.ndarray, pos: np.ndarray, weights: np.ndarray) -> np.ndarray:
    y = np.zeros((pos.shape[0], ys.shape[1]))
    for t, j in zip(*np.nonzero(pos >= 0)):
        y[t] += float(weights[t, j]) * ys[pos[t, j]]
    return y


def gather_grad(dxs: np.ndarray, pos: np.ndarray) -> np.ndarray:
    return combine(dxs, pos, np.ones(pos.shape))


def combine_grad(dy: np.ndarray, ys: np.ndarray, pos: np.ndarray, weights: np.ndarray):
    dys, dw = np.zeros_like(ys, dtype=np.float64), np.zeros(pos.shape)
    for t, j in zip(*np.nonzero(pos >= 0)):
        dys[pos[t, j]] = float(weights[t, j]) * dy[t]
        dw[t, j] = dy[t] @ ys[pos[t, j]]
    return dys, dw
