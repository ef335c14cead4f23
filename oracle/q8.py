"""Rows in 8 bits in float64: the quantizer (its fp32 divisions as defined), the norm that ends in it and its gradient, and
the product of two operands with a scale per row."""
import numpy as np


def quantize(x):
    """int8 codes and fp32 scales of rows: s = max|x| / 127, code = RNE(x / s), fp32 divisions (x exact in fp32)."""
    x = np.asarray(x, np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        most = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
        bad = ~np.isfinite(x).all(axis=1)
        s = np.where(bad, np.float32(np.nan), most / np.float32(127))
        d = np.where(bad | (s == 0), np.float32(1), s)[:, None]
        q = np.clip(np.rint(x / d), -127, 127)
    return np.where((bad | (s == 0))[:, None], 0, q).astype(np.int8), s.astype(np.float32)


def rmsnorm(h, gamma, eps):
    """y = h / sqrt(mean(h^2) + eps) * gamma, and max|y| / 127 of each row."""
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * gamma
    return y, np.abs(y).max(axis=1) / 127


def rmsnorm_grad(dy, h, gamma, eps, dh=None):
    r = 1 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    n, g = h * r, dy * gamma
    dx = r * (g - n * (g * n).mean(axis=1, keepdims=True))
    return dx if dh is None else dx + dh, (dy * n).sum(axis=0)


def gemm(xq, sx, wq, sw):
    """(y, magnitude): the product, and the sum of its 1024-k parts' magnitudes, both scaled."""
    x, w = xq.astype(np.float64), wq.astype(np.float64)
    scale = np.outer(sx.astype(np.float64), sw.astype(np.float64))
    parts = [x[:, k:k + 1024] @ w[:, k:k + 1024].T for k in range(0, x.shape[1], 1024)]
    zero = np.zeros(scale.shape)
    return sum(parts, zero) * scale, sum((np.abs(p) for p in parts), zero) * np.abs(scale)
