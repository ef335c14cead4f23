"""Oracle for microscaled 4-bit floating point (test infrastructure only; NumPy, float64).

e2m1 codes 0..7 stand for 0, 0.5, 1, 1.5, 2, 3, 4, 6, bit 3 is the sign.  MXFP4: blocks of 32 with the scale
2^(byte - 127); NVFP4: blocks of 16 with an e4m3 scale and a tensor scale.  The integer decisions follow the
method's definition: MXFP4's are exact, NVFP4's divide in fp32 (absmax / (6 t), x / (s t)).
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"MXFP4": 32, "NVFP4": 16}


def e4m3_values() -> np.ndarray:
    """Value of every e4m3 byte (exponent bias 7, no infinities, 0x7F and 0xFF NaN)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, np.ldexp(1.0 + m / 8.0, e - 7), np.ldexp(m / 8.0, -6))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


E4M3 = e4m3_values()


def e4m3_encode(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 byte of non-negative values, ties to the even byte, above 448 -> 448."""
    grid = E4M3[:0x7F]
    v = np.minimum(v, 448.0)
    hi = np.searchsorted(grid, v)                      # first value >= v
    lo = np.maximum(hi - 1, 0)
    dl, dh = v - grid[lo], grid[hi] - v
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo).astype(np.uint8)


def e2m1_encode(a: np.ndarray) -> np.ndarray:
    """Nearest e2m1 magnitude code of non-negative values, ties to the even code, above 6 -> 6."""
    a = np.minimum(a, 6.0)
    hi = np.searchsorted(GRID, a)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - GRID[lo], GRID[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo).astype(np.uint8)


def quantize(x: np.ndarray, fmt: str, tscale: float = 1.0):
    """x fp32 [rows][K] -> (codes uint8 [rows][K], scale bytes uint8 [rows][K/block])."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    n = BLOCK[fmt]
    b = x.reshape(rows, K // n, n)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[..., None], np.float32(0), b)
    amax = np.abs(b).max(axis=2)
    if fmt == "MXFP4":
        e = np.frexp(amax.astype(np.float64))[1] - 3            # floor(log2 a) - 2
        byte = np.where(amax > 0, np.clip(e, -127, 127) + 127, 0)
        q = np.ldexp(b.astype(np.float64), 127 - byte[..., None])
        byte = np.where(bad, 255, byte).astype(np.uint8)
    else:
        t = np.float32(tscale)
        byte = e4m3_encode((amax / (np.float32(6) * t)).astype(np.float64))
        d = E4M3[byte].astype(np.float32) * t
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.where(d[..., None] > 0, b / d[..., None], np.float32(0)).astype(np.float64)
        byte = np.where(bad, 0x7F, byte).astype(np.uint8)
    codes = e2m1_encode(np.abs(q)) | (np.signbit(b).astype(np.uint8) << 3)
    return codes.reshape(rows, K), byte


def scale_values(byte: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "MXFP4":
        return np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return E4M3[byte]


def values(codes: np.ndarray, byte: np.ndarray, fmt: str, tscale: float = 1.0) -> np.ndarray:
    """float64 values: code * scale * tensor scale."""
    v = np.where(codes & 8, -GRID[codes & 7], GRID[codes & 7])
    s = scale_values(byte, fmt) * float(np.float32(tscale))
    return v * np.repeat(s, BLOCK[fmt], axis=-1)


def pack_codes(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack_codes(packed: np.ndarray) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)


def scale_rows(rows: int, offsets=None) -> np.ndarray:
    """Row of the scale tiles of every operand row (-1: belongs to no segment)."""
    if offsets is None:
        return np.arange(rows)
    at = np.full(rows, -1, dtype=np.int64)
    for e in range(len(offsets) - 1):
        o, end = int(offsets[e]), int(offsets[e + 1])
        at[o:end] = (o // 128 + e) * 128 + np.arange(end - o)
    return at


def tile_scales(byte: np.ndarray, fmt: str, offsets=None, fill: int = 0) -> np.ndarray:
    """Scale bytes [rows][blocks] -> the 512-byte tiles, element by element from the layout's formula."""
    rows, nb = byte.shape
    kt = -(-nb // 4)
    rt = -(-rows // 128) if offsets is None else rows // 128 + len(offsets) - 1
    out = np.full(rt * kt * 512, fill, dtype=np.uint8)
    at = scale_rows(rows, offsets)
    for blk in range(kt * 4):
        r = at[at >= 0]
        off = ((r // 128) * kt + blk // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + blk % 4
        out[off] = byte[at >= 0, blk] if blk < nb else 0
    return out


def product(xv: np.ndarray, wv: np.ndarray):
    """y = x w^T in float64 and the bound's sum |x w|."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def error_ratio(y, y_ref, bound, K: int, out: str = "bf16") -> np.ndarray:
    """|y - y_ref| over what the method allows: one rounding of the output (2^-8 bf16, 2^-11 fp16, 2^-24 fp32 of
    |y_ref|, half the smallest subnormal for fp16) and an fp32 accumulation of K exact products, each of which may
    lose 2^-23 of the running sum of magnitudes."""
    u = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}[out]
    return np.abs(y - y_ref) / (u * np.abs(y_ref) + K * 2.0 ** -23 * bound + 2.0 ** -25)
