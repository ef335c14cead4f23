"""Pins of the microscaled 4-bit oracle and of the routing oracle (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import moe, mx


def test_e4m3_table_fields():
    v = mx.E4M3
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[7] == 7 * 2.0 ** -9 and v[8] == 2.0 ** -6
    assert v[0x38] == 1.0 and v[0x7E] == 448.0 and np.isnan(v[0x7F]) and v[0xB8] == -1.0
    assert np.all(np.diff(v[:0x7F]) > 0)


@pytest.mark.parametrize("grid,encode", [(mx.GRID, mx.e2m1_encode), (mx.E4M3[:0x7F], mx.e4m3_encode)])
def test_encoders_are_nearest_with_ties_to_even(grid, encode):
    assert np.array_equal(encode(grid), np.arange(len(grid)))
    mid = (grid[:-1] + grid[1:]) / 2
    lower = np.arange(len(mid))
    assert np.array_equal(encode(mid), np.where(lower % 2 == 0, lower, lower + 1))
    assert np.array_equal(encode(np.nextafter(mid, 0)), lower)
    assert np.array_equal(encode(np.nextafter(mid, 1e9)), lower + 1)
    assert encode(np.array([grid[-1] * 3]))[0] == len(grid) - 1


def test_mxfp4_hand_worked_block():
    x = np.zeros((1, 32), np.float32)
    x[0, :8] = [7.9, -2.5, 0.25, 0.75, -0.2, 5.0, 3.5, 1.75]    # absmax 7.9 -> 2^2, scale 2^0
    codes, byte = mx.quantize(x, "MXFP4")
    assert byte[0, 0] == 127
    assert list(mx.values(codes, byte, "MXFP4")[0, :8]) == [6.0, -2.0, 0.0, 1.0, 0.0, 4.0, 4.0, 2.0]
    assert np.signbit(mx.values(codes, byte, "MXFP4")[0, 4])
    x *= np.float32(2.0 ** -20)
    codes2, byte2 = mx.quantize(x, "MXFP4")
    assert np.array_equal(codes, codes2) and byte2[0, 0] == 107


def test_mxfp4_scale_limits_and_non_finite():
    x = np.zeros((5, 32), np.float32)
    x[1, 3] = 2.0 ** -149
    x[2, 3] = np.finfo(np.float32).max
    x[3, 3] = np.inf
    x[4, 3] = np.nan
    codes, byte = mx.quantize(x, "MXFP4")
    assert list(byte[:, 0]) == [0, 0, 252, 255, 255]
    assert codes[1, 3] == 0 and codes[2, 3] == 7
    v = mx.values(codes, byte, "MXFP4")
    assert np.all(v[0] == 0) and np.all(np.isnan(v[3:])) and v[2, 3] == 6 * 2.0 ** 125


def test_nvfp4_hand_worked_block():
    x = np.zeros((1, 16), np.float32)
    x[0, :4] = [12.0, -5.0, 0.5, 1.5]                            # scale 2: 6, -2.5 -> -2, 0.25 -> 0, 0.75 -> 1
    codes, byte = mx.quantize(x, "NVFP4")
    assert mx.E4M3[byte[0, 0]] == 2.0
    assert list(mx.values(codes, byte, "NVFP4")[0, :4]) == [12.0, -4.0, 0.0, 2.0]
    c2, b2 = mx.quantize(x * 4, "NVFP4", tscale=4.0)
    assert np.array_equal(c2, codes) and np.array_equal(b2, byte)
    c3, b3 = mx.quantize(np.full((1, 16), 2.0 ** -9, np.float32), "NVFP4")   # 2^-9 / 6 rounds to scale 0
    assert b3[0, 0] == 0 and not c3.any()


def test_nvfp4_codes_are_nearest_by_exact_rationals():
    rng = np.random.default_rng(3)
    x = (np.round(rng.normal(size=(4, 64)) * 32) / 32).astype(np.float32)     # coarse values: many ties
    codes, byte = mx.quantize(x, "NVFP4")
    grid = [Fraction(g) for g in mx.GRID]
    for r in range(4):
        for k in range(64):
            s = Fraction(float(mx.E4M3[byte[r, k // 16]]))
            q = abs(Fraction(float(x[r, k]))) / s
            best = min(range(8), key=lambda i: (abs(grid[i] - q), i % 2))
            assert codes[r, k] & 7 == best


def test_scale_tile_layout_formula():
    byte = np.arange(130 * 5, dtype=np.int64).reshape(130, 5).astype(np.uint8)
    t = mx.tile_scales(byte, "MXFP4").reshape(2, 2, 32, 4, 4)     # [row tile][k tile][r % 32][r / 32][block]
    assert t[0, 0, 3, 2, 1] == byte[67, 1] and t[1, 1, 1, 0, 0] == byte[129, 4] and t[0, 1, 0, 0, 1] == 0
    offsets = [0, 1, 1, 130]
    at = mx.scale_rows(130, offsets)
    assert at[0] == 0 and at[1] == 2 * 128 and at[129] == 3 * 128     # third segment starts at tile 0 + 2


def test_segments_never_share_a_tile():
    rng = np.random.default_rng(5)
    for _ in range(200):
        E = int(rng.integers(1, 9))
        off = np.concatenate([[0], np.cumsum(rng.integers(0, 300, E))])
        at = mx.scale_rows(int(off[-1]), off)
        assert len(set(at.tolist())) == len(at)
        assert at.size == 0 or at.max() < (off[-1] // 128 + E) * 128
        tiles = [set((at[off[e]:off[e + 1]] // 128).tolist()) for e in range(E)]
        assert sum(len(s) for s in tiles) == len(set().union(*tiles))


def test_routing_hand_worked():
    ids = np.array([[2, 0], [-1, 2], [0, 5]])
    order, pos, off = moe.sort(ids, 3)
    assert list(order) == [1, 4, 0, 3, -1, -1] and pos.tolist() == [[2, 0], [-1, 3], [1, -1]] and list(off) == [0, 2, 2, 4]
    x = np.array([[1.0], [2.0], [3.0]])
    xs = moe.gather(x, pos)
    assert xs[:, 0].tolist() == [1, 3, 1, 2, 0, 0]
    w = np.array([[0.25, 0.75], [0.5, 0.5], [1.0, 0.0]])
    assert moe.combine(xs, pos, w)[:, 0].tolist() == [1.0, 1.0, 3.0]


def test_routing_gradients_by_differences():
    rng = np.random.default_rng(7)
    ids = rng.integers(-1, 4, (6, 3))
    _, pos, _ = moe.sort(ids, 4)
    x, ys, w = rng.normal(size=(6, 5)), rng.normal(size=(18, 5)), rng.random((6, 3))
    dy, dxs = rng.normal(size=(6, 5)), rng.normal(size=(18, 5))
    dys, dw = moe.combine_grad(dy, ys, pos, w)
    dx = moe.gather_grad(dxs, pos)
    loss_c = lambda a, b: (moe.combine(a, pos, b) * dy).sum()                # noqa: E731
    loss_g = lambda a: (moe.gather(a, pos) * dxs).sum()                     # noqa: E731
    h = 1e-6
    for arr, grad, f in ((ys, dys, lambda a: loss_c(a, w)), (w, dw, lambda a: loss_c(ys, a)), (x, dx, loss_g)):
        for i in np.ndindex(arr.shape):
            up, dn = arr.copy(), arr.copy()
            up[i] += h
            dn[i] -= h
            assert abs((f(up) - f(dn)) / (2 * h) - grad[i]) < 1e-6
