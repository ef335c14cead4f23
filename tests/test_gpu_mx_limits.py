"""Microscaled operands at their limits, against the oracle: quotients past the fp32 range, 16-bit values next to the
element grid's midpoints under a tensor scale, and gate values out to where e^-g leaves the range.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import mx as omx  # noqa: E402

DEV = torch.device("cuda:0")
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _quantized(x, fmt, tscale=1.0):
    """The oracle's packed codes and values; a quotient past the fp32 range is infinite there, and goes to 6."""
    with np.errstate(over="ignore"):
        codes, byte = omx.quantize(x, fmt, tscale)
    return omx.pack_codes(codes), omx.values(codes, byte, fmt, tscale), byte


@pytest.mark.parametrize("tscale", [1e-3, 1e-6, 2.0 ** -60, 2.0 ** -90])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_magnitudes_over_six_keep_their_sign(dtype, tscale):
    """A tensor scale so small that the block scale saturates and x / (s t) exceeds fp32: magnitudes go to 6, signs stay.
    Through quantize_mx and through the product, which quantizes one row in its own kernel and five in one before."""
    K = 64
    big = torch.finfo(DTYPE[dtype]).max
    x = torch.zeros(5, K)
    x[0, :6] = torch.tensor([-3e38, 3e38, -big, big, 1.0, -1.0])
    x[1, 16] = -big
    x[2] = torch.where(torch.arange(K) % 2 == 0, -1.0, 1.0) * 2.0 ** torch.linspace(-100, 127, K).floor()
    x[3] = -x[2]
    x[4, 40:48] = torch.tensor([-1e30, 1e30, -1e35, 1e35, -1e20, 1e20, -0.0, 0.0])
    x = x.to(DTYPE[dtype])
    want, values, byte = _quantized(x.float().numpy(), "NVFP4", tscale)
    codes, scales = uq.quantize_mx(x.to(DEV), "NVFP4", tscale=tscale)
    assert np.array_equal(codes.cpu().numpy(), want)
    # the product with a scaled identity: every output is one exact product, times the tensor scale in fp32
    wc, wb = omx.quantize(np.eye(K, dtype=np.float32), "NVFP4")
    w = (torch.from_numpy(omx.pack_codes(wc)).to(DEV), torch.from_numpy(omx.tile_scales(wb, "NVFP4")).to(DEV))
    one = np.diag(omx.values(wc, wb, "NVFP4"))
    ref = (values / float(np.float32(tscale)) * one).astype(np.float32) * np.float32(tscale)
    for rows in (slice(0, 5), slice(0, 1), slice(2, 4)):
        y = uq.gemm_mx(x[rows].to(DEV), w, "NVFP4", tscale=tscale, dtype=torch.float32)
        assert np.array_equal(y.cpu().numpy(), ref[rows])
    assert uq.device_fault() == 0


def _step(v, dtype, up):
    """The neighbouring value of the 16-bit type, away from zero (up) or towards it; v > 0."""
    bits = v.view(torch.int16) + (1 if up else -1)
    return bits.to(torch.int16).view(DTYPE[dtype])


@pytest.mark.parametrize("tscale", [1.0, 0.1, 1.0 / 3, 0.0371, 1.7])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_16_bit_quotients_next_to_ties(dtype, tscale):
    """The 16-bit values on both sides of every midpoint of the element grid, for every scale mantissa: bit for bit the
    fp32 quotient's codes."""
    t = np.float32(tscale)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for b in range(0x20, 0x60):                                                     # e4m3 scales 2^-3 .. 2^4
        d = float(np.float32(omx.E4M3[b]) * t)
        c = (mids * d).to(DTYPE[dtype])
        x = torch.zeros(32, dtype=DTYPE[dtype])
        x[0] = x[16] = 6 * d
        x[1:8], x[8:15] = c, _step(c, dtype, False)
        x[17:24], x[24:31] = _step(c, dtype, True), -c
        rows.append(x)
    x = torch.stack(rows)
    want, _, _ = _quantized(x.float().numpy(), "NVFP4", tscale)
    codes, _ = uq.quantize_mx(x.to(DEV), "NVFP4", tscale=tscale)
    assert np.array_equal(codes.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("power", [-20, -3, 0, 2])
def test_quotients_nearest_to_an_fp32_midpoint(dtype, power):
    """x / d lies 2^-48 (relative) above the middle between 0.25, a tie of the element grid, and the fp32 value after it,
    for x = 2^(power - 1) and d = (2 - 2^-23) 2^power.  Of all divisors and 16-bit values it is the nearest to such a
    middle; the next are 2^-43 away (enumerated over all 2^23 divisor mantissas and the seven midpoints)."""
    t = float(np.float32(2.0 - 2.0 ** -23) * np.float32(2.0 ** power))
    x = torch.zeros(4, 32, dtype=torch.float32)
    for r, s in enumerate((1.0, -1.0)):
        x[r, 0] = x[r, 16] = 12.0 * 2.0 ** power                                    # block scale 1
        x[r, 1:9] = s * 2.0 ** (power - 1)
        x[r, 17:25] = s * 2.0 ** (power - 1) * torch.tensor([1.0, 3.0, 5.0, 7.0, 10.0, 14.0, 20.0, 0.5])
    x = x.to(DTYPE[dtype])
    want, _, byte = _quantized(x.float().numpy(), "NVFP4", t)
    assert (byte[:2] == 0x38).all() and (want[0, 1] & 15) == 1
    codes, _ = uq.quantize_mx(x.to(DEV), "NVFP4", tscale=t)
    assert np.array_equal(codes.cpu().numpy(), want)


def _sums(values, K):
    """Weight rows fp32 [len(values)][K] of multiples of 0.5 up to 4 that add up to each value (multiples of 0.5)."""
    w = np.zeros((len(values), K), np.float32)
    for r, v in enumerate(values):
        left, s = abs(v), np.sign(v)
        for k in range(K):
            step = min(4.0, left) if min(4.0, left) in omx.GRID else max(c for c in omx.GRID if c <= min(4.0, left))
            w[r, k] = s * step
            left -= step
        assert left == 0
    return w


@pytest.mark.parametrize("R", [1, 20, 700])
def test_gate_values_out_to_the_range_of_fp32(R):
    """silu(g) for g to +-130.  Its relative error is that of ex2 (2^-22), 1 + e^-g (2^-24), the reciprocal (2^-23, and half
    a subnormal step where it is subnormal) and two products (2^-24 each), under 2^-20 in all; past g = -88.72 e^-g
    exceeds fp32 and the result is zero."""
    K = 64
    g = np.arange(-130, 130.5, 0.5)
    # one block scale for all: the values are the e2m1 grid's, at scale 1
    wc = omx.e2m1_encode(np.abs(_sums(g, K))) | (np.signbit(_sums(g, K)).astype(np.uint8) << 3)
    byte = np.full((len(g), K // 32), 127, np.uint8)
    w = (torch.from_numpy(omx.pack_codes(wc)).to(DEV)[None], torch.from_numpy(omx.tile_scales(byte, "MXFP4")).to(DEV)[None])
    uc = np.zeros((len(g), K), np.uint8)
    uc[:, 0] = 2                                                                     # up = 1
    up = (torch.from_numpy(omx.pack_codes(uc)).to(DEV)[None], w[1])
    off = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    q = uq.quantize_mx(torch.ones(R, K, dtype=torch.bfloat16, device=DEV), "MXFP4", offsets=off)
    for scale in (1.0, 0.99, 0.9871):
        alpha = torch.tensor([scale], dtype=torch.float32, device=DEV)
        y = uq.gemm_mx_grouped(q, w, off, "MXFP4", up=up, alpha=alpha, dtype=torch.float32).cpu().numpy().astype(np.float64)
        gs = (g.astype(np.float32) * np.float32(scale)).astype(np.float64)
        ref = gs / (1 + np.exp(-gs))
        inside = gs > -88.72
        assert np.array_equal(y, np.broadcast_to(y[0], y.shape))
        lim = 2.0 ** -20 * np.abs(ref) + np.abs(gs) * 2.0 ** -149
        assert np.all(np.abs(y[0] - ref)[inside] <= lim[inside]), np.max((np.abs(y[0] - ref) / lim)[inside])
        assert not y[0][~inside].any()


def test_gate_of_infinities_and_nan():
    """alpha carries the gate to +-inf and NaN: silu(inf) u = inf u, silu(-inf) and silu(NaN) are NaN as g / (1 + e^-g) is."""
    x = torch.ones(3, 64, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    q = uq.quantize_mx(x, "MXFP4", offsets=off)
    w1 = uq.quantize_mx(torch.ones(130, 64, dtype=torch.bfloat16, device=DEV), "MXFP4")
    w = (w1[0].repeat(3, 1, 1), w1[1].repeat(3, 1))
    alpha = torch.tensor([float("inf"), float("-inf"), float("nan")], device=DEV)
    y = uq.gemm_mx_grouped(q, w, off, "MXFP4", up=w, alpha=alpha, dtype=torch.float32)
    assert torch.isposinf(y[0]).all() and torch.isnan(y[1:]).all()
