"""Microscaled operands at their limits, against the oracle: quotients past the fp32 range."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import mx as omx  # noqa: E402

DEV = torch.device("cuda:0")
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


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
