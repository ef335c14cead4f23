"""Microscaled operators on the branches that only larger calls take, against the oracle: the quantizer's and the reader's
long units, and more experts than one pass of the products' table takes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import moe as omoe  # noqa: E402
from oracle import mx as omx  # noqa: E402

DEV = torch.device("cuda:0")
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FMTS = ["MXFP4", "NVFP4"]


def _quantized(x, fmt):
    """The oracle's packed codes, values and scale bytes."""
    codes, byte = omx.quantize(x, fmt)
    return omx.pack_codes(codes), omx.values(codes, byte, fmt), byte


def _x(seed, rows, K, dtype):
    g = np.random.default_rng([seed, 17])
    x = g.normal(size=(rows, K))
    x[g.random((rows, K)) < 0.01] *= 20
    x[:, :32] *= (g.random((rows, 1)) < 0.7)                                        # some zero blocks
    return torch.from_numpy(x.astype(np.float32)).to(DTYPE[dtype])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(2500, 288), (1300, 4128)])
def test_quantize_in_long_units(fmt, dtype, rows, K):
    """Enough rows that a warp takes 2048 k at a time: codes, scales and values bit for bit, a last unit that is cut."""
    x = _x(rows, rows, K, dtype)
    want, values, byte = _quantized(x.float().numpy(), fmt)
    codes, scales = uq.quantize_mx(x.to(DEV), fmt)
    assert np.array_equal(codes.cpu().numpy(), want)
    live = omx.tile_scales(np.full_like(byte, 1), fmt) == 1
    assert np.array_equal(scales.cpu().numpy()[live], omx.tile_scales(byte, fmt)[live])
    v = uq.dequant_mx((codes, scales), fmt, dtype=torch.float32)
    assert np.array_equal(v.cpu().numpy().astype(np.float64), values)
    for d in ("bf16", "fp16"):
        assert torch.equal(uq.dequant_mx((codes, scales), fmt, dtype=DTYPE[d]), v.to(DTYPE[d]))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_gathered_in_long_units(fmt, dtype):
    T, K, k, E = 1300, 4128, 3, 7
    x = _x(3, T, K, dtype)
    ids = np.random.default_rng(5).integers(-1, E, (T, k)).astype(np.int32)
    _, pos, off = omoe.sort(ids, E)
    offd = torch.from_numpy(off).to(DEV)
    q = uq.quantize_mx(x.to(DEV), fmt, offsets=offd, pos=torch.from_numpy(pos).to(DEV))
    _, values, _ = _quantized(x.float().numpy(), fmt)
    v = uq.dequant_mx(q, fmt, offsets=offd, dtype=torch.float32)
    assert np.array_equal(v.cpu().numpy().astype(np.float64), omoe.gather(values, pos))


# experts, rows, share of experts without a row, N, K: past one pass of the table (128 experts), its largest, and so many
# rows an expert that a gated tile of the finer format is left one stage beside the table
MANY = [(129, 300, 0.3, 136, 96), (300, 1000, 0.6, 136, 96), (1024, 2000, 0.5, 72, 96), (1024, 1, 0.0, 72, 64),
        (700, 52000, 0.05, 136, 96)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,R,empty,N,K", MANY)
def test_grouped_with_many_experts(fmt, E, R, empty, N, K, gated):
    """Operands of -1, 0 and 1, so that every sum is exact in fp32 whatever its order."""
    g = torch.Generator(device=DEV).manual_seed(E + R)
    p = (torch.rand(E, generator=g, device=DEV) >= empty).float() + 1e-9
    count = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=E)
    off = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), count.cumsum(0))).to(torch.int32)
    x = torch.randint(-1, 2, (R, K), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)

    def weight():
        parts = [uq.quantize_mx(torch.randint(-1, 2, (N, K), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16), fmt)
                 for _ in range(E)]
        return torch.stack([a for a, _ in parts]), torch.stack([b for _, b in parts])

    q = uq.quantize_mx(x, fmt, offsets=off)
    w, up = weight(), weight() if gated else None
    alpha = torch.rand(E, generator=g, device=DEV) + 0.5
    y = uq.gemm_mx_grouped(q, w, off, fmt, up=up, alpha=alpha, dtype=torch.float32)
    xv = uq.dequant_mx(q, fmt, offsets=off, dtype=torch.float32).double()
    o = off.tolist()
    for e in range(E):
        if o[e] == o[e + 1]:
            continue
        rows = xv[o[e]:o[e + 1]]
        s = [rows @ uq.dequant_mx((m[0][e], m[1][e]), fmt, dtype=torch.float32).double().t() for m in (w, up) if m is not None]
        got, sums = y[o[e]:o[e + 1]], s[0].float() * alpha[e]
        if not gated:
            assert torch.equal(got, sums), f"expert {e}"
        else:
            ref = sums.double() * torch.sigmoid(sums.double()) * s[1]
            assert (got.double() - ref).abs().le(2.0 ** -20 * ref.abs()).all(), f"expert {e}"
    assert uq.device_fault() == 0
