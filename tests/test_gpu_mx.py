"""Microscaled 4-bit operands on the GPU against the oracle: quantization (bit-exact), its inverse, the scale tiles,
the product and the product grouped by expert.

The product's tolerance (oracle/mx.py) is one rounding of the output plus an fp32 accumulation of K exact products,
K * 2^-23 of the sum of magnitudes.  The gated product adds the first-order effect of both sums' errors on silu(g) * u
(|silu'| <= 1.1) and 2^-20 of the result for the fp32 exponential, quotient and product.
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


def _x(seed, rows, K, dtype="bf16", scale=1.0):
    g = np.random.default_rng([seed, 11])
    x = g.normal(size=(rows, K)) * scale
    x[g.random((rows, K)) < 0.01] *= 20
    x[:, : min(K, 32)] *= (g.random((rows, 1)) < 0.7)              # some zero blocks
    return torch.from_numpy(x.astype(np.float32)).to(DTYPE[dtype])


def _np(t):
    return t.float().cpu().numpy()


def _operand(w, fmt, tscale=1.0):
    """Oracle-quantized weight fp32 [N][K] -> ((codes, scales) on the device, float64 values)."""
    codes, byte = omx.quantize(w, fmt, tscale)
    q = (torch.from_numpy(omx.pack_codes(codes)).to(DEV), torch.from_numpy(omx.tile_scales(byte, fmt)).to(DEV))
    return q, omx.values(codes, byte, fmt, tscale)


def _live(byte_tiles, byte, fmt, offsets=None):
    """Where the tiles hold a defined byte: blocks of existing rows (and the zero padding along k)."""
    return omx.tile_scales(np.full_like(byte, 1), fmt, offsets, fill=0) == 1


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 4096), (3, 96), (130, 288), (257, 1056), (64, 14336)])
def test_quantize_is_the_oracles(fmt, dtype, rows, K):
    x = _x(rows + K, rows, K, dtype)
    codes, scales = uq.quantize_mx(x.to(DEV), fmt)
    oc, ob = omx.quantize(_np(x), fmt)
    assert np.array_equal(codes.cpu().numpy(), omx.pack_codes(oc))
    live = _live(None, ob, fmt)
    got = scales.cpu().numpy()
    assert np.array_equal(got[live], omx.tile_scales(ob, fmt)[live])
    v = uq.dequant_mx((codes, scales), fmt, dtype=torch.float32)
    assert np.array_equal(v.cpu().numpy().astype(np.float64), omx.values(oc, ob, fmt))
    if dtype == "bf16":
        assert torch.equal(uq.dequant_mx((codes, scales), fmt).float(), v)          # exact in bf16


def test_quantize_pads_the_last_scale_tile_with_zeros():
    for fmt, K in (("MXFP4", 160), ("NVFP4", 96)):
        codes, scales = uq.quantize_mx(_x(1, 128, K).to(DEV), fmt)
        _, ob = omx.quantize(_np(_x(1, 128, K)), fmt)
        assert np.array_equal(scales.cpu().numpy(), omx.tile_scales(ob, fmt))


@pytest.mark.parametrize("tscale", [0.25, 0.0371])
def test_quantize_nvfp4_tensor_scale(tscale):
    x = _x(5, 33, 512)
    q = uq.quantize_mx(x.to(DEV), "NVFP4", tscale=tscale)
    oc, ob = omx.quantize(_np(x), "NVFP4", tscale)
    assert np.array_equal(q[0].cpu().numpy(), omx.pack_codes(oc))
    v = uq.dequant_mx(q, "NVFP4", tscale=tscale, dtype=torch.float32).cpu().numpy()
    ref = omx.values(oc, ob, "NVFP4", tscale)
    assert np.all(np.abs(v - ref) <= 2.0 ** -22 * np.abs(ref))      # two fp32 roundings


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_limits_and_non_finite(fmt):
    x = torch.zeros(6, 64)
    x[1, 3] = 2.0 ** -149
    x[2, 3] = torch.finfo(torch.float32).max
    x[3, 3] = float("inf")
    x[4, 40] = float("nan")
    x[5] = torch.linspace(-8, 8, 64)
    codes, scales = uq.quantize_mx(x.to(DEV), fmt)
    oc, ob = omx.quantize(x.numpy(), fmt)
    got = uq.dequant_mx((codes, scales), fmt, dtype=torch.float32).cpu().numpy()
    ref = omx.values(oc, ob, fmt).astype(np.float32)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])
    n = omx.BLOCK[fmt]
    assert np.isnan(got[3, :n]).all() and np.isfinite(got[3, n:]).all()             # the block only


@pytest.mark.parametrize("tscale", [1.0, 0.0371, 2.0 ** -110])
def test_quantize_nvfp4_quotients_at_and_next_to_ties(tscale):
    """fp32 values on, one ulp below and one ulp above every midpoint of the element grid, for every scale mantissa: the
    fp32 quotient decides, so the codes are the oracle's bit for bit (also where the scale is too small for a reciprocal)."""
    t = np.float32(tscale)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    rows = []
    for b in range(0x20, 0x60):                                                     # e4m3 scales 2^-3 .. 2^4
        d = np.float32(omx.E4M3[b]) * t
        x = np.zeros(32, np.float32)
        x[0] = x[16] = np.float32(6) * d
        for i, m in enumerate(mids):
            c = m * d
            x[1 + i], x[8 + i] = c, np.nextafter(c, np.float32(0))
            x[17 + i], x[24 + i] = np.nextafter(c, np.float32(np.inf)), -c
        rows.append(x)
    x = np.stack(rows)
    codes, _ = uq.quantize_mx(torch.from_numpy(x).to(DEV), "NVFP4", tscale=tscale)
    oc, _ = omx.quantize(x, "NVFP4", tscale)
    assert np.array_equal(codes.cpu().numpy(), omx.pack_codes(oc))


def test_quantize_strided_rows():
    big = _x(9, 20, 1024).to(DEV)
    part = big[3:17:2, 64:576]                                                      # row stride 2048, offset 64
    a, b = uq.quantize_mx(part, "MXFP4"), uq.quantize_mx(part.contiguous(), "MXFP4")
    assert torch.equal(a[0], b[0])
    assert torch.equal(uq.dequant_mx(a, "MXFP4"), uq.dequant_mx(b, "MXFP4"))


def _routes(seed, T, k, E, drop=0.15, empty=()):
    g = np.random.default_rng([seed, 13])
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    ids[np.isin(ids, empty)] = -1
    ids[g.random(ids.shape) < drop] = -1
    return ids


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,K", [(1, 1, 1, 64), (7, 2, 4, 96), (300, 3, 5, 288), (64, 8, 64, 512)])
def test_quantize_gathered_by_expert(fmt, T, k, E, K):
    x = _x(T, T, K)
    order, pos, off = omoe.sort(_routes(T, T, k, E), E)
    q = uq.quantize_mx(x.to(DEV), fmt, offsets=torch.from_numpy(off).to(DEV), pos=torch.from_numpy(pos).to(DEV))
    v = uq.dequant_mx(q, fmt, offsets=torch.from_numpy(off).to(DEV), dtype=torch.float32).cpu().numpy()
    ref = omoe.gather(omx.values(*omx.quantize(_np(x), fmt), fmt), pos)
    assert np.array_equal(v.astype(np.float64), ref)
    # rows already sorted: the same operand
    xs = torch.from_numpy(omoe.gather(_np(x).astype(np.float64), pos).astype(np.float32)).to(torch.bfloat16).to(DEV)
    q2 = uq.quantize_mx(xs, fmt, offsets=torch.from_numpy(off).to(DEV))
    n = int(off[-1])
    assert torch.equal(q2[0][:n], q[0][:n])
    assert np.array_equal(uq.dequant_mx(q2, fmt, offsets=torch.from_numpy(off).to(DEV), dtype=torch.float32).cpu().numpy(), v)


@pytest.mark.parametrize("fmt", FMTS)
def test_pack_mx_scales(fmt):
    for E, N, K in ((1, 1, 32), (3, 130, 160), (2, 256, 1024)):
        nat = np.random.default_rng(N).integers(0, 120, (E, N, K // omx.BLOCK[fmt])).astype(np.uint8)
        got = uq.pack_mx_scales(torch.from_numpy(nat).to(DEV), fmt).cpu().numpy()
        for e in range(E):
            assert np.array_equal(got[e], omx.tile_scales(nat[e], fmt))


# (M, N, K): one row to several token tiles, odd N, K of one block, K that ends inside a step, split k
SHAPES = [(1, 128, 32), (1, 1, 256), (3, 200, 96), (17, 384, 1056), (32, 130, 320), (33, 257, 512), (64, 1024, 4096),
          (65, 512, 2080), (100, 136, 14336), (129, 640, 1024), (300, 1000, 544), (520, 2320, 256),
          (1100, 4100, 544), (2049, 2304, 96), (1000, 8100, 4128),
          (16, 1024, 8224), (200, 900, 9248), (500, 4000, 800), (256, 2304, 1056)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_parity(fmt, M, N, K):
    w = np.random.default_rng([M, N]).normal(size=(N, K)).astype(np.float32) * 0.02
    wq, wv = _operand(w, fmt)
    x = _x(M + N, M, K)
    xv = omx.values(*omx.quantize(_np(x), fmt), fmt)
    ref, bound = omx.product(xv, wv)
    for out in ("bf16", "fp16", "fp32"):
        y = uq.gemm_mx(x.to(DEV), wq, fmt, dtype=DTYPE[out])
        r = omx.error_ratio(_np(y).astype(np.float64), ref, bound, K, out)
        assert r.max() <= 1.0, f"{out}: max error ratio {r.max():.3g}"
    y2 = uq.gemm_mx(uq.quantize_mx(x.to(DEV), fmt), wq, fmt, dtype=torch.float32)     # x quantized before
    assert torch.equal(y, y2)
    assert torch.equal(y, uq.gemm_mx(x.to(DEV), wq, fmt, dtype=torch.float32))        # the same bits again
    assert uq.device_fault() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 20000, 544), (2, 20000, 1056), (2, 130, 14336), (1, 19, 32), (3, 20000, 544)])
def test_product_of_few_tokens_quantizes_the_same_in_one_launch(fmt, dtype, M, N, K):
    """Up to three tokens are quantized inside the product's kernel: the same bits as quantized before, for every type,
    strided rows, several tiles a CTA, K that ends inside a step, and a k split."""
    rng = np.random.default_rng([M, N, K])
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2), dtype=np.uint8)).to(DEV)
    byte = rng.integers(110, 130, (N, K // omx.BLOCK[fmt])).astype(np.uint8) if fmt == "MXFP4" else \
        rng.integers(0x08, 0x60, (N, K // omx.BLOCK[fmt])).astype(np.uint8)
    w = (codes, torch.from_numpy(omx.tile_scales(byte, fmt)).to(DEV))
    x = _x(M + K, 2 * M, K + 64, dtype).to(DEV)[::2, 32:32 + K]
    t = 1.0 if fmt == "MXFP4" else 0.5
    y = uq.gemm_mx(x, w, fmt, tscale=t, dtype=torch.float32)
    z = uq.gemm_mx(uq.quantize_mx(x, fmt, tscale=t), w, fmt, alpha=t, dtype=torch.float32)
    assert torch.equal(y, z) and uq.device_fault() == 0


def test_product_scales_strides_and_empty():
    N, K = 192, 512
    w = np.random.default_rng(2).normal(size=(N, K)).astype(np.float32)
    wq, wv = _operand(w, "NVFP4", 0.5)
    x = _x(3, 40, 1024, "fp16").to(DEV)[::2, 256:768]
    xv = omx.values(*omx.quantize(_np(x), "NVFP4", 0.125), "NVFP4", 0.125)
    ref, bound = omx.product(xv, wv)
    y = uq.gemm_mx(x, wq, "NVFP4", tscale=0.125, alpha=0.5)                          # the weight's tensor scale as alpha
    assert y.dtype == torch.float16
    assert omx.error_ratio(_np(y).astype(np.float64), ref, bound, K, "fp16").max() <= 1.0
    assert uq.gemm_mx(x[:0], wq, "NVFP4").shape == (0, N)
    e = torch.empty((4, 0), dtype=torch.bfloat16, device=DEV)
    z = uq.gemm_mx(e, (torch.empty((N, 0), dtype=torch.uint8, device=DEV), torch.empty(0, dtype=torch.uint8, device=DEV)), "MXFP4")
    assert z.shape == (4, N) and not z.any()


def test_product_nan_block_stays_in_its_row():
    wq, _ = _operand(np.ones((130, 128), np.float32), "MXFP4")
    x = torch.ones(5, 128, dtype=torch.bfloat16)
    x[2, 70] = float("inf")
    y = uq.gemm_mx(x.to(DEV), wq, "MXFP4")
    assert torch.isnan(y[2]).all() and torch.equal(y[[0, 1, 3, 4]], torch.full((4, 130), 128.0, dtype=torch.bfloat16, device=DEV))


# T, k, E, N, K, empty experts
GROUPS = [(1, 1, 1, 128, 64, ()), (3, 2, 8, 640, 1024, ()), (5, 4, 16, 200, 288, (3, 15)), (70, 2, 4, 257, 544, (0,)),
          (333, 4, 40, 136, 512, (7, 8, 9)), (400, 2, 3, 384, 1024, ()), (9, 2, 2, 128, 4096, (0, 1)),
          (1500, 2, 5, 4100, 288, (2,)), (1100, 1, 3, 4352, 544, ()), (1500, 1, 2, 4351, 288, ()),
          (7, 2, 4, 200, 8224, (1,)), (150, 1, 2, 130, 6176, ()), (800, 1, 8, 300, 544, ())]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,N,K,empty", GROUPS)
def test_grouped_parity(fmt, T, k, E, N, K, empty, gated):
    rng = np.random.default_rng([T, E, N])
    x = _x(T + E, T, K)
    order, pos, off = omoe.sort(_routes(T + E, T, k, E, empty=empty), E)
    offd = torch.from_numpy(off).to(DEV)
    q = uq.quantize_mx(x.to(DEV), fmt, offsets=offd, pos=torch.from_numpy(pos).to(DEV))
    xv = omoe.gather(omx.values(*omx.quantize(_np(x), fmt), fmt), pos)

    def weight():
        parts = [_operand(rng.normal(size=(N, K)).astype(np.float32) * 0.05, fmt) for _ in range(E)]
        return (torch.stack([p[0][0] for p in parts]), torch.stack([p[0][1] for p in parts])), [p[1] for p in parts]

    wq, wv = weight()
    alpha = rng.uniform(0.5, 2.0, E).astype(np.float32)
    up, upv, alpha_up = None, None, None
    if gated:
        up, upv = weight()
        alpha_up = rng.uniform(0.5, 2.0, E).astype(np.float32)
    dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)               # noqa: E731
    y = uq.gemm_mx_grouped(q, wq, offd, fmt, up=up, alpha=dev(alpha), alpha_up=dev(alpha_up), dtype=torch.float32)
    ref, tol = np.zeros((T * k, N)), np.full((T * k, N), 2.0 ** -25)
    acc = K * 2.0 ** -23
    for e in range(E):
        s = slice(off[e], off[e + 1])
        g, bg = omx.product(xv[s], wv[e])
        g, bg = g * float(alpha[e]), (bg * acc + 2.0 ** -23 * np.abs(g)) * float(alpha[e])
        if not gated:
            ref[s], tol[s] = g, tol[s] + bg + 2.0 ** -23 * np.abs(g)
            continue
        u, bu = omx.product(xv[s], upv[e])
        u, bu = u * float(alpha_up[e]), (bu * acc + 2.0 ** -23 * np.abs(u)) * float(alpha_up[e])
        silu = g / (1 + np.exp(-g))
        ref[s] = silu * u
        tol[s] += 1.1 * bg * np.abs(u) + np.abs(silu) * bu + 1.1 * bg * bu + 2.0 ** -20 * np.abs(ref[s])
    got = _np(y).astype(np.float64)
    assert np.all(np.abs(got - ref) <= tol), f"max ratio {np.max(np.abs(got - ref) / tol):.3g}"
    n = int(off[-1])
    assert not got[n:].any()                                                         # rows that belong to nobody
    y16 = uq.gemm_mx_grouped(q, wq, offd, fmt, up=up, alpha=dev(alpha), alpha_up=dev(alpha_up))
    assert np.all(np.abs(_np(y16) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))
    assert torch.equal(y, uq.gemm_mx_grouped(q, wq, offd, fmt, up=up, alpha=dev(alpha), alpha_up=dev(alpha_up), dtype=torch.float32))
    assert uq.device_fault() == 0


def test_grouped_rows_equal_the_dense_product_of_each_expert():
    """One expert with all rows: the grouped call and the dense one form the same sums."""
    wq, _ = _operand(np.random.default_rng(4).normal(size=(256, 512)).astype(np.float32), "MXFP4")
    x = _x(8, 50, 512).to(DEV)
    off = torch.tensor([0, 50], dtype=torch.int32, device=DEV)
    q = uq.quantize_mx(x, "MXFP4", offsets=off)
    y = uq.gemm_mx_grouped(q, (wq[0][None], wq[1][None]), off, "MXFP4", dtype=torch.float32)
    d = uq.gemm_mx(x, wq, "MXFP4", dtype=torch.float32)
    assert torch.allclose(y, d, rtol=2.0 ** -14, atol=2.0 ** -14 * float(d.abs().max()))


def test_product_on_another_stream_and_in_a_graph():
    wq, wv = _operand(np.random.default_rng(6).normal(size=(320, 1024)).astype(np.float32), "NVFP4")
    x = _x(10, 6, 1024).to(DEV)
    want = uq.gemm_mx(x, wq, "NVFP4")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = uq.gemm_mx(x, wq, "NVFP4")                                               # this stream's workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            uq.gemm_mx(x, wq, "NVFP4", y=y)
        y.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_operands_past_32_bit_offsets():
    """2.3e9 elements (codes past 2^30 bytes, values past 2^32): the last rows equal those of a small call.  Small
    integers, so every sum is exact whatever the kernel and its order."""
    T, K, N, n = 70001, 32768, 128, 37
    x = torch.randint(-1, 2, (T, K), device=DEV, dtype=torch.int8).to(torch.bfloat16)
    w = torch.randint(-1, 2, (N, K), device=DEV, dtype=torch.int8).to(torch.bfloat16)
    wq = uq.quantize_mx(w, "MXFP4")
    q = uq.quantize_mx(x, "MXFP4")
    tail = x[-n:].contiguous()
    qt = uq.quantize_mx(tail, "MXFP4")
    assert torch.equal(q[0][-n:], qt[0])
    assert torch.equal(uq.dequant_mx(q, "MXFP4")[-n:], tail)
    y = uq.gemm_mx(q, wq, "MXFP4", dtype=torch.float32)
    assert torch.equal(y[-n:], tail.float() @ w.float().t())
    off = torch.tensor([0, T - n, T], dtype=torch.int32, device=DEV)
    qs = uq.quantize_mx(x, "MXFP4", offsets=off)
    ys = uq.gemm_mx_grouped(qs, (wq[0].repeat(2, 1, 1), wq[1].repeat(2, 1)), off, "MXFP4", dtype=torch.float32)
    assert torch.equal(ys, y)
    assert uq.device_fault() == 0


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    w = (torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.zeros(512, dtype=torch.uint8, device=DEV))

    def status(f):
        with pytest.raises(uq.UqError) as e:
            f()
        return e.value.status

    assert status(lambda: uq.quantize_mx(x[:, :48].contiguous(), "MXFP4")) == 1                # K % 32
    assert status(lambda: uq.quantize_mx(x, "MXFP4", tscale=2.0)) == 1                         # MXFP4 has none
    assert status(lambda: uq.quantize_mx(x, "NVFP4", tscale=0.0)) == 1
    assert status(lambda: uq.quantize_mx(x, "NVFP4", tscale=float("nan"))) == 1
    assert status(lambda: uq.quantize_mx(x, "MXFP4", pos=torch.zeros(4, 2, dtype=torch.int32, device=DEV))) == 1
    flat = torch.zeros(4 * 72 + 8, dtype=torch.bfloat16, device=DEV)
    assert status(lambda: uq.quantize_mx(flat[1:1 + 4 * 64].view(4, 64), "MXFP4")) == 3         # misaligned base
    assert status(lambda: uq.quantize_mx(flat[:4 * 68].view(4, 68)[:, :64], "MXFP4")) == 3      # misaligned rows
    assert status(lambda: uq.gemm_mx(x, w, "NVFP4", tscale=-1.0)) == 1
    assert status(lambda: uq.gemm_mx(flat[:4 * 68].view(4, 68)[:, :64], w, "MXFP4")) == 3
    with pytest.raises(AssertionError):
        uq.gemm_mx(x[:, :32].contiguous(), w, "MXFP4")                                          # K differs
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    q = uq.quantize_mx(x, "MXFP4", offsets=off)
    wg = (w[0][None], w[1][None])
    with pytest.raises(AssertionError):
        uq.gemm_mx_grouped(q, wg, off[:1], "MXFP4")                                             # offsets per expert
    a = torch.ones(1, device=DEV)
    assert status(lambda: uq.gemm_mx_grouped(q, wg, off, "MXFP4", alpha_up=a)) == 1             # no up weight
