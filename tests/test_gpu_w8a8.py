"""uq_gemm_w8a8 on the GPU against the oracle.

Tolerance: every 1024 k are summed exactly; their sums are added in fp32 (one rounding each, of at most the parts' summed
magnitudes), then the integer's rounding, two products and the rounding to the type: (K / 1024 + 4) u of the magnitudes and
half a step."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import q8 as oq  # noqa: E402

DEV = torch.device("cuda:0")
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}
U = 2.0 ** -24


def n(t):
    return t.double().cpu().numpy()


def _operand(seed, rows, K, kind="random"):
    g = np.random.default_rng([seed, rows, K])
    if kind == "largest":
        q = g.choice(np.array([-128, 127], np.int8), (rows, 1)) * np.ones((1, K), np.int8)
    else:
        q = np.clip(np.rint(g.normal(size=(rows, K)) * 40), -128, 127)
    s = np.exp(g.normal(size=rows)).astype(np.float32) * 0.01
    return torch.from_numpy(q.astype(np.int8)).to(DEV), torch.from_numpy(s).to(DEV)


def _check(y, x, w, dtype):
    ref, mag = oq.gemm(x[0].cpu().numpy(), x[1].cpu().numpy(), w[0].cpu().numpy(), w[1].cpu().numpy())
    K = x[0].shape[1]
    tol = ROUND[dtype] * np.abs(ref) * 1.0001 + (K / 1024 + 4) * U * mag + TINY[dtype]
    bad = np.abs(n(y) - ref) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, first at {np.argwhere(bad)[0]}"


SHAPES = [(1, 1, 16), (1, 33, 48), (2, 128, 1024), (7, 100, 2064), (8, 31, 64), (9, 257, 512), (16, 129, 1040), (17, 64, 4096),
          (33, 640, 2048), (64, 300, 160), (65, 384, 1536), (128, 128, 128), (129, 513, 272), (200, 130, 2304), (256, 256, 1024),
          (300, 1000, 528), (513, 257, 3088), (700, 96, 4112), (1000, 1100, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_codes(M, N, K, dtype):
    x, w = _operand(1, M, K), _operand(2, N, K)
    y = uq.gemm_w8a8(x, w, dtype=DTYPE[dtype])
    _check(y, x, w, dtype)
    assert torch.equal(y, uq.gemm_w8a8(x, w, dtype=DTYPE[dtype]))
    assert uq.device_fault() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(1, 96, 1024), (3, 1000, 4096), (8, 64, 16), (20, 200, 2064), (150, 257, 1040), (600, 512, 512)])
def test_rows_quantized_in_the_call(M, N, K, dtype):
    """The call with rows is quantize_q8 followed by the call with codes, bit for bit; strided rows too."""
    g = np.random.default_rng([M, K])
    x = torch.from_numpy(g.normal(size=(M, K + 8))).to(DTYPE[dtype]).to(DEV)[:, :K]
    w = _operand(2, N, K)
    y = uq.gemm_w8a8(x, w)
    assert y.dtype == DTYPE[dtype]
    q = uq.quantize_q8(x)
    assert torch.equal(y, uq.gemm_w8a8(q, w, dtype=DTYPE[dtype]))
    _check(y, q, w, dtype)


@pytest.mark.parametrize("M", [1, 5, 12, 40, 300])
@pytest.mark.parametrize("K", [1024, 4096, 14336])
def test_the_largest_sums(M, K):
    """All codes at the ends of their range: the sums pass 2^24 and stay exact to the tolerance."""
    x, w = _operand(1, M, K, "largest"), _operand(2, 200, K, "largest")
    _check(uq.gemm_w8a8(x, w, dtype=torch.float32), x, w, "fp32")


@pytest.mark.parametrize("M,N", [(1, 256), (24, 256), (200, 256), (520, 512)])
def test_small_integers_are_exact(M, N):
    """Sums below 2^24 with scales of one come back as they are."""
    K = 8192
    g = np.random.default_rng(7)
    x, w = (torch.from_numpy(g.integers(-30, 31, (r, K)).astype(np.int8)).to(DEV) for r in (M, N))
    one = lambda r: torch.ones(r, device=DEV)                                        # noqa: E731
    y = uq.gemm_w8a8((x, one(M)), (w, one(N)), dtype=torch.float32)
    assert np.array_equal(n(y), x.cpu().numpy().astype(np.float64) @ w.cpu().numpy().astype(np.float64).T)


def test_nan_and_zero_rows():
    K, N = 512, 160
    for M in (6, 70):
        x = torch.randn(M, K, device=DEV)
        x[1], x[2, 3], x[4, 5] = 0, float("nan"), float("inf")
        w = _operand(2, N, K)
        y = uq.gemm_w8a8(x, w)
        assert torch.isnan(y[[2, 4]]).all() and not y[1].any() and torch.isfinite(y[[0, 3, 5]]).all()


def test_nothing_to_do():
    w = _operand(2, 64, 256)
    assert uq.gemm_w8a8(torch.empty(0, 256, device=DEV), w).shape == (0, 64)
    assert uq.gemm_w8a8(torch.randn(5, 256, device=DEV), (w[0][:0], w[1][:0])).shape == (5, 0)
    none = torch.zeros(5, 0, dtype=torch.int8, device=DEV), torch.ones(5, device=DEV)
    y = torch.full((5, 64), 7.0, device=DEV)
    assert not uq.gemm_w8a8(none, (w[0][:, :0].contiguous(), w[1]), y=y).any()


def test_rows_behind_y_are_left():
    for M, N in ((3, 100), (50, 130), (300, 258)):
        x, w = _operand(1, M, 512), _operand(2, N, 512)
        whole = torch.full((M + 2, N), 3.0, device=DEV)
        uq.gemm_w8a8(x, w, y=whole[:M])
        assert (whole[M:] == 3.0).all()
        _check(whole[:M], x, w, "fp32")


def test_streams_and_graphs():
    """Two streams at once have workspaces of their own; two graphs of one stream share its."""
    K, N = 2048, 512
    w = _operand(2, N, K)
    xs = [torch.randn(m, K, device=DEV).bfloat16() for m in (4, 90, 400)]
    want = [uq.gemm_w8a8(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(4):
        got = [uq.gemm_w8a8(x, w, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s, graphs, outs = streams[0], [], []
    uq.gemm_w8a8(xs[2], w, stream=s)
    with torch.cuda.stream(s):
        for x in xs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(uq.gemm_w8a8(x, w))
            graphs.append(g)
        for o in outs:
            o.zero_()
        for _ in range(2):
            for g in graphs:
                g.replay()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert uq.device_fault() == 0


@pytest.mark.parametrize("M,N,K", [(2560, 2048, 128), (2500, 2100, 1184), (2305, 2304, 2048), (2560, 2304, 4112), (4100, 1300, 640),
                                   (1024, 4096, 128), (1000, 4100, 1184), (2305, 1792, 2048), (2000, 2304, 4112), (4100, 1000, 640),
                                   (2300, 3900, 1296), (2100, 4097, 3088)])
def test_pairs_of_ctas(M, N, K):
    """Enough tiles of 256 x 256 for a pair of CTAs on every two SMs, ragged ends, chunks of all lengths; against integer sums
    in 64 bits on the device."""
    for kind in ("random", "largest"):
        x, w = _operand(1, M, K, kind), _operand(2, N, K)
        y = uq.gemm_w8a8(x, w, dtype=torch.float32)
        a, b = x[0].double() * x[1].double()[:, None], w[0].double() * w[1].double()[:, None]
        mag = sum((a[:, k:k + 1024] @ b[:, k:k + 1024].t()).abs() for k in range(0, K, 1024))
        bad = (y.double() - a @ b.t()).abs() > (K / 1024 + 4) * U * mag + 2.0 ** -149 + (a.abs() @ b.abs().t()) * 2.0 ** -50
        assert not bool(bad.any()), f"{int(bad.sum())} outputs off, first at {bad.nonzero()[0].tolist()}"
        y16 = uq.gemm_w8a8(x, w)
        assert torch.equal(y16, y.bfloat16())
    assert uq.device_fault() == 0


@pytest.mark.parametrize("M,N,K", [(70000, 32768, 64), (3, 70000, 32768), (40, 70000, 32768)])
def test_offsets_past_32_bits(M, N, K):
    """Over 2^31 outputs, or weights: the ends against integer sums of those rows and columns."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=DEV, generator=g)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV, generator=g)
    sx, sw = torch.rand(M, device=DEV, generator=g), torch.rand(N, device=DEV, generator=g)
    y = uq.gemm_w8a8((x, sx), (w, sw))
    for rows, cols in ((slice(-9, None), slice(-300, None)), (slice(0, 9), slice(0, 300))):
        _check(y[rows, cols], (x[rows].contiguous(), sx[rows]), (w[cols].contiguous(), sw[cols]), "bf16")
    assert uq.device_fault() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(1, 96, 4096), (8, 512, 4096), (20, 128, 4096), (20, 20000, 1024), (50, 200, 4096), (50, 20000, 1024),
                                   (100, 257, 4096), (100, 20000, 1024), (2500, 2100, 1184)])
def test_scales_whose_product_leaves_fp32(M, N, K, dtype):
    """Scales that together are below fp32's smallest number while the outputs are not, in each form of the product: single
    tokens, tiles that share k, whole tiles, pairs.  Rounded as ever: each factor once."""
    x, w = _operand(1, M, K, "largest"), _operand(2, N, K, "largest")
    x, w = ((q, (1 + torch.rand(len(q), device=DEV)) * 2.0 ** -73) for q, _ in (x, w))
    y = uq.gemm_w8a8(x, w, dtype=DTYPE[dtype])
    a, b = x[0].double() * x[1].double()[:, None], w[0].double() * w[1].double()[:, None]
    want = a @ b.t()
    assert float(want.abs().min()) > 2.0 ** -126
    mag = sum((a[:, k:k + 1024] @ b[:, k:k + 1024].t()).abs() for k in range(0, K, 1024))
    tol = ROUND[dtype] * want.abs() * 1.0001 + (K / 1024 + 4) * U * mag + (a.abs() @ b.abs().t()) * 2.0 ** -50
    bad = (y.double() - want).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outputs off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("M,N,K", [(1000, 4100, 2832), (2040, 4090, 2944), (2305, 1792, 3088), (2000, 2304, 3216), (2300, 3900, 3344),
                                   (4600, 4090, 2832), (1024, 4096, 1024), (8192, 2304, 512)])
def test_pairs_of_ctas_and_the_sizes_that_leave_them(M, N, K):
    """Tiles that pairs take, with ragged ends and chunks of several lengths, and some that they leave for their few k."""
    for kind in ("random", "largest"):
        x, w = _operand(3, M, K, kind), _operand(4, N, K)
        y = uq.gemm_w8a8(x, w, dtype=torch.float32)
        a, b = x[0].double() * x[1].double()[:, None], w[0].double() * w[1].double()[:, None]
        mag = sum((a[:, k:k + 512] @ b[:, k:k + 512].t()).abs() for k in range(0, K, 512))
        bad = (y.double() - a @ b.t()).abs() > (K / 512 + 4) * U * mag + 2.0 ** -149 + (a.abs() @ b.abs().t()) * 2.0 ** -50
        assert not bool(bad.any()), f"{int(bad.sum())} outputs off, first at {bad.nonzero()[0].tolist()}"
        for dtype in ("bf16", "fp16"):
            assert torch.equal(uq.gemm_w8a8(x, w, dtype=DTYPE[dtype]), y.to(DTYPE[dtype]))
    assert uq.device_fault() == 0
