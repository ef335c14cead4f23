"""Rows in 8 bits, the norm that ends in them and its gradient, on the GPU against the oracle.

Tolerances.  u = 2^-24.  A sum of D terms: a thread adds at most ceil(D / 32) in sequence, then at most 12 levels of a tree:
S = D / 32 + 16 roundings.  r = 1 / sqrt(...) loses half of the sum's relative error and three roundings.  Codes are the
nearest integers of quotients <= 127 that lose four roundings.  A rounding to the type is at most half a step."""
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
SIZES = [(1, 1), (1, 16), (3, 31), (2, 100), (5, 257), (129, 64), (33, 1001), (7, 4096), (300, 1026), (2, 8200), (3, 16384),
         (2, 33001), (1, 40000)]


def n(t):
    return t.double().cpu().numpy()


def _rows(seed, T, D, dtype):
    g = np.random.default_rng([seed, T, D])
    x = g.normal(size=(T, D)) * np.exp(g.normal(size=(T, 1)))
    x[g.random((T, D)) < 0.003] *= 20
    if T > 2:
        x[1] = 0
    return torch.from_numpy(x).to(DTYPE[dtype]).to(DEV)


def f32(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_quantize_equals_the_definition(T, D, dtype):
    x = _rows(1, T, D, dtype)
    codes, scales = uq.quantize_q8(x)
    rq, rs = oq.quantize(f32(x))
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rq)
    for out in DTYPE.values():
        got = uq.dequant_q8((codes, scales), dtype=out)
        assert torch.equal(got, (codes.float() * scales[:, None]).to(out))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,ld", [(64, 80), (64, 66), (64, 65), (100, 200), (33, 64)])
def test_strided_rows(D, ld, dtype):
    whole = _rows(2, 9, ld, dtype)
    x = whole[:, :D]
    assert all(torch.equal(a, b) for a, b in zip(uq.quantize_q8(x), uq.quantize_q8(x.contiguous())))
    gamma = _rows(3, 1, D, dtype)[0]
    # (another stride may be read in other accesses, whose squares are added in another order: not bit for bit)
    h, y, q = uq.rmsnorm_q8(x, gamma, 1e-5, normed=True)
    assert h is x
    _check_norm(x, gamma, 1e-5, y, q, dtype)


def test_quantize_extremes():
    """Scales at both ends of fp32, ties, infinities and NaN; the definition's values throughout."""
    big, small = 3.4e38, 1e-45
    rows = [[big, -big, big / 2, 1e30], [small, -small, 0, small * 3], [1e-38, 3e-39, -2e-39, 1e-40], [0, -0.0, 0, 0],
            [np.nan, 1, 2, 3], [np.inf, 1, 2, 3], [-np.inf, np.nan, 0, 0], [127, 0.5, 1.5, -2.5], [2.0 ** -100, 2.0 ** -101, 2.0 ** -107, 0],
            [2.0 ** 100, 2.0 ** 99, 2.0 ** 93, -2.0 ** 94]]
    g = np.random.default_rng(5)
    more = np.ldexp(g.normal(size=(200, 4)), g.integers(-140, 120, (200, 1)))
    x = np.concatenate([np.array(rows, np.float32), more.astype(np.float32)])
    codes, scales = uq.quantize_q8(torch.from_numpy(x).to(DEV))
    rq, rs = oq.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), rq)
    back = uq.dequant_q8((codes, scales), dtype=torch.float32).cpu().numpy()
    assert np.isnan(back[4:7]).all() and not back[3].any()


def _check_norm(h, gamma, eps, y, q, dtype):
    D = h.shape[1]
    ref, rs = oq.rmsnorm(n(h), n(gamma), eps)
    rel = (D / 32 + 16) / 2 + 8
    if y is not None:
        assert np.all(np.abs(n(y) - ref) <= ROUND[dtype] * np.abs(ref) * 1.0001 + rel * U * np.abs(ref) + TINY[dtype])
    if q is not None:
        codes, scales = n(q[0]), n(q[1])
        assert np.all(np.abs(scales - rs) <= rel * U * rs + 2.0 ** -149)
        on = rs > 0
        assert np.all(np.abs(codes[on] - ref[on] / rs[on, None]) <= 0.5 + 127 * 8 * U)
        assert not codes[~on].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_norm(T, D, dtype):
    x, r, gamma = _rows(1, T, D, dtype), _rows(2, T, D, dtype), _rows(3, 1, D, dtype)[0]
    for residual in (None, r):
        h, y, q = uq.rmsnorm_q8(x, gamma, 1e-5, residual=residual, normed=True)
        want = x if residual is None else (x.float() + r.float()).to(x.dtype)
        assert torch.equal(h, want)
        _check_norm(want, gamma, 1e-5, y, q, dtype)
        # each output alone
        only = uq.rmsnorm_q8(x, gamma, 1e-5, residual=residual, normed=True, quantized=False)
        assert only[2] is None and torch.equal(only[1], y)
        only = uq.rmsnorm_q8(x, gamma, 1e-5, residual=residual)
        assert only[1] is None and torch.equal(only[2][0], q[0]) and torch.equal(only[2][1], q[1])
    # the fused call is the norm of the stored sum
    again = uq.rmsnorm_q8(h, gamma, 1e-5, normed=True)
    assert torch.equal(again[1], y) and torch.equal(again[2][0], q[0])


@pytest.mark.parametrize("T,D", [(5, 100), (3, 4096), (2, 33000)])
def test_norm_in_place(T, D):
    x, r, gamma = (_rows(i, T, D, "bf16") for i in (1, 2, 3))
    gamma = gamma[0].contiguous()
    h, y, q = uq.rmsnorm_q8(x, gamma, 1e-6, residual=r, normed=True)
    for over in (0, 1):
        a = [x.clone(), r.clone()]
        got = uq.rmsnorm_q8(a[0], gamma, 1e-6, residual=a[1], normed=True, h=a[over])
        assert got[0] is a[over] and torch.equal(a[over], h) and torch.equal(got[1], y) and torch.equal(got[2][0], q[0])
        assert torch.equal(a[1 - over], (x, r)[1 - over])


def test_norm_extremes():
    """Rows of zeros, of the smallest values, and with an infinity or a NaN: NaN scale and codes 0 for those alone."""
    D = 96
    x = torch.zeros(8, D, device=DEV)
    x[1] = 1e-30
    x[2, 5] = 1e-44
    x[3] = 1e15
    x[4, 7] = float("nan")
    x[5, 7] = float("inf")
    x[6] = torch.linspace(-1, 1, D, device=DEV)
    gamma = torch.linspace(0.5, 1.5, D, device=DEV)
    for eps in (1e-5, 1e-30):
        _, y, (codes, scales) = uq.rmsnorm_q8(x, gamma, eps, normed=True)
        keep = [0, 1, 3, 6, 7]
        _check_norm(x[keep], gamma, eps, y[keep], (codes[keep], scales[keep]), "fp32")
        assert torch.isnan(scales[4:6]).all() and not codes[4:6].any()
        assert torch.isfinite(scales[[0, 1, 2, 3, 6, 7]]).all()
        assert torch.isnan(y[4]).all() and torch.isnan(y[5]).any()
    gamma[3] = float("nan")
    _, y, (codes, scales) = uq.rmsnorm_q8(x[6:7], gamma, 1e-5, normed=True)
    assert torch.isnan(scales).all() and not codes.any() and int(torch.isnan(y).sum()) == 1


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,D", SIZES + [(700, 96), (2000, 40), (1300, 513)])
def test_norm_gradient(T, D, dtype, with_dh):
    h, dy, gamma, dh = _rows(1, T, D, dtype), _rows(2, T, D, dtype), _rows(3, 1, D, dtype)[0], _rows(4, T, D, dtype)
    eps = 1e-2
    dx, dgamma = uq.rmsnorm_grad(dy, h, gamma, eps, dh=dh if with_dh else None)
    rx, rg = oq.rmsnorm_grad(n(dy), n(h), n(gamma), eps, n(dh) if with_dh else None)
    H, G = n(h), n(dy) * n(gamma)
    r = 1 / np.sqrt((H * H).mean(axis=1, keepdims=True) + eps)
    mag = r * (np.abs(G) + np.abs(H) * r * r * np.abs(G * H).mean(axis=1, keepdims=True)) + (np.abs(n(dh)) if with_dh else 0)
    steps = 3 * (D / 32 + 16) + 16
    assert np.all(np.abs(n(dx) - rx) <= ROUND[dtype] * np.abs(rx) * 1.0001 + steps * U * mag + TINY[dtype])
    assert np.all(np.abs(n(dgamma) - rg) <= (T + steps) * U * np.abs(n(dy) * H * r).sum(axis=0) + 2.0 ** -140)
    again = uq.rmsnorm_grad(dy, h, gamma, eps, dh=dh if with_dh else None)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dgamma)


def test_nothing_to_do():
    e = torch.empty(0, 64, device=DEV)
    gamma = torch.ones(64, device=DEV)
    codes, scales = uq.quantize_q8(e)
    assert codes.shape == (0, 64) and scales.shape == (0,)
    dx, dgamma = uq.rmsnorm_grad(e, e, gamma, 1e-5)
    assert dx.shape == (0, 64) and not dgamma.any()
    assert uq.dequant_q8((codes, scales)).shape == (0, 64)
    codes, scales = uq.quantize_q8(torch.empty(5, 0, device=DEV))
    assert codes.shape == (5, 0) and not scales.any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,D", [(1, 5), (306, 3), (1000, 9), (400, 127), (2500, 1001), (3, 4099), (700, 4097), (320, 9001), (2, 16379)])
def test_rows_that_begin_anywhere(T, D, dtype):
    """Rows that are not whole 16-byte parts, many of them too: in place, beside a row of NaN, and nothing behind the last one."""
    n_, pad, code = T * D, 64, uq.DTYPES[DTYPE[dtype]]
    x, r, gamma = _rows(1, T, D, dtype), _rows(2, T, D, dtype), _rows(3, 1, D, dtype)[0].contiguous()
    if T > 5:
        x[4] = float("nan")
    h = (x.float() + r.float()).to(x.dtype)
    keep = [i for i in range(T) if i != 4 or T <= 5]
    buf = lambda t: torch.full((n_ + pad,), 77, dtype=t, device=DEV)                # noqa: E731
    hx, y, codes, scales = buf(x.dtype), buf(x.dtype), buf(torch.int8), torch.full((T + pad,), 77.0, device=DEV)
    hx[:n_] = x.reshape(-1)
    assert uq.lib().uq_rmsnorm_q8(hx.data_ptr(), r.data_ptr(), gamma.data_ptr(), code, D, hx.data_ptr(), y.data_ptr(),
                                  codes.data_ptr(), scales.data_ptr(), T, D, 1e-5, None) == 0
    got = hx[:n_].view(T, D)
    assert torch.equal(got[keep], h[keep])
    _check_norm(h[keep], gamma, 1e-5, y[:n_].view(T, D)[keep], (codes[:n_].view(T, D)[keep], scales[:T][keep]), dtype)
    if T > 5:
        assert torch.isnan(got[4]).all() and torch.isnan(y[:n_].view(T, D)[4]).all()
        assert torch.isnan(scales[4]) and not codes[:n_].view(T, D)[4].any()
    for t, m in ((hx, n_), (y, n_), (codes, n_), (scales, T)):
        assert (t[m:] == 77).all()
    q = buf(torch.int8)
    s2, back = torch.full((T + pad,), 77.0, device=DEV), buf(torch.bfloat16)
    assert uq.lib().uq_quantize_q8(h.data_ptr(), code, D, q.data_ptr(), s2.data_ptr(), T, D, None) == 0
    assert uq.lib().uq_dequant_q8(q.data_ptr(), s2.data_ptr(), back.data_ptr(), uq.DTYPES[torch.bfloat16], T, D, None) == 0
    rq, rs = oq.quantize(f32(h))
    assert np.array_equal(q[:n_].view(T, D).cpu().numpy(), rq) and np.array_equal(s2[:T].cpu().numpy(), rs, equal_nan=True)
    want = (q[:n_].view(T, D).float() * s2[:T, None]).to(torch.bfloat16)
    assert torch.equal(back[:n_].view(T, D).isnan(), want.isnan()) and torch.equal(back[:n_].view(T, D).nan_to_num(), want.nan_to_num())
    for t, m in ((q, n_), (back, n_), (s2, T)):
        assert (t[m:] == 77).all()
    # the gradient, over dy; a row of NaN reaches its own dx alone
    dy, hh = buf(x.dtype), h.clone()
    dy[:n_] = r.reshape(-1)
    dgamma = torch.full((D + pad,), 77.0, device=DEV)
    assert uq.lib().uq_rmsnorm_grad(dy.data_ptr(), hh.data_ptr(), gamma.data_ptr(), None, code, dy.data_ptr(), dgamma.data_ptr(),
                                    T, D, 1e-2, None) == 0
    rx, rg = oq.rmsnorm_grad(n(r[keep]), n(h[keep]), n(gamma), 1e-2, None)
    H, G = n(h[keep]), n(r[keep]) * n(gamma)
    rr = 1 / np.sqrt((H * H).mean(axis=1, keepdims=True) + 1e-2)
    mag = rr * (np.abs(G) + np.abs(H) * rr * rr * np.abs(G * H).mean(axis=1, keepdims=True))
    steps = 3 * (D / 32 + 16) + 16
    dx = dy[:n_].view(T, D)
    assert np.all(np.abs(n(dx[keep]) - rx) <= ROUND[dtype] * np.abs(rx) * 1.0001 + steps * U * mag + TINY[dtype])
    if T > 5:
        assert torch.isnan(dx[4]).all() and torch.isnan(dgamma[:D]).all()
    else:
        assert np.all(np.abs(n(dgamma[:D]) - rg) <= (T + steps) * U * np.abs(n(r) * H * rr).sum(axis=0) + 2.0 ** -140)
    assert (dy[n_:] == 77).all() and (dgamma[D:] == 77).all()


def test_rows_without_elements_have_scale_zero():
    e = torch.empty(5, 0, device=DEV)
    for scales in (uq.rmsnorm_q8(e, e[0], 1e-5)[2][1], uq.rmsnorm_q8(e, e[0], 1e-5, residual=e, normed=True)[2][1]):
        assert scales.shape == (5,) and not scales.any()


def test_on_another_stream_and_in_graphs():
    """Results on a given stream; two graphs captured on one stream share its workspace and are replayed one after the other."""
    T, D = 200, 2048
    h, dy, gamma = _rows(1, T, D, "bf16"), _rows(2, T, D, "bf16"), _rows(3, 1, D, "bf16")[0]
    want = uq.rmsnorm_grad(dy, h, gamma, 1e-5)
    half = uq.rmsnorm_grad(dy[:50], h[:50], gamma, 1e-5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = uq.rmsnorm_grad(dy, h, gamma, 1e-5, stream=s)
    graphs, outs = [], []
    with torch.cuda.stream(s):
        for rows in (T, 50):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(uq.rmsnorm_grad(dy[:rows], h[:rows], gamma, 1e-5) + uq.rmsnorm_q8(h[:rows], gamma, 1e-5)[2])
            graphs.append(g)
        for _ in range(3):
            for g in graphs:
                g.replay()
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q = uq.rmsnorm_q8(h, gamma, 1e-5)[2]
    for o, w, rows in ((outs[0], want, T), (outs[1], half, 50)):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
        assert torch.equal(o[2], q[0][:rows]) and torch.equal(o[3], q[1][:rows])


def test_offsets_past_32_bits():
    """Over 2^31 elements: the last rows of the quantizer, the norm, its gradient and the values."""
    T, D = 70000, 32768
    x = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    x.zero_()
    x[-3:] = _rows(1, 3, D, "bf16")
    gamma = _rows(3, 1, D, "bf16")[0].contiguous()
    tail = x[-3:].clone()
    q = uq.quantize_q8(x)
    want = uq.quantize_q8(tail)
    assert torch.equal(q[0][-3:], want[0]) and torch.equal(q[1][-3:], want[1]) and not q[0][:100].any()
    assert torch.equal(uq.dequant_q8(q)[-3:], uq.dequant_q8(want))
    h, y, q = uq.rmsnorm_q8(x, gamma, 1e-5, residual=x, normed=True)
    _check_norm((tail.float() * 2).bfloat16(), gamma, 1e-5, y[-3:], (q[0][-3:], q[1][-3:]), "bf16")
    assert torch.equal(h[-3:], (tail.float() * 2).bfloat16()) and not y[:100].any()
    del h, y, q
    dx, dgamma = uq.rmsnorm_grad(x, x, gamma, 1e-2)
    ref, rg = oq.rmsnorm_grad(n(tail), n(tail), n(gamma), 1e-2)
    assert np.all(np.abs(n(dx[-3:]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2e-3 * np.abs(ref).max())
    assert np.all(np.abs(n(dgamma) - rg) <= 1e-2 * np.abs(rg).max()) and not dx[:100].any()


def test_many_short_rows():
    """Groups of one warp and of several, more rows than the grid takes at once."""
    for T, D, dtype in ((40000, 8, "bf16"), (5000, 256, "fp16"), (3000, 1024, "fp32"), (1000, 8192, "bf16"), (700, 8200, "bf16")):
        x, r, gamma = _rows(1, T, D, dtype), _rows(2, T, D, dtype), _rows(3, 1, D, dtype)[0]
        h, y, q = uq.rmsnorm_q8(x, gamma, 1e-5, residual=r, normed=True)
        assert torch.equal(h, (x.float() + r.float()).to(x.dtype))
        _check_norm(h, gamma, 1e-5, y, q, dtype)
        rq, rs = oq.quantize(f32(x))
        codes, scales = uq.quantize_q8(x)
        assert np.array_equal(codes.cpu().numpy(), rq) and np.array_equal(scales.cpu().numpy(), rs)
        # in place, with the next rows' copies under way
        a = x.clone()
        got = uq.rmsnorm_q8(a, gamma, 1e-5, residual=r, h=a)
        assert torch.equal(a, h) and torch.equal(got[2][0], q[0])


def _loud(seed, T, D, dtype, kind):
    """Rows whose squares, or whose squares' sum, leave fp32 while their mean does not; every third row is ordinary."""
    x = _rows(seed, T, D, "fp32")
    x[x == 0] = 0.5
    if kind == "all":
        x[::3] *= 2.0 ** 65 / x[::3].abs().amax(dim=1, keepdim=True)
    else:
        x[::3, D // 2] = 2.0 ** 65
    return x.to(DTYPE[dtype])


@pytest.mark.parametrize("kind", ["all", "one"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D", [(4, 8192), (5, 8191), (700, 8192), (340, 9001), (900, 4000), (2000, 4001), (3, 33001), (400, 16384)])
def test_squares_whose_sum_leaves_fp32(T, D, dtype, kind):
    h, gamma = _loud(1, T, D, dtype, kind), _rows(3, 1, D, dtype)[0].contiguous()
    for eps in (1e-5, 0.0):
        got, y, q = uq.rmsnorm_q8(h, gamma, eps, normed=True)
        assert got is h
        _check_norm(h, gamma, eps, y, q, dtype)
    half = (h.float() * 0.5).to(h.dtype)
    again = uq.rmsnorm_q8(half, gamma, 0.0, residual=half, normed=True)
    assert torch.equal(again[0], h) and torch.equal(again[1], y) and torch.equal(again[2][0], q[0]) and torch.equal(again[2][1], q[1])


@pytest.mark.parametrize("kind", ["all", "one"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D", [(4, 8192), (5, 8191), (700, 8192), (340, 9001), (900, 4000), (2000, 4001), (3, 33001), (400, 16384)])
def test_gradient_where_the_squares_sum_leaves_fp32(T, D, dtype, kind):
    h, gamma, eps = _loud(1, T, D, dtype, kind), _rows(3, 1, D, dtype)[0].contiguous(), 1e-2
    dy = _rows(2, T, D, dtype)
    dx, dgamma = uq.rmsnorm_grad(dy, h, gamma, eps)
    rx, rg = oq.rmsnorm_grad(n(dy), n(h), n(gamma), eps, None)
    H, G = n(h), n(dy) * n(gamma)
    r = 1 / np.sqrt((H * H).mean(axis=1, keepdims=True) + eps)
    mag = r * (np.abs(G) + np.abs(H) * r * r * np.abs(G * H).mean(axis=1, keepdims=True))
    steps = 3 * (D / 32 + 16) + 16
    assert np.all(np.abs(n(dx) - rx) <= ROUND[dtype] * np.abs(rx) * 1.0001 + steps * U * mag + TINY[dtype])
    assert np.all(np.abs(n(dgamma) - rg) <= (T + steps) * U * np.abs(n(dy) * H * r).sum(axis=0) + 2.0 ** -140)
