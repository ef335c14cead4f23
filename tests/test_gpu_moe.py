"""Expert routing on the GPU against the oracle: the stable sort (equal), rows to experts and back with weights, and the
gradients of both.

Tolerances: a sum of k products of fp32 weights and exact inputs in fp32 loses at most (k + 1) * 2^-24 of the sum of
magnitudes, a dot product over H in fp32 (any order) H * 2^-24; then one rounding of the output type.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import moe as omoe  # noqa: E402

DEV = torch.device("cuda:0")
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def _ids(seed, T, k, E, kind="random"):
    g = np.random.default_rng([seed, 3])
    if kind == "one":
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":
        return g.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (T, k)).astype(np.int32)
    p = g.dirichlet(np.full(E, 0.5))
    ids = g.choice(E, (T, k), p=p).astype(np.int32)
    ids[g.random((T, k)) < 0.1] = -1
    ids[g.random((T, k)) < 0.02] = E
    return ids


def _t(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(DTYPE[dtype])


@pytest.mark.parametrize("kind", ["random", "one", "none"])
@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (5, 2, 8), (33, 3, 7), (1000, 8, 64), (4096, 2, 128),
                                   (5000, 8, 1024), (20001, 1, 33)])
def test_sort_is_stable(T, k, E, kind):
    ids = _ids(T + E, T, k, E, kind)
    order, pos, off = uq.moe_sort(_t(ids), E)
    ro, rp, rf = omoe.sort(ids, E)
    assert np.array_equal(off.cpu().numpy(), rf)
    assert np.array_equal(pos.cpu().numpy(), rp)
    assert np.array_equal(order.cpu().numpy(), ro)


CASES = [(1, 1, 1, 1), (1, 2, 4, 4096), (7, 3, 5, 1001), (64, 8, 16, 264), (200, 2, 300, 96), (33, 5, 4, 2050), (300, 1, 8, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,k,E,H", CASES)
def test_rows_there_and_back(T, k, E, H, dtype):
    g = np.random.default_rng([T, H])
    order, pos, off = omoe.sort(_ids(T, T, k, E), E)
    x = _t(g.normal(size=(T, H)), dtype)
    ys, dxs = _t(g.normal(size=(T * k, H)), dtype), _t(g.normal(size=(T * k, H)), dtype)
    w = g.random((T, k)).astype(np.float32)
    n = lambda t: t.double().cpu().numpy()                                           # noqa: E731
    xs = uq.moe_gather(x, _t(pos), _t(off))
    assert np.array_equal(n(xs), omoe.gather(n(x), pos))
    for got, ref, mag in (
            (uq.moe_combine(ys, _t(pos), _t(w)), omoe.combine(n(ys), pos, w), omoe.combine(np.abs(n(ys)), pos, w)),
            (uq.moe_gather_grad(dxs, _t(pos)), omoe.gather_grad(n(dxs), pos), omoe.gather_grad(np.abs(n(dxs)), pos))):
        tol = ROUND[dtype] * np.abs(ref) + (k + 1) * 2.0 ** -24 * mag + 2.0 ** -25
        assert np.all(np.abs(n(got) - ref) <= tol)
    assert not n(uq.moe_combine(ys, _t(np.full_like(pos, -1)), _t(w))).any()         # no route kept


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,k,E,H", CASES)
def test_combine_gradients(T, k, E, H, dtype):
    g = np.random.default_rng([T, H, 1])
    _, pos, off = omoe.sort(_ids(T, T, k, E), E)
    dy, ys = _t(g.normal(size=(T, H)), dtype), _t(g.normal(size=(T * k, H)), dtype)
    w = g.random((T, k)).astype(np.float32)
    n = lambda t: t.double().cpu().numpy()                                           # noqa: E731
    dys, dw = uq.moe_combine_grad(dy, ys, _t(pos), _t(w), _t(off))
    rdys, rdw = omoe.combine_grad(n(dy), n(ys), pos, w)
    _, mag = omoe.combine_grad(np.abs(n(dy)), np.abs(n(ys)), pos, w)
    assert np.all(np.abs(n(dys) - rdys) <= (ROUND[dtype] + 2.0 ** -24) * np.abs(rdys) + 2.0 ** -25)
    assert np.all(np.abs(n(dw) - rdw) <= H * 2.0 ** -24 * mag + 2.0 ** -40)
    again = uq.moe_combine_grad(dy, ys, _t(pos), _t(w), _t(off))
    assert torch.equal(again[0], dys) and torch.equal(again[1], dw)


def test_gradients_agree_with_differences_of_the_forward_calls():
    """fp32, central differences of the framework's own forward calls: linear maps, so any step is exact up to rounding."""
    T, k, E, H = 6, 3, 4, 8
    g = np.random.default_rng(17)
    _, pos, off = omoe.sort(_ids(1, T, k, E), E)
    p, o = _t(pos), _t(off)
    ys, dy, w = _t(g.normal(size=(T * k, H)).astype(np.float32)), _t(g.normal(size=(T, H)).astype(np.float32)), _t(g.random((T, k)).astype(np.float32))
    x, dxs = _t(g.normal(size=(T, H)).astype(np.float32)), _t(g.normal(size=(T * k, H)).astype(np.float32))
    dys, dw = uq.moe_combine_grad(dy, ys, p, w, o)
    dx = uq.moe_gather_grad(dxs, p)
    f = lambda a, b: float((uq.moe_combine(a, p, b).double() * dy.double()).sum())   # noqa: E731
    h = lambda a: float((uq.moe_gather(a, p, o).double() * dxs.double()).sum())      # noqa: E731
    for arr, grad, fn in ((ys, dys, lambda a: f(a, w)), (w, dw, lambda a: f(ys, a)), (x, dx, h)):
        for i in range(0, arr.numel(), 5):
            d = torch.zeros_like(arr).view(-1)
            d[i] = 1.0
            d = d.view(arr.shape)
            assert abs((fn(arr + d) - fn(arr - d)) / 2 - float(grad.view(-1)[i])) < 1e-4


def test_rows_past_32_bit_offsets():
    """R * H = 2.4e9: each of the row calls at the far end."""
    T, k, E, H = 18433, 8, 8, 16384
    ids = torch.arange(T * k, device=DEV, dtype=torch.int32).view(T, k) % E
    _, pos, off = uq.moe_sort(ids, E)
    x = torch.randint(-4, 5, (T, H), device=DEV, dtype=torch.int8).to(torch.bfloat16)
    xs = uq.moe_gather(x, pos, off)
    assert torch.equal(xs[pos[-1].long()], x[-1:].expand(k, -1)) and torch.equal(xs[-1], x[(pos == T * k - 1).nonzero()[0, 0]])
    w = torch.full((T, k), 0.5, device=DEV)
    assert torch.equal(uq.moe_combine(xs, pos, w), x * 4)
    assert torch.equal(uq.moe_gather_grad(xs, pos), x * 8)
    dys, dw = uq.moe_combine_grad(x, xs, pos, w, off)
    assert torch.equal(dys, xs * 0.5)
    assert torch.equal(dw[-3:], x[-3:].float().square().sum(1, keepdim=True).expand(-1, k))


def test_refusals():
    ids = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    for E, status in ((0, 1), (1025, 2)):
        with pytest.raises(uq.UqError) as e:
            uq.moe_sort(ids, E)
        assert e.value.status == status
    x = torch.zeros(3 * 16 + 8, dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    with pytest.raises(uq.UqError) as e:
        uq.moe_gather(x[1:49].view(3, 16), ids, off)                                 # misaligned x
    assert e.value.status == 3
    with pytest.raises(AssertionError):
        uq.moe_combine(x[:48].view(3, 16), ids, torch.zeros(3, 2, device=DEV))       # ys has T*k rows
