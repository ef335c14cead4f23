"""The router on the GPU against the oracle: the choice is equal, weights and gradients to fp32.

Tolerances, u = 2^-24: an exponential 4 u and |x - max| u of its argument's rounding, a sum over E (E / 32 + 8) u, a quotient
and products 8 u; the gradient the same on the summed magnitudes, twice (scores and the weighted mean)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import router as orr  # noqa: E402

DEV = torch.device("cuda:0")
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}
U = 2.0 ** -24


def n(t):
    return t.double().cpu().numpy()


def _logits(seed, T, E, dtype, mask=0.0, spread=1.0):
    g = np.random.default_rng([seed, T, E])
    x = g.normal(size=(T, E)) * spread
    x[g.random((T, E)) < mask] = -np.inf
    return torch.from_numpy(x).to(DTYPE[dtype]).to(DEV)


def _check(x, ids, w, k, score, renorm, scale, **kw):
    ref = orr.choose(n(x), k, score, **kw)
    assert np.array_equal(ids.cpu().numpy(), ref)
    rw = orr.weights(n(x), ref, score, renorm, scale)
    span = float(np.ptp(n(x)[np.isfinite(n(x))])) if np.isfinite(n(x)).any() else 0.0
    tol = 2 * (x.shape[1] / 32 + 24 + span) * U
    assert np.all(np.abs(n(w) - rw) <= tol * np.abs(rw) + 2.0 ** -126)


CASES = [(1, 1, 1, 1, 1), (5, 8, 2, 1, 1), (33, 7, 3, 1, 1), (64, 60, 4, 4, 2), (200, 256, 8, 8, 4), (17, 160, 6, 8, 3), (9, 1024, 32, 32, 7),
         (40, 33, 1, 3, 1), (300, 100, 8, 5, 5), (12, 64, 2, 32, 1), (3, 1023, 8, 1, 1)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,G,tg", CASES)
def test_choice_and_weights(T, E, k, G, tg, dtype, score, renorm):
    for mask in (0.0, 0.3):
        x = _logits(1, T, E, dtype, mask)
        bias = torch.from_numpy(np.random.default_rng(E).normal(size=E).astype(np.float32) * 0.1).to(DEV)
        if mask:
            bias[E // 2] = float("-inf")
        for b in (None, bias):
            for gt in (1, 2) if G > 1 else (1,):
                ids, w = uq.moe_route(x, k, score=score, bias=b, groups=G, top_groups=tg, group_top=gt, renormalize=renorm, scale=1.5)
                _check(x, ids, w, k, score, renorm, 1.5, bias=None if b is None else n(b), groups=G, top_groups=tg, group_top=gt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties_are_decided_as_in_64_bits(score):
    """Choice values that fp32 cannot tell apart: scores next to biases that undo their differences to a few 2^-26."""
    g = np.random.default_rng(11)
    T, E, k = 64, 96, 6
    base = g.normal(size=E).astype(np.float32)
    x = torch.from_numpy(np.tile(base, (T, 1)) + (g.integers(-3, 4, (T, E)) * 2.0 ** -22)).float().to(DEV)
    s = orr.scores(base[None].astype(np.float64), score)[0]
    bias = torch.from_numpy((1.0 - s).astype(np.float32)).to(DEV)
    for G, tg, gt in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        ids, w = uq.moe_route(x, k, score=score, bias=bias, groups=G, top_groups=tg, group_top=gt)
        _check(x, ids, w, k, score, True, 1.0, bias=n(bias), groups=G, top_groups=tg, group_top=gt)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(score, bias):
    x = torch.zeros(4, 70, device=DEV)
    x[1, 40:] = 1.0
    x[2] = torch.tensor([-0.0, 0.0], device=DEV).repeat(35)
    x[3, 69] = 2.0
    b = torch.full((70,), 0.25, device=DEV) if bias else None
    for G, tg, gt in ((1, 1, 1), (10, 4, 2), (10, 4, 1)):
        ids, _ = uq.moe_route(x, 5, score=score, bias=b, groups=G, top_groups=tg, group_top=gt)
        assert np.array_equal(ids.cpu().numpy(), orr.choose(n(x), 5, score, None if b is None else n(b), G, tg, gt))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masked_nan_and_far_logits(dtype):
    low = float("-inf")
    x = torch.full((8, 40), low, device=DEV)
    x[1, 3] = 2.0
    x[2] = torch.linspace(-3, 3, 40, device=DEV)
    x[2, 7] = float("nan")
    x[3] = -300.0
    x[3, 5], x[3, 9] = -100.0, -101.0
    x[4] = 500.0
    x[4, :20] = -500.0
    x[5] = torch.finfo(DTYPE[dtype]).min
    x[6, :2] = torch.tensor([-120.0, -119.0], device=DEV)
    x[7] = 1.0
    x = x.to(DTYPE[dtype])
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, w = uq.moe_route(x, 3, score=score, renormalize=renorm)
            ref = orr.choose(n(x), 3, score)
            assert np.array_equal(ids.cpu().numpy(), ref)
            keep = [0, 1, 3, 4, 6, 7]
            rw = orr.weights(n(x), ref, score, renorm)[keep]
            got = n(w)[keep]
            assert np.all(np.abs(got - rw) <= 1100 * U * np.abs(rw) + 2.0 ** -126)
            assert not w[0].any() and (ids[0] == -1).all()
            if score == "softmax":
                assert torch.isnan(w[2]).all()
            else:
                assert torch.isfinite(w[2]).all()                        # the NaN is not among the chosen
    ids, w = uq.moe_route(x[2:3], 32)
    assert 7 not in ids[0].tolist()
    x[2, 8:] = low                                                       # now it is the last that can be chosen
    ids, w = uq.moe_route(x[2:3], 9, score="sigmoid")
    assert ids[0].tolist() == [6, 5, 4, 3, 2, 1, 0, 7, -1] and torch.isnan(w[0, :8]).all() and w[0, 8] == 0


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (33, 7, 3), (129, 60, 4), (200, 256, 8), (9, 1024, 32), (40, 33, 1), (20, 70, 6)])
def test_gradient(T, E, k, dtype, score, renorm):
    x = _logits(3, T, E, dtype, 0.1)
    g = np.random.default_rng([T, k])
    ids = orr.choose(n(x), k, score)
    if T > 4:
        ids[1] = -1                                                      # no route
        ids[2, 0] = E                                                    # none either
        ids[3] = 0                                                       # one expert named k times
        x[3, 0] = 0.5
    dw = torch.from_numpy(g.normal(size=(T, k)).astype(np.float32)).to(DEV)
    dx = uq.moe_route_grad(x, torch.from_numpy(ids).to(DEV), dw, score=score, renormalize=renorm, scale=2.5)
    ref, mag = orr.grad(n(x), ids, n(dw), score, renorm, 2.5)
    tol = ROUND[dtype] * np.abs(ref) * 1.0001 + 4 * (E / 32 + 40) * U * mag + TINY[dtype]
    assert np.all(np.abs(n(dx) - ref) <= tol)


def test_nothing_to_do():
    x = torch.randn(4, 8, device=DEV)
    ids, w = uq.moe_route(x[:0], 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    ids, w = uq.moe_route(x, 0)
    assert ids.shape == (4, 0)
    assert not uq.moe_route_grad(x, ids, w).any()


def test_many_tokens_and_a_graph():
    x = _logits(5, 20001, 64, "bf16")
    ids, w = uq.moe_route(x, 6)
    top, ref = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(ids, ref[:, :6].int())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = uq.moe_route(x, 6)
            dx = uq.moe_route_grad(x, got[0], got[1])
        g.replay()
    s.synchronize()
    assert torch.equal(got[0], ids) and torch.equal(got[1], w)
    assert torch.equal(dx, uq.moe_route_grad(x, ids, w))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_gradient_of_routes_to_masked_experts(dtype, score, renorm):
    """Routes whose experts' logits are all minus infinity have weights of 0, and the logits no gradient from them."""
    x = _logits(7, 6, 20, dtype)
    x[1, 3:6] = float("-inf")
    x[2] = float("-inf")
    x[3, 4] = float("-inf")
    ids = torch.tensor([[0, 1, 2], [3, 4, 5], [0, 1, 2], [4, 5, 6], [-1, -1, -1], [7, 7, 20]], dtype=torch.int32)
    dw = torch.from_numpy(np.random.default_rng(3).normal(size=(6, 3)).astype(np.float32)).to(DEV)
    dx = uq.moe_route_grad(x, ids.to(DEV), dw, score=score, renormalize=renorm, scale=1.5)
    ref, mag = orr.grad(n(x), ids.numpy(), n(dw), score, renorm, 1.5)
    tol = ROUND[dtype] * np.abs(ref) * 1.0001 + 4 * (20 / 32 + 40) * U * mag + TINY[dtype]
    assert np.all(np.abs(n(dx) - ref) <= tol)
    assert not dx[2].any() and not dx[4].any()
    if renorm:
        assert not dx[1].any()
