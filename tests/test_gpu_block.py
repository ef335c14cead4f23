"""The parts of a mixture-of-experts block together: residual and norm, the router, the sort, microscaled experts, a shared
expert in 8 bits, and the way back; then the gradients of norm and router behind those of the routing calls."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from examples.moe_layer import block, moe_layer, quantize_weights  # noqa: E402
from oracle import q8 as oq, router as orr  # noqa: E402

DEV = torch.device("cuda:0")
EPS = 1e-5


def n(t):
    return t.double().cpu().numpy()


def _weights(g, E, H, F):
    def w(*s):
        return (torch.randn(*s, generator=g, device=DEV) * s[-1] ** -0.5).bfloat16()
    experts = [quantize_weights(w(E, F, H), "MXFP4"), quantize_weights(w(E, F, H), "MXFP4"), quantize_weights(w(E, H, F), "MXFP4")]
    shared = [uq.quantize_q8(w(F, H)), uq.quantize_q8(w(F, H)), uq.quantize_q8(w(H, F))]
    return experts, shared, w(E, H).float()


@pytest.mark.parametrize("T", [1, 5, 33, 300])
def test_block(T):
    """Every step of the block against the oracle of that step on the step's own inputs, and the captured block equal to it."""
    E, H, F, k = 16, 512, 768, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    (gate, up, down), shared, router = _weights(g, E, H, F)
    gamma = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).bfloat16()
    bias = 0.05 * torch.randn(E, generator=g, device=DEV)
    x, res = (torch.randn(T, H, generator=g, device=DEV).bfloat16() for _ in range(2))
    out = block(x, res, gamma, router, bias, k, (gate, up, down), shared, "MXFP4", groups=4, top_groups=2)
    h, y, q = uq.rmsnorm_q8(x, gamma, EPS, residual=res, normed=True)
    assert torch.equal(out["h"], h)
    ref, scale = oq.rmsnorm(n(h), n(gamma), EPS)
    assert np.all(np.abs(n(q[0]) * n(q[1])[:, None] - ref) <= 0.51 * scale[:, None])
    logits = y.float() @ router.t()
    ids, weights = uq.moe_route(logits, k, score="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2)
    assert np.array_equal(ids.cpu().numpy(), orr.choose(n(logits), k, "sigmoid", n(bias), 4, 2, 2))
    # the shared expert: two products of the norm's codes, one of rows quantized in the call
    a, b = (uq.gemm_w8a8(q, w, dtype=torch.float32) for w in shared[:2])
    for got, w in ((a, shared[0]), (b, shared[1])):
        want, mag = oq.gemm(*(t.cpu().numpy() for t in q + w))
        assert np.all(np.abs(n(got) - want) <= (H / 1024 + 5) * 2.0 ** -24 * mag + 2.0 ** -149)
    mid = (torch.nn.functional.silu(a) * b).bfloat16()
    total = moe_layer(y, ids, weights, gate, up, down, "MXFP4") + uq.gemm_w8a8(mid, shared[2])
    assert torch.equal(out["y"], total)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        again = block(x, res, gamma, router, bias, k, (gate, up, down), shared, "MXFP4", groups=4, top_groups=2)
        with torch.cuda.graph(graph, stream=s):
            again = block(x, res, gamma, router, bias, k, (gate, up, down), shared, "MXFP4", groups=4, top_groups=2)
        for t in again.values():
            t.zero_()
        graph.replay()
    s.synchronize()
    assert torch.equal(again["h"], out["h"]) and torch.equal(again["y"], out["y"])
    assert uq.device_fault() == 0


def test_overlapping_products_behind_the_quantizer():
    """With launch overlap a microscaled product behind an 8-bit call on the stream reads that call's result complete."""
    T, H, N = 64, 2048, 1024
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    w8 = uq.quantize_q8(torch.randn(H, H, generator=g, device=DEV).bfloat16())
    wm = uq.quantize_mx(torch.randn(N, H, generator=g, device=DEV).bfloat16(), "MXFP4")
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    want = uq.gemm_mx(uq.gemm_w8a8(x, w8), wm, "MXFP4")
    uq.set_launch_overlap(True)
    try:
        for _ in range(20):
            got = uq.gemm_mx(uq.gemm_w8a8(x, w8), wm, "MXFP4")
            assert torch.equal(got, want)
    finally:
        uq.set_launch_overlap(False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradients_through_routing_and_norm(score):
    """Loss of the combined routes, back through combine, router and norm, against autograd in 64 bits on the same numbers."""
    T, E, H, k = 96, 8, 256, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    h, gamma = torch.randn(T, H, generator=g, device=DEV), 1 + 0.1 * torch.randn(H, generator=g, device=DEV)
    router, dy = torch.randn(E, H, generator=g, device=DEV) * H ** -0.5, torch.randn(T, H, generator=g, device=DEV)
    rows = torch.randn(T * k, H, generator=g, device=DEV)                   # the experts' outputs, sorted
    y = uq.rmsnorm_q8(h, gamma, EPS, normed=True, quantized=False)[1]
    logits = y @ router.t()
    ids, weights = uq.moe_route(logits, k, score=score, scale=2.0)
    _, pos, offsets = uq.moe_sort(ids, E)
    _, dw = uq.moe_combine_grad(dy, rows, pos, weights, offsets)
    dlogits = uq.moe_route_grad(logits, ids, dw, score=score, scale=2.0)
    dx, dgamma = uq.rmsnorm_grad(dlogits @ router, h, gamma, EPS)

    H64, G64 = h.double().requires_grad_(), gamma.double().requires_grad_()
    y64 = H64 * torch.rsqrt(H64.pow(2).mean(dim=1, keepdim=True) + EPS) * G64
    l64 = y64 @ router.double().t()
    s64 = torch.softmax(l64, dim=1) if score == "softmax" else torch.sigmoid(l64)
    w64 = s64.gather(1, ids.long())
    w64 = 2.0 * w64 / w64.sum(dim=1, keepdim=True)
    out = (w64[..., None] * rows.double()[pos.long()]).sum(dim=1)
    wx, wg = torch.autograd.grad(out, (H64, G64), dy.double())
    # each step in fp32: dot products over H twice, sums over 8 experts and 96 rows; the matrix products are torch's own
    for got, want in ((dx, wx), (dgamma, wg)):
        assert float((got.double() - want).norm() / want.norm()) <= 4 * (H + T) * 2.0 ** -24
