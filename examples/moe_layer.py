"""A mixture-of-experts layer whose weights and activations are microscaled 4-bit floating point, and the block around it.

    python examples/moe_layer.py [--tokens 4 --experts 8 --topk 2 --hidden 4096 --inner 14336 --fmt MXFP4]

block(): the residual's addition and the norm, in 8 bits too (rmsnorm_q8), the router (moe_route), the layer, and beside it a
shared expert on 8-bit weights (gemm_w8a8) that takes the norm's codes.

Per call: the router's routes are sorted by expert (moe_sort), the tokens quantized once and gathered by expert
(quantize_mx with pos), gate and up multiplied and combined by silu(g) * u (gemm_mx_grouped with up), the result
quantized in its segments, multiplied with the down weights (gemm_mx_grouped), and brought back with the router's
weights (moe_combine).  Nothing is read on the host, so the call can be captured in a CUDA graph.  The gradients of the
two routing steps, for training with the experts' products in another precision, are moe_combine_grad and
moe_gather_grad.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_uq_gb300 as uq  # noqa: E402


def route(x: torch.Tensor, router: torch.Tensor, topk: int):
    """Expert ids int32 [T][topk] and weights fp32 [T][topk] (softmax over the chosen experts)."""
    return uq.moe_route(x.float() @ router.t(), topk)


def quantize_weights(w: torch.Tensor, fmt: str):
    """bf16 [experts][N][K] -> (codes [experts][N][K/2], scale tiles [experts][...]); once, at load time."""
    parts = [uq.quantize_mx(e, fmt) for e in w]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def moe_layer(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate, up, down, fmt: str) -> torch.Tensor:
    """y[t] = sum_j weights[t][j] * down_e( silu(gate_e x[t]) * up_e x[t] ), e = ids[t][j]; bf16 [T][hidden]."""
    _, pos, offsets = uq.moe_sort(ids, gate[0].shape[0])
    xq = uq.quantize_mx(x, fmt, offsets=offsets, pos=pos)
    h = uq.gemm_mx_grouped(xq, gate, offsets, fmt, up=up)
    hq = uq.quantize_mx(h, fmt, offsets=offsets)
    y = uq.gemm_mx_grouped(hq, down, offsets, fmt)
    return uq.moe_combine(y, pos, weights)


def block(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor, router: torch.Tensor, bias, topk: int, experts, shared,
          fmt: str, groups: int = 1, top_groups: int = 1, eps: float = 1e-5) -> dict:
    """h = x + residual; y = the routed experts' and the shared expert's outputs of the normed rows.

    ``experts``: gate, up, down of moe_layer; ``shared``: gate, up, down as (codes, scales) of quantize_q8."""
    h, normed, q = uq.rmsnorm_q8(x, gamma, eps, residual=residual, normed=True)
    ids, weights = uq.moe_route(normed.float() @ router.t(), topk, score="sigmoid", bias=bias, groups=groups, top_groups=top_groups,
                                group_top=2)
    y = moe_layer(normed, ids, weights, *experts, fmt)
    gate, up = (uq.gemm_w8a8(q, w, dtype=torch.float32) for w in shared[:2])
    return {"h": h, "y": y + uq.gemm_w8a8((torch.nn.functional.silu(gate) * up).to(x.dtype), shared[2])}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--topk", type=int, default=2)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--fmt", choices=sorted(uq.MX_FORMATS), default="MXFP4")
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    E, H, F = a.experts, a.hidden, a.inner

    def weight(n, k):
        return quantize_weights((torch.randn(E, n, k, generator=g, device="cuda") * k ** -0.5).bfloat16(), a.fmt)

    gate, up, down = weight(F, H), weight(F, H), weight(H, F)
    router = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5
    x = torch.randn(a.tokens, H, generator=g, device="cuda").bfloat16()
    ids, weights = route(x, router, a.topk)
    y = moe_layer(x, ids, weights, gate, up, down, a.fmt)

    # the same layer in fp32 from the weights' values, activations not quantized
    want = torch.zeros(a.tokens, H, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            g_, u_, d_ = (uq.dequant_mx((w[0][e], w[1][e]), a.fmt, dtype=torch.float32) for w in (gate, up, down))
            xt = x[t].float()
            want.index_add_(0, t, weights[t, j, None] * ((torch.nn.functional.silu(xt @ g_.t()) * (xt @ u_.t())) @ d_.t()))
    rel = float((y.float() - want).norm() / want.norm())
    print(f"{a.tokens} tokens, {E} experts, top {a.topk}, {H} -> {F} -> {H}, {a.fmt}: "
          f"relative distance to unquantized activations {rel:.3f}")

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            moe_layer(x, ids, weights, gate, up, down, a.fmt)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert uq.device_fault() == 0
    print(f"{start.elapsed_time(end) / 20 * 1e3:.1f} us a layer (graph replay)")


if __name__ == "__main__":
    main()
