"""GPU: uq_set_launch_overlap (programmatic dependent launch) keeps chained calls correct --
the second linear reads the first one's output as its x, on the same stream, eagerly and inside a
captured CUDA graph -- and gives bit-identical results to the plain launches."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import quant as oquant  # noqa: E402
from synth import activations, normal_weights  # noqa: E402
from tests.uq_helpers import device_weights, device_x  # noqa: E402

DEV = torch.device("cuda:0")


def _layer(seed, N, K):
    qz = oquant.quantize(normal_weights(seed, N, K, 0.02), "INT4_ASYM", 128)
    return device_weights(qz, DEV)


def _chain(layers, x, M, reps):
    outs = []
    for _ in range(reps):
        h = x
        for (wq, sc, zc), N in layers:
            h = uq.gemm(h, wq, sc, zc, N, 128, "INT4_ASYM")
        outs.append(h)
    return outs


@pytest.mark.parametrize("M", [1, 5, 16, 33])
def test_overlap_chain_matches_plain(M):
    # K of every layer a multiple of 1024, so M >= 16 runs the tensor-core path
    dims = [4096, 2048, 4096, 3072, 4096]
    layers = [(_layer(900 + i, dims[i + 1], dims[i]), dims[i + 1]) for i in range(len(dims) - 1)]
    x = device_x(activations(901, M, dims[0]), DEV)
    try:
        uq.set_launch_overlap(False)
        ref = _chain(layers, x, M, 3)
        torch.cuda.synchronize()
        uq.set_launch_overlap(True)
        got = _chain(layers, x, M, 3)
        torch.cuda.synchronize()
        for r, g in zip(ref, got):
            assert torch.equal(r.view(torch.int16), g.view(torch.int16))
        # the same chain captured in a graph and replayed
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            _chain(layers, x, M, 1)          # workspace for this stream, outside capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = _chain(layers, x, M, 1)[0]
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), ref[0].view(torch.int16))
    finally:
        uq.set_launch_overlap(False)
    assert uq.device_fault() == 0


def _mx_chain(layers, x, fmt, reps):
    outs = []
    for _ in range(reps):
        h = x
        for w in layers:
            h = uq.gemm_mx(h, w, fmt)
        outs.append(h)
    return outs


@pytest.mark.parametrize("M", [1, 3, 17, 200, 1100])
@pytest.mark.parametrize("fmt", ["MXFP4", "NVFP4"])
def test_overlap_microscaled_chain_matches_plain(M, fmt):
    """Each product reads the one before it, whichever kernel takes it: quantizing in the product, split along k, many
    rows; buffers come round again from call to call."""
    dims = [2048, 9216, 1056, 4352, 2048]
    layers = [uq.quantize_mx(device_x(activations(910 + i, dims[i + 1], dims[i]), DEV), fmt) for i in range(len(dims) - 1)]
    x = device_x(activations(911, M, dims[0]), DEV)
    try:
        uq.set_launch_overlap(False)
        ref = _mx_chain(layers, x, fmt, 1)[0]
        torch.cuda.synchronize()
        assert torch.isfinite(ref.float()).all()
        uq.set_launch_overlap(True)
        for g in _mx_chain(layers, x, fmt, 10):
            assert torch.equal(ref.view(torch.int16), g.view(torch.int16))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _mx_chain(layers, x, fmt, 1)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = _mx_chain(layers, x, fmt, 3)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for g in outs:
            assert torch.equal(ref.view(torch.int16), g.view(torch.int16))
    finally:
        uq.set_launch_overlap(False)
    assert uq.device_fault() == 0


@pytest.mark.parametrize("T", [1, 5, 400])
def test_overlap_expert_layer_matches_plain(T):
    """Sort, quantize and gather, gated product, quantize, product, combine; the counts change from call to call."""
    E, k, H, F, fmt = 8, 2, 1024, 1536, "MXFP4"
    def weight(seed, n, kk):
        parts = [uq.quantize_mx(device_x(activations(seed + e, n, kk), DEV), fmt) for e in range(E)]
        return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    gate, up, down = weight(920, F, H), weight(940, F, H), weight(960, H, F)
    x = device_x(activations(912, T, H), DEV) * 0.02
    rng = np.random.default_rng(T)
    ids = [torch.from_numpy(rng.integers(-1, E, (T, k)).astype(np.int32)).to(DEV) for _ in range(6)]
    weights = torch.rand(T, k, device=DEV)

    def layer(i):
        order, pos, off = uq.moe_sort(i, E)
        q = uq.quantize_mx(x, fmt, offsets=off, pos=pos)
        h = uq.gemm_mx_grouped(q, gate, off, fmt, up=up)
        y = uq.gemm_mx_grouped(uq.quantize_mx(h, fmt, offsets=off), down, off, fmt)
        return uq.moe_combine(y, pos, weights)

    try:
        uq.set_launch_overlap(False)
        ref = [layer(i) for i in ids]
        torch.cuda.synchronize()
        uq.set_launch_overlap(True)
        for _ in range(5):
            for r, i in zip(ref, ids):
                assert torch.equal(r.view(torch.int16), layer(i).view(torch.int16))
    finally:
        uq.set_launch_overlap(False)
    assert uq.device_fault() == 0


@pytest.mark.parametrize("M", [1, 5, 130])
def test_overlap_weights_quantized_in_the_same_stream(M):
    """Weights that quantize_mx writes one or two calls before the product that reads them."""
    N, K = 2304, 2048
    ws = [device_x(activations(970 + i, N, K), DEV) for i in range(4)]
    x = device_x(activations(971, M, K), DEV)
    other = uq.quantize_mx(ws[0], "MXFP4")
    try:
        uq.set_launch_overlap(False)
        ref = [uq.gemm_mx(x, uq.quantize_mx(w, "MXFP4"), "MXFP4") for w in ws]
        torch.cuda.synchronize()
        uq.set_launch_overlap(True)
        for rep in range(8):
            for w, r in zip(ws, ref):
                fresh = uq.quantize_mx(w, "MXFP4")
                if rep % 2:
                    uq.gemm_mx(x, other, "MXFP4")
                assert torch.equal(r.view(torch.int16), uq.gemm_mx(x, fresh, "MXFP4").view(torch.int16))
    finally:
        uq.set_launch_overlap(False)
    assert uq.device_fault() == 0
