"""The binding's care for memory: results of a call on a given stream come from that stream's pool."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402

DEV = torch.device("cuda:0")


def _pool_stream(t):
    """The stream that owns the allocator segment a tensor lies in."""
    p = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= p < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not an allocation of the caching allocator")


def test_results_come_from_the_pool_of_the_given_stream():
    """Memory of the current stream's pool may still be in use by work queued there, and may be given out again there
    while the given stream writes it."""
    s = torch.cuda.Stream()
    x = torch.zeros(8, 256, dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    weights = torch.ones(8, 2, device=DEV)
    nat = torch.zeros(8, 8, dtype=torch.uint8, device=DEV)
    codes = torch.zeros(16, 256, dtype=torch.int8, device=DEV)
    torch.cuda.synchronize()
    q = uq.quantize_mx(x, "MXFP4", stream=s)
    order, pos, off = uq.moe_sort(ids, 4, stream=s)
    qg = uq.quantize_mx(x, "MXFP4", offsets=off, pos=pos, stream=s)
    w = (q[0].repeat(4, 1, 1), q[1].repeat(4, 1))
    torch.cuda.synchronize()
    ys = uq.gemm_mx_grouped(qg, w, off, "MXFP4", stream=s)
    xs = uq.moe_gather(x, pos, off, stream=s)
    dys, dw = uq.moe_combine_grad(torch.zeros(8, 8, dtype=ys.dtype, device=DEV), ys, pos, weights, off, stream=s)
    results = [*q, order, pos, off, *qg, ys, xs, dys, dw, uq.pack_mx_scales(nat, "MXFP4", stream=s),
               uq.dequant_mx(q, "MXFP4", stream=s), uq.gemm_mx(x, q, "MXFP4", stream=s),
               uq.moe_gather_grad(xs, pos, stream=s), uq.moe_combine(ys, pos, weights, stream=s)]
    wq = uq.pack_layout(codes, 128, "INT4_SYM", stream=s)
    scales = torch.zeros(16, 2, dtype=torch.int16, device=DEV)
    torch.cuda.synchronize()
    results += [wq, uq.gemm(x, wq, scales, None, 16, 128, "INT4_SYM", stream=s),
                uq.gemm_gated(x, (wq, scales, None), (wq, scales, None), 16, 128, "INT4_SYM", stream=s),
                uq.gemm_w4a8(x, wq, scales, None, 16, 128, "INT4_SYM", stream=s),
                uq.unpack_codes(wq, 16, 256, 128, "INT4_SYM", stream=s),
                uq.dequant(wq, scales, None, 16, 256, 128, "INT4_SYM", stream=s)]
    torch.cuda.synchronize()
    for i, t in enumerate(results):
        assert _pool_stream(t) == s.cuda_stream, f"result {i}"
    assert _pool_stream(uq.gemm_mx(x, q, "MXFP4")) == torch.cuda.current_stream().cuda_stream
