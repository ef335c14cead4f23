"""The binding's care for memory: results of a call on a given stream come from that stream's pool, and operands of a
type that the kernels would misread are refused."""
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


def test_operands_of_another_type_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    w = (torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.zeros(512, dtype=torch.uint8, device=DEV))
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    q, qs = uq.quantize_mx(x, "MXFP4"), uq.quantize_mx(x, "MXFP4", offsets=off)
    wg = (w[0][None], w[1][None])

    def wide(t):
        return t.to(torch.int32)

    def refused(f):
        with pytest.raises(AssertionError):
            f()

    for i in range(2):
        other = tuple(wide(t) if j == i else t for j, t in enumerate(q))
        refused(lambda: uq.dequant_mx(other, "MXFP4"))
        refused(lambda: uq.gemm_mx(other, w, "MXFP4"))
        refused(lambda: uq.gemm_mx(x, tuple(wide(t) if j == i else t for j, t in enumerate(w)), "MXFP4"))
        refused(lambda: uq.gemm_mx_grouped(tuple(wide(t) if j == i else t for j, t in enumerate(qs)), wg, off, "MXFP4"))
        other_w = tuple(wide(t) if j == i else t for j, t in enumerate(wg))
        refused(lambda: uq.gemm_mx_grouped(qs, other_w, off, "MXFP4"))
        refused(lambda: uq.gemm_mx_grouped(qs, wg, off, "MXFP4", up=other_w))
    refused(lambda: uq.dequant_mx(q, "MXFP4", offsets=off.long()))
    refused(lambda: uq.quantize_mx(x.cpu(), "MXFP4"))
    refused(lambda: uq.gemm_mx(x, (w[0].cpu(), w[1]), "MXFP4"))
    refused(lambda: uq.gemm_mx(x, w, "MXFP4", y=torch.zeros(4, 8, dtype=torch.bfloat16)))
    refused(lambda: uq.moe_sort(torch.zeros(4, 2, dtype=torch.int32), 4))
