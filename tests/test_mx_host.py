"""Host-side rules of the microscaled and routing calls: sizes, refusals and empty calls are answered before any CUDA call,
so they are checked here without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from gemm_uq_gb300.build import build
    build()
    import gemm_uq_gb300 as uq
    return uq.lib()


@pytest.fixture(scope="module")
def al():
    buf = (ctypes.c_uint8 * 64)()
    al.keep = buf
    base = ctypes.addressof(buf)
    return base + (-base) % 16


def test_scales_size(L):
    import gemm_uq_gb300 as uq
    for rows, K, fmt, seg in ((1, 32, "MXFP4", 0), (128, 128, "MXFP4", 0), (129, 160, "MXFP4", 0), (8192, 4096, "NVFP4", 0),
                              (300, 96, "NVFP4", 5), (0, 64, "MXFP4", 0), (0, 64, "MXFP4", 3), (127, 64, "NVFP4", 1)):
        block = uq.MX_BLOCK[fmt]
        row_tiles = rows // 128 + seg if seg else -(-rows // 128)
        want = row_tiles * -(-K // (4 * block)) * 512
        assert uq.mx_scales_size(rows, K, fmt, seg) == want == uq._scale_bytes(rows, K, fmt, seg)


@pytest.mark.parametrize("rows,K,fmt,seg", [(1, 33, 0, 0), (1, 16, 1, 0), (-1, 32, 0, 0), (1, 32, 2, 0), (1, 32, 0, -1)])
def test_scales_size_rejects(L, rows, K, fmt, seg):
    v = ctypes.c_size_t()
    assert L.uq_mx_scales_size(rows, K, fmt, seg, ctypes.byref(v)) == 1
    assert len(L.uq_last_error()) > 0


def test_quantize_refusals(L, al):
    q = lambda x=al, t=0, ld=64, c=al, s=al, rows=2, K=64, fmt=0, ts=1.0, off=None, seg=0, pos=None, k=0: \
        L.uq_quantize_mx(x, t, ld, c, s, rows, K, fmt, ts, off, seg, pos, k, None)   # noqa: E731
    assert q(rows=0) == 0 and q(K=0) == 0                                    # nothing to do
    assert q(x=None) == 1 and q(c=None) == 1 and q(s=None) == 1
    assert q(t=3) == 1 and q(K=48) == 1 and q(ld=63) == 1 and q(fmt=7) == 1
    assert q(ts=2.0) == 1 and q(fmt=1, ts=float("inf")) == 1 and q(fmt=1, ts=-1.0) == 1
    assert q(off=al) == 1 and q(seg=2) == 1 and q(pos=al, k=2) == 1          # offsets and segments go together
    assert q(x=al + 8) == 3 and q(ld=68) == 3 and q(c=al + 4) == 3
    assert q(off=al, seg=1, pos=al, k=2 ** 30, rows=4) == 1                  # 2^32 routes


def test_product_refusals(L, al):
    g = lambda x=al, t=0, ld=64, xs=None, ts=1.0, w=al, ws=al, y=al, yt=0, M=2, N=8, K=64, fmt=0: \
        L.uq_gemm_mx(x, t, ld, xs, ts, w, ws, y, yt, M, N, K, fmt, 1.0, None)        # noqa: E731
    assert g(M=0) == 0 and g(N=0) == 0
    assert g(M=-1) == 1 and g(N=-1) == 1 and g(K=40) == 1 and g(yt=5) == 1 and g(fmt=-1) == 1
    assert g(x=None) == 1 and g(w=None) == 1 and g(ws=None) == 1 and g(y=None) == 1
    assert g(y=al + 2) == 3 and g(w=al + 8) == 3 and g(xs=al + 8) == 3 and g(x=al + 8) == 3
    r = lambda x=al, xs=al, w=al, ws=al, up=None, us=None, off=al, a=None, au=None, y=al, yt=0, rows=4, E=2, N=8, K=64, fmt=0: \
        L.uq_gemm_mx_grouped(x, xs, w, ws, up, us, off, a, au, y, yt, rows, E, N, K, fmt, None)   # noqa: E731
    assert r(rows=0) == 0 and r(N=0) == 0
    assert r(E=0) == 1 and r(E=1025) == 2 and r(N=2 ** 30, E=4) == 2
    assert r(up=al) == 1 and r(us=al) == 1 and r(au=al) == 1                 # both parts of up, alpha_up only with it
    assert r(off=None) == 1 and r(x=None) == 1 and r(xs=None) == 1
    assert r(off=al + 4) == 3 and r(a=al + 4) == 3


def test_routing_refusals(L, al):
    assert L.uq_moe_sort(al, 2, 2, 0, al, al, al, None) == 1
    assert L.uq_moe_sort(al, 2, 2, 1025, al, al, al, None) == 2
    assert L.uq_moe_sort(None, 2, 2, 4, al, al, al, None) == 1
    assert L.uq_moe_sort(al, 2, 2, 4, al, al, None, None) == 1
    assert L.uq_moe_sort(al + 4, 2, 2, 4, al, al, al, None) == 3
    assert L.uq_moe_sort(al, 2 ** 20, 2 ** 12, 4, al, al, al, None) == 1
    assert L.uq_moe_gather(al, 0, al, al, 4, al, 0, 2, 8, None) == 0
    assert L.uq_moe_gather(al, 9, al, al, 4, al, 1, 2, 8, None) == 1
    assert L.uq_moe_gather(None, 0, al, al, 4, al, 1, 2, 8, None) == 1
    assert L.uq_moe_combine(al, 0, al, None, al, 1, 2, 8, None) == 1          # weights are needed
    assert L.uq_moe_combine(al, 0, al, al, al + 8, 1, 2, 8, None) == 3
    assert L.uq_moe_gather_grad(al, 0, None, al, 1, 2, 8, None) == 1
    assert L.uq_moe_combine_grad(al, al, 0, al, al, al, 4, None, al, 1, 2, 8, None) == 1
    assert L.uq_moe_combine_grad(al, al, 0, al, al, al, 4, al, al, 0, 2, 8, None) == 0


def test_sizes_next_to_2_31_are_refused(L, al):
    """Within a tile of 2^31 the sizes rounded up to tiles and steps leave 32 bits."""
    for big in (2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 256, 2 ** 31 - 4096):
        assert L.uq_gemm_mx(al, 0, 64, al, 1.0, al, al, al, 0, big, 1, 64, 0, 1.0, None) == 2
        assert L.uq_gemm_mx(al, 0, 64, al, 1.0, al, al, al, 0, 1, big, 64, 0, 1.0, None) == 2
        assert L.uq_gemm_mx_grouped(al, al, al, al, None, None, al, None, None, al, 0, big, 1, 1, 64, 0, None) == 2
        assert L.uq_gemm_mx_grouped(al, al, al, al, None, None, al, None, None, al, 0, 1, 1, big, 64, 0, None) == 2
        assert L.uq_moe_gather(al, 0, al, al, 4, al, 1, 2, big, None) == 2
        assert L.uq_moe_combine(al, 0, al, al, al, 1, 2, big, None) == 2
        assert L.uq_moe_gather_grad(al, 0, al, al, 1, 2, big, None) == 2
        assert L.uq_moe_combine_grad(al, al, 0, al, al, al, 4, al, al, 1, 2, big, None) == 2
        assert L.uq_gemm_mx_grouped(al, al, al, al, None, None, al, None, None, al, 0, 1, 2, 2 ** 30 - 1, 64, 0, None) == 2
        K = big // 32 * 32
        assert L.uq_gemm_mx(al, 0, K, al, 1.0, al, al, al, 0, 1, 1, K, 0, 1.0, None) == 2
        assert L.uq_quantize_mx(al, 0, K, al, al, 1, K, 0, 1.0, None, 0, None, 0, None) == 2
        assert L.uq_dequant_mx(al, al, al, 0, 1, K, 0, 1.0, None, 0, None) == 2
        assert L.uq_pack_mx_scales(al, al, 1, 1, K, 0, None) == 2
