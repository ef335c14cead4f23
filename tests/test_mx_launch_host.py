"""What the microscaled and routing calls launch, and how, on a host stand-in for the CUDA runtime."""
import ctypes

import pytest

from tests.fake_cuda import load


@pytest.fixture
def cuda(tmp_path):
    f = load(tmp_path)
    yield f
    f.lib.uq_set_launch_overlap(0)


def _product(f, M, stream=None, pair=False):
    a = f.at
    return f.launches(lambda: f.lib.uq_gemm_mx(a, 0, 2048, a if pair else None, 1.0, a, a, a, 0, M, 1024, 2048, 0, 1.0, stream))


def _quantize(f, stream=None):
    a = f.at
    return f.launches(lambda: f.lib.uq_quantize_mx(a, 0, 2048, a, a, 4, 2048, 0, 1.0, None, 0, None, 0, stream))


@pytest.mark.parametrize("M,pair", [(1, False), (3, False), (5, False), (2000, False), (5, True)])
def test_a_product_after_a_call_that_writes_operands_does_not_overlap_it(cuda, M, pair):
    """quantize_mx and pack_mx_scales may have written the weights that an overlapping product requests before its wait."""
    f, a = cuda, cuda.at
    f.lib.uq_set_launch_overlap(1)
    other = ctypes.c_void_p(64)
    kernels = 1 if pair or M <= 3 else 2
    for write in (lambda: _quantize(f), lambda: f.launches(lambda: f.lib.uq_pack_mx_scales(a, a, 1, 128, 2048, 0, None))):
        write()
        assert [x.overlap for x in _product(f, M, other, pair)] == [1] * kernels          # another stream
        first = _product(f, M, None, pair)
        assert [x.overlap for x in first] == [0, 1][:kernels]                             # its quantizer, if it has one
        assert [x.overlap for x in _product(f, M, None, pair)] == [1] * kernels           # the one after overlaps again
    # rows by expert: the kernel waits for the offsets before it requests weights
    _quantize(f)
    grouped = f.launches(lambda: f.lib.uq_gemm_mx_grouped(a, a, a, a, None, None, a, None, None, a, 0, 8, 2, 256, 512, 0, None))
    assert [x.overlap for x in grouped] == [1]
    assert [x.overlap for x in _product(f, M, None, pair)] == [1] * kernels


def test_a_product_that_fails_does_not_settle_fresh_operands(cuda):
    """Operands are written, a product that needs a workspace gets none, the next product may still have them as weights."""
    f, a = cuda, cuda.at
    f.lib.uq_set_launch_overlap(1)
    _quantize(f)
    f.lib.fake_set_no_memory(1)
    assert f.lib.uq_gemm_mx(a, 0, 2048, None, 1.0, a, a, a, 0, 5, 1024, 2048, 0, 1.0, None) == 5     # UQ_ERR_NOMEM
    f.lib.fake_set_no_memory(0)
    assert [x.overlap for x in _product(f, 1)] == [0]
    assert [x.overlap for x in _product(f, 1)] == [1]


def test_no_overlap_unless_asked_for(cuda):
    _quantize(cuda)
    for M in (1, 5):
        launched = _product(cuda, M)
        # a product's own quantizer lets the product start under it in any case
        assert [x.overlap for x in launched] == ([0] if M == 1 else [0, 1])


@pytest.mark.parametrize("largest", [16, 8, 4, 1])
def test_route_sort_takes_the_cluster_that_can_be_placed(cuda, largest):
    """A cluster of 16 CTAs is not portable: where none can be placed the sort takes a smaller one (any size is right)."""
    f, a = cuda, cuda.at
    f.lib.fake_set_largest_cluster(largest)
    for n, ctas in ((1, 1), (1024, 1), (1025, 2), (8193, 16), (100000, 16)):
        launched = f.launches(lambda: f.lib.uq_moe_sort(a, n, 1, 64, a, a, a, None))
        assert [(x.grid, x.cluster) for x in launched] == [(min(ctas, largest),) * 2]
