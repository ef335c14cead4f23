"""Launch overlap of the microscaled calls: weights that earlier work on the same stream writes, and inputs that the call
before writes, whatever they are."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import moe as omoe  # noqa: E402

DEV = torch.device("cuda:0")


def _rand(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


@pytest.fixture
def overlap():
    yield uq.set_launch_overlap
    uq.set_launch_overlap(False)
    assert uq.device_fault() == 0


@pytest.mark.parametrize("M", [1, 5, 130, 1100])
def test_weights_copied_two_calls_before(M, overlap):
    """A copy writes the weights, a product on other weights follows, then the product that reads them: everything
    before a microscaled call is complete when the next one requests its weights."""
    N, K = 2304, 2048
    sources = [uq.quantize_mx(_rand(i, N, K), "MXFP4") for i in range(4)]
    other = uq.quantize_mx(_rand(9, K, K), "MXFP4")
    x = _rand(10, M, K)
    w = tuple(torch.empty_like(t) for t in sources[0])
    overlap(False)
    ref = [uq.gemm_mx(x, s, "MXFP4") for s in sources]
    torch.cuda.synchronize()
    overlap(True)
    for _ in range(8):
        got = []
        for s in sources:
            for a, b in zip(w, s):
                a.copy_(b)
            uq.gemm_mx(x, other, "MXFP4")
            got.append(uq.gemm_mx(x, w, "MXFP4"))
        for r, g in zip(ref, got):
            assert torch.equal(r, g)


@pytest.mark.parametrize("T", [1, 40, 700])
def test_inputs_that_change_between_overlapping_calls(T, overlap):
    """Rows, routes, offsets and factors are rewritten in place before every call of a chain of overlapping kernels."""
    E, k, H, N, fmt = 6, 2, 512, 640, "NVFP4"
    parts = [uq.quantize_mx(_rand(20 + e, N, H), fmt) for e in range(E)]
    w = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    rng = np.random.default_rng(T)
    sets = []
    for i in range(5):
        _, pos, off = omoe.sort(rng.integers(-1, E, (T, k)).astype(np.int32), E)
        sets.append((_rand(30 + i, T, H), torch.from_numpy(pos).to(DEV), torch.from_numpy(off).to(DEV),
                     torch.rand(E, device=DEV)))
    buf = tuple(t.clone() for t in sets[0])

    def chain(i):
        for b, t in zip(buf, sets[i]):
            b.copy_(t)
        x, pos, off, alpha = buf
        q = uq.quantize_mx(x, fmt, offsets=off, pos=pos)
        return uq.gemm_mx_grouped(q, w, off, fmt, alpha=alpha)

    overlap(False)
    ref = [chain(i) for i in range(5)]
    torch.cuda.synchronize()
    overlap(True)
    for _ in range(6):
        got = [chain(i) for i in range(5)]
        for r, g in zip(ref, got):
            assert torch.equal(r, g)
