"""The example layer (examples/moe_layer.py): every step in the order a user runs them, against the oracle.

Each step is checked from the step before as the layer computed it (a quantization is a step function, so a rounding
difference ahead of it would move whole codes): the gated product within its rule, then the layer's output within the
down product's rule, one rounding of its bf16 rows and of the combined sum.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import moe as omoe  # noqa: E402
from oracle import mx as omx  # noqa: E402

DEV = torch.device("cuda:0")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)


def _values(w, fmt):
    codes, scales = w
    return [uq.dequant_mx((c, s), fmt, dtype=torch.float32).double().cpu().numpy() for c, s in zip(codes, scales)]


@pytest.mark.parametrize("fmt", ["MXFP4", "NVFP4"])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 4, 2, 256, 320), (37, 6, 3, 512, 384), (600, 4, 2, 256, 512)])
def test_layer(fmt, T, E, k, H, F):
    g = torch.Generator().manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g)                                    # noqa: E731
    gate, up, down = (ex.quantize_weights((rnd(E, n, kk) * kk ** -0.5).bfloat16().to(DEV), fmt)
                      for n, kk in ((F, H), (F, H), (H, F)))
    x, router = rnd(T, H).bfloat16().to(DEV), (rnd(E, H) * H ** -0.5).to(DEV)
    ids, weights = ex.route(x, router, k)
    y = ex.moe_layer(x, ids, weights, gate, up, down, fmt)
    assert torch.equal(y, ex.moe_layer(x, ids, weights, gate, up, down, fmt))

    order, pos, off = omoe.sort(ids.cpu().numpy(), E)
    offd, posd = torch.from_numpy(off).to(DEV), torch.from_numpy(pos).to(DEV)
    h = uq.gemm_mx_grouped(uq.quantize_mx(x, fmt, offsets=offd, pos=posd), gate, offd, fmt, up=up)
    xv = omoe.gather(omx.values(*omx.quantize(x.float().cpu().numpy(), fmt), fmt), pos)
    hf = h.float().cpu().numpy()
    hv = omx.values(*omx.quantize(hf, fmt), fmt)
    G, U, D = (_values(w, fmt) for w in (gate, up, down))
    rows, tol = np.zeros((T * k, H)), np.zeros((T * k, H))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        gg, bg = omx.product(xv[s], G[e])
        uu, bu = omx.product(xv[s], U[e])
        silu = gg / (1 + np.exp(-gg))
        acc = H * 2.0 ** -23
        want = silu * uu
        lim = acc * (1.1 * bg * np.abs(uu) + np.abs(silu) * bu) + 1.1 * acc * acc * bg * bu + 2.0 ** -20 * np.abs(want)
        assert np.all(np.abs(hf[s] - want) <= lim + 2.0 ** -8 * (np.abs(want) + lim) + 2.0 ** -25)
        rows[s], b = omx.product(hv[s], D[e])
        tol[s] = F * 2.0 ** -23 * b
        tol[s] += 2.0 ** -8 * (np.abs(rows[s]) + tol[s])
    w = weights.cpu().numpy()
    want, lim = omoe.combine(rows, pos, w), omoe.combine(tol + 2.0 ** -22 * np.abs(rows), pos, w)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= lim + 2.0 ** -8 * (np.abs(want) + lim) + 2.0 ** -25)
    assert uq.device_fault() == 0
