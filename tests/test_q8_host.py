"""Refusals of the 8-bit row, norm and router calls, answered on the host before any CUDA call, and what they launch on the
stand-in for the CUDA runtime."""
import ctypes

import pytest

from tests.fake_cuda import Launch, load

INVALID, UNSUPPORTED, ALIGN = 1, 2, 3
BIG = 0x7FFFF000                                 # past 2^31 - 4097


@pytest.fixture(scope="module")
def L():
    from gemm_uq_gb300.build import build
    build()
    import gemm_uq_gb300 as uq
    return uq.lib()


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_uint8 * 256)()
    base = ctypes.addressof(buf)
    yield base + (-base) % 16
    del buf


def _bad(L, status, got):
    assert got == status and len(L.uq_last_error()) > 0


def test_quantize_and_dequant(L, p):
    q, d = L.uq_quantize_q8, L.uq_dequant_q8
    assert q(None, 0, 8, None, None, 0, 8, None) == 0 and d(None, None, None, 0, 0, 8, None) == 0
    assert d(None, None, None, 0, 3, 0, None) == 0
    _bad(L, INVALID, q(None, 0, 8, None, None, 3, 0, None))   # rows without elements have scales, too
    _bad(L, INVALID, q(p, 0, 8, p, p, -1, 8, None))
    _bad(L, INVALID, q(p, 3, 8, p, p, 1, 8, None))
    _bad(L, INVALID, q(p, 0, 7, p, p, 1, 8, None))            # rows closer than they are long
    _bad(L, INVALID, q(None, 0, 8, p, p, 1, 8, None))
    _bad(L, INVALID, q(p, 0, 8, None, p, 1, 8, None))
    _bad(L, INVALID, q(p, 0, 8, p, None, 1, 8, None))
    _bad(L, UNSUPPORTED, q(p, 0, 8, p, p, BIG, 8, None))
    _bad(L, UNSUPPORTED, q(p, 0, BIG, p, p, 1, BIG, None))
    _bad(L, ALIGN, q(p + 2, 0, 8, p, p, 1, 8, None))
    _bad(L, ALIGN, q(p, 0, 8, p + 8, p, 1, 8, None))
    _bad(L, INVALID, d(p, p, p, 5, 1, 8, None))
    _bad(L, INVALID, d(p, p, None, 0, 1, 8, None))
    _bad(L, ALIGN, d(p, p + 4, p, 0, 1, 8, None))


def test_norm(L, p):
    f, o = L.uq_rmsnorm_q8, p + 64
    ok = [p, None, p, 0, 8, None, o, p + 128, p + 160, 2, 8, 1e-5, None]

    def call(**kw):
        names = ["x", "residual", "gamma", "type", "ldx", "h", "y", "codes", "scales", "rows", "D", "eps", "stream"]
        a = dict(zip(names, ok))
        a.update(kw)
        return f(*(a[k] for k in names))
    assert call(rows=0, x=None) == 0 and call(D=0, ldx=0, x=None) == 0
    for kw in ({"rows": -1}, {"D": -1}, {"type": 4}, {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"x": None},
               {"gamma": None}, {"codes": None}, {"scales": None}, {"ldx": 7}, {"y": None, "codes": None, "scales": None},
               {"h": o}, {"h": p, "ldx": 16}, {"y": p, "ldx": 16}):
        _bad(L, INVALID, call(**kw))
    for kw in ({"x": p + 2}, {"residual": p + 2}, {"gamma": p + 2}, {"h": p + 4}, {"y": o + 8}, {"codes": p + 136}, {"scales": p + 164}):
        _bad(L, ALIGN, call(**kw))
    _bad(L, UNSUPPORTED, call(rows=BIG))
    _bad(L, UNSUPPORTED, call(D=BIG, ldx=BIG))


def test_norm_gradient(L, p):
    f, o = L.uq_rmsnorm_grad, p + 64
    assert f(None, None, None, None, 0, None, None, 4, 0, 1e-5, None) == 0
    _bad(L, INVALID, f(p, p, p, None, 0, o, None, 2, 8, 1e-5, None))
    _bad(L, INVALID, f(p, p, p, None, 0, o, None, 0, 8, 1e-5, None))          # dgamma is written for no rows, too
    for a in ((None, p, p, None, 0, o, o), (p, None, p, None, 0, o, o), (p, p, None, None, 0, o, o), (p, p, p, None, 0, None, o),
              (p, p, p, None, 3, o, o), (o, p, p, None, 0, p, o)):
        _bad(L, INVALID, f(*a, 2, 8, 1e-5, None))
    _bad(L, INVALID, f(p, p, p, None, 0, o, o, 2, 8, -1e-5, None))
    for a in ((p + 2, p, p, None, 0, o, o), (p, p + 2, p, None, 0, o, o), (p, p, p, p + 2, 0, o, o), (p, p, p, None, 0, o, o + 4)):
        _bad(L, ALIGN, f(*a, 2, 8, 1e-5, None))
    _bad(L, UNSUPPORTED, f(p, p, p, None, 0, o, o, BIG, 8, 1e-5, None))


def test_product(L, p):
    f, o = L.uq_gemm_w8a8, p + 64
    assert f(None, 0, 0, None, None, None, None, 0, 0, 8, 64, None) == 0
    assert f(None, 0, 0, None, None, None, None, 0, 8, 0, 64, None) == 0
    for a in ((p, 0, 64, None, p, p, o, 0, -1, 8, 64), (p, 0, 64, None, p, p, o, 0, 1, 8, 40), (p, 0, 64, None, p, p, o, 3, 1, 8, 64),
              (p, 3, 64, None, p, p, o, 0, 1, 8, 64), (p, 0, 63, None, p, p, o, 0, 1, 8, 64), (None, 0, 64, None, p, p, o, 0, 1, 8, 64),
              (p, 0, 64, None, None, p, o, 0, 1, 8, 64), (p, 0, 64, None, p, None, o, 0, 1, 8, 64), (p, 0, 64, p, p, p, None, 0, 1, 8, 64)):
        _bad(L, INVALID, f(*a, None))
    for a in ((p, 0, 64, None, p, p, o, 0, 1, 8, 131072), (p, 0, 64, p, p, p, o, 0, BIG, 8, 64), (p, 0, 64, p, p, p, o, 0, 8, BIG, 64),
              (p, 0, 64, p, p, p, o, 0, 0x7FFFEFFF, 0x7FFFEFFF, 64)):
        _bad(L, UNSUPPORTED, f(*a, None))
    for a in ((p + 2, 0, 64, None, p, p, o, 0, 1, 8, 64), (p, 0, 64, p + 4, p, p, o, 0, 1, 8, 64), (p, 0, 64, p, p + 8, p, o, 0, 1, 8, 64),
              (p, 0, 64, p, p, p + 4, o, 0, 1, 8, 64), (p, 0, 64, p, p, p, o + 2, 0, 1, 8, 64)):
        _bad(L, ALIGN, f(*a, None))


def test_router(L, p):
    f, o = L.uq_moe_route, p + 64

    def call(**kw):
        a = dict(logits=p, type=0, bias=None, score=0, groups=1, top_groups=1, group_top=1, renorm=1, scale=1.0, ids=o, weights=p + 128,
                 T=2, experts=8, topk=2, stream=None)
        a.update(kw)
        return f(*a.values())
    assert call(T=0, logits=None) == 0 and call(topk=0, ids=None) == 0
    for kw in ({"T": -1}, {"topk": -1}, {"experts": 0}, {"type": 7}, {"score": 2}, {"scale": float("inf")}, {"scale": float("nan")},
               {"groups": 0}, {"groups": 3}, {"groups": 2, "top_groups": 0}, {"groups": 2, "top_groups": 3}, {"group_top": 0}, {"group_top": 3},
               {"topk": 9}, {"groups": 4, "topk": 3}, {"T": 0x7FFFFFFF}, {"logits": None}, {"ids": None}, {"weights": None}):
        _bad(L, INVALID, call(**kw))
    for kw in ({"experts": 1025}, {"experts": 64, "topk": 33}, {"experts": 128, "groups": 64, "top_groups": 8}):
        _bad(L, UNSUPPORTED, call(**kw))
    for kw in ({"logits": p + 2}, {"bias": p + 4}, {"ids": o + 4}, {"weights": o + 8}):
        _bad(L, ALIGN, call(**kw))


def test_router_gradient(L, p):
    f, o = L.uq_moe_route_grad, p + 64

    def call(**kw):
        a = dict(logits=p, type=0, ids=p, dweights=p, score=0, renorm=1, scale=1.0, dlogits=o, T=2, experts=8, topk=2, stream=None)
        a.update(kw)
        return f(*a.values())
    assert call(T=0, logits=None) == 0
    for kw in ({"T": -1}, {"topk": -1}, {"experts": 0}, {"type": -1}, {"score": -1}, {"scale": float("-inf")}, {"logits": None}, {"ids": None},
               {"dweights": None}, {"dlogits": None}, {"dlogits": p}):
        _bad(L, INVALID, call(**kw))
    for kw in ({"experts": 2000}, {"topk": 40}):
        _bad(L, UNSUPPORTED, call(**kw))
    for kw in ({"logits": p + 2}, {"ids": p + 4}, {"dweights": p + 4}, {"dlogits": o + 8}):
        _bad(L, ALIGN, call(**kw))


def test_the_binding_refuses_what_it_cannot_pass():
    torch = pytest.importorskip("torch")
    import gemm_uq_gb300 as uq
    x, w = torch.zeros(4, 32), (torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8))
    for call in (lambda: uq.quantize_q8(x), lambda: uq.dequant_q8(w), lambda: uq.rmsnorm_q8(x, torch.ones(32), 1e-5),
                 lambda: uq.rmsnorm_grad(x, x, torch.ones(32), 1e-5), lambda: uq.gemm_w8a8(x, w), lambda: uq.moe_route(x, 2),
                 lambda: uq.rmsnorm_q8(x, torch.ones(31), 1e-5), lambda: uq.gemm_w8a8(x, (w[0], w[1][:7])),
                 lambda: uq.moe_route(x, 2, bias=torch.zeros(31)),
                 lambda: uq.moe_route_grad(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 3))):
        with pytest.raises((AssertionError, RuntimeError)):       # CPU tensors among them
            call()


def test_no_memory_is_an_error_and_nothing_is_launched(tmp_path):
    f = load(tmp_path)
    a = f.at
    f.launches(lambda: f.lib.uq_quantize_q8(a, 0, 64, a, a, 4, 64, None))          # the device's words
    f.lib.fake_set_no_memory(1)
    f.lib.fake_clear()
    assert f.lib.uq_gemm_w8a8(a, 0, 64, None, a, a, a, 0, 7, 64, 64, None) == 5
    assert f.lib.uq_gemm_w8a8(a, 0, 64, None, a, a, a, 0, 40, 64, 64, None) == 5
    assert f.lib.uq_rmsnorm_grad(a, a, a, None, 0, a + 256, a, 4, 64, 1e-5, None) == 5
    assert f.lib.fake_launch_count() == 0
    f.lib.fake_set_no_memory(0)
    assert len(f.launches(lambda: f.lib.uq_gemm_w8a8(a, 0, 64, None, a, a, a, 0, 7, 64, 64, None))) == 2
    assert len(f.launches(lambda: f.lib.uq_rmsnorm_grad(a, a, a, None, 0, a + 256, a, 4, 64, 1e-5, None))) == 2


def test_calls_of_several_threads_on_one_stream_do_not_mix(tmp_path):
    """The launches of a call that hand each other the stream's workspace follow one another, whichever threads call."""
    import threading
    f = load(tmp_path)
    a, L = f.at, f.lib
    calls = [lambda: L.uq_gemm_w8a8(a, 0, 64, None, a, a, a, 0, 7, 64, 64, None),
             lambda: L.uq_gemm_w8a8(a, 0, 64, None, a, a, a, 0, 40, 64, 64, None),
             lambda: L.uq_gemm_w8a8(a, 0, 64, a, a, a, a, 0, 50, 64, 64, None),
             lambda: L.uq_rmsnorm_grad(a, a, a, None, 0, a + 256, a, 4, 64, 1e-5, None),
             lambda: L.uq_gemm_mx(a, 0, 64, None, 1.0, a, a, a, 0, 40, 64, 64, 0, 1.0, None),
             lambda: L.uq_gemm_w4a8(a, a, a, None, a, 11, 64, 256, 64, 0, None),
             lambda: L.uq_gemm(a, a, a, None, a, 20, 64, 256, 256, 5, None),
             lambda: L.uq_gemm_gated(a, a, a, None, a, a, None, a, 20, 64, 256, 64, 0, None)]
    alone = [tuple(f.launches(c)) for c in calls]
    assert all(len(s) > 1 for s in alone)
    f.lib.fake_clear()
    bad = []

    def many(i):
        for _ in range(400):
            if calls[i]() != 0:
                bad.append(i)
    threads = [threading.Thread(target=many, args=(i % len(calls),)) for i in range(2 * len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    n = f.lib.fake_launch_count()
    assert n == 800 * sum(len(s) for s in alone)
    seen, at = [], 0
    for i in range(n):
        v = [ctypes.c_uint() for _ in range(3)] + [ctypes.c_int()]
        seen.append(Launch(f.lib.fake_launch(i, *(ctypes.byref(x) for x in v)).decode(), *(x.value for x in v)))
    while at < n:
        whole = [s for s in alone if tuple(seen[at:at + len(s)]) == s]
        assert whole, f"launches of different calls follow one another: {[x.kernel[:80] for x in seen[at:at + 4]]}"
        at += len(whole[0])
