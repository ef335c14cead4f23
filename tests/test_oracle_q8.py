"""The oracle of the 8-bit rows, the norm and the router: hand-worked values, and gradients against central differences."""
import numpy as np
import pytest

from oracle import q8, router


def test_quantize_worked():
    q, s = q8.quantize(np.array([[0, 127, -63.5, 0.5, 1.5], [0, 0, 0, 0, 0], [1, np.nan, 0, 0, 0], [2, np.inf, 0, 0, 0]]))
    assert np.array_equal(q, [[0, 127, -64, 0, 2], [0] * 5, [0] * 5, [0] * 5])      # ties to even
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3])


def test_norm_worked():
    y, s = q8.rmsnorm(np.array([[3.0, -4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), -8 / np.sqrt(12.5)]]) and np.allclose(s, 8 / np.sqrt(12.5) / 127)


def test_product_worked():
    y, mag = q8.gemm(np.array([[1, -2]]), np.array([0.5]), np.array([[3, 4], [127, -128]]), np.array([2.0, 1.0]))
    assert np.array_equal(y, [[-5.0, 191.5]]) and np.array_equal(mag, [[5.0, 191.5]])


def test_router_worked():
    x = np.array([[0.0, 1.0, 1.0, -np.inf], [2.0, np.nan, 1.0, 0.0], [-np.inf] * 4])
    assert np.array_equal(router.choose(x, 3), [[1, 2, 0], [0, 2, 3], [-1, -1, -1]])
    assert np.array_equal(router.choose(x, 4), [[1, 2, 0, -1], [0, 2, 3, 1], [-1] * 4])
    bias = np.array([1.0, 0.0, -np.inf, 0.0])
    assert np.array_equal(router.choose(x, 2, "sigmoid", bias), [[0, 1], [0, 3], [-1, -1]])
    # groups (0, 1) and (2, 3): by the best member the first (tie, lower index); by the best two the first
    assert np.array_equal(router.choose(x[:1], 2, "softmax", None, 2, 1, 1), [[1, 0]])
    assert np.array_equal(router.choose(np.array([[3.0, -9, 2.9, 2.9]]), 2, "sigmoid", None, 2, 1, 2), [[2, 3]])
    w = router.weights(np.array([[0.0, np.log(3)]]), np.array([[1, 0, -1]]), "softmax", False, 2.0)
    assert np.allclose(w, [[1.5, 0.5, 0]])


def _differences(f, x, dy, h=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = ((f(a) - f(b)) * dy).sum() / (2 * h)
    return out


@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_gradient_is_the_difference_quotient(with_dh):
    g = np.random.default_rng(1)
    h, gamma, dy = g.normal(size=(3, 7)), g.normal(size=7), g.normal(size=(3, 7))
    dh = g.normal(size=(3, 7)) if with_dh else None
    dx, dg = q8.rmsnorm_grad(dy, h, gamma, 1e-3, dh)
    want = _differences(lambda v: q8.rmsnorm(v, gamma, 1e-3)[0], h, dy) + (dh if with_dh else 0)
    assert np.allclose(dx, want, atol=1e-8)
    assert np.allclose(dg, _differences(lambda v: q8.rmsnorm(h, v, 1e-3)[0], gamma, dy), atol=1e-8)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_gradient_is_the_difference_quotient(score, renorm):
    g = np.random.default_rng(2)
    x, dw = g.normal(size=(4, 6)), g.normal(size=(4, 3))
    ids = np.array([[0, 1, 2], [5, -1, 3], [2, 2, 4], [-1, -1, 9]], np.int32)

    def f(v):
        return router.weights(v, np.where((ids >= 0) & (ids < 6), ids, -1), score, renorm, 2.5)
    dx, mag = router.grad(x, ids, dw, score, renorm, 2.5)
    assert np.allclose(dx, _differences(f, x, dw), atol=1e-8)
    assert np.all(np.abs(dx) <= mag + 1e-12)
