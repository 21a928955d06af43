"""The 64-bit forms of the feed-forward operators (oracle/ffn.py): their slopes
and gradients against differences, their activations against other ways to write
them, and their bounds against a simulation of the roundings they count."""
import math

import numpy as np
import pytest

import oracle
from oracle import ffn


@pytest.mark.parametrize("name", ffn.ACTS)
def test_slopes_are_the_differences_of_the_activations(name):
    z = np.linspace(-9, 9, 721) + 1e-3     # (not at relu's kink)
    h = 1e-5
    d = (ffn.act(z + h, name)[0] - ffn.act(z - h, name)[0]) / (2 * h)
    # central differences: h^2/6 of the third derivative (below 4), and 1e-16 / h
    assert np.abs(d - ffn.slope(z, name)[0]).max() < 1e-9


def test_activations_as_usually_written():
    z = np.linspace(-6, 6, 241)
    assert np.allclose(ffn.act(z, "silu")[0], z / (1 + np.exp(-z)), rtol=1e-13)
    assert np.allclose(ffn.act(z, "gelu")[0], 0.5 * z * (1 + np.vectorize(math.erf)(z / math.sqrt(2))), rtol=1e-9, atol=1e-15)
    assert np.allclose(ffn.act(z, "gelu_tanh")[0],
                       0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))), rtol=1e-9, atol=1e-12)
    assert np.array_equal(ffn.act(z, "relu")[0], np.where(z > 0, z, 0)) and np.array_equal(ffn.act(z, "none")[0], z)


def weights(rng, N, K):
    return oracle.quantize_weight((rng.standard_normal((N, K)) * 0.05).astype(np.float16))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", ffn.ACTS)
def test_gradients_are_the_differences_of_the_product(gated, name):
    """dX and dbias against differences of the smooth product X (Wq sW)^T + b (whose
    gradient the operators are defined to give)."""
    rng = np.random.default_rng(5)
    T, K, F = 4, 32, 6
    N = 2 * F if gated else F
    Wq, sW = weights(rng, N, K)
    W = Wq.astype(np.float64) * sW.astype(np.float64)[:, None]
    X, b = rng.standard_normal((T, K)), rng.standard_normal(N)
    dY = rng.standard_normal((T, F)).astype(np.float16)

    def value(X, b):
        z = X @ W.T + b
        y = ffn.act(z[:, :F], name)[0] * z[:, F:] if gated else ffn.act(z, name)[0]
        return (dY.astype(np.float64) * y).sum()

    pre = X @ W.T + b
    r = ffn.backward(dY, pre, Wq, sW, name, gated)
    h = 1e-5
    for _ in range(6):
        V, c = rng.standard_normal(X.shape), rng.standard_normal(N)
        dx = (value(X + h * V, b) - value(X - h * V, b)) / (2 * h)
        db = (value(X, b + h * c) - value(X, b - h * c)) / (2 * h)
        assert abs(dx - (r["dX"][0] * V).sum()) < 1e-7 * max(1, abs(dx))
        assert abs(db - (r["dbias"][0] * c).sum()) < 1e-7 * max(1, abs(db))


def half(x):
    return x.astype(np.float16).astype(np.float64)


def test_the_bounds_hold_for_the_roundings_and_not_for_mistakes():
    rng = np.random.default_rng(6)
    T, K, F = 40, 96, 50
    Wq, sW = weights(rng, 2 * F, K)
    pre = rng.standard_normal((T, 2 * F)).astype(np.float16)
    dH = rng.standard_normal((T, F)).astype(np.float16)
    r = ffn.backward(dH, pre, Wq, sW, "silu", True)
    z, s = ffn.grad_pre(dH, pre, "silu", True)[0], sW.astype(np.float64)
    a = z * s
    unit = 2.0 ** (14 - np.floor(np.log2(np.abs(a).max(axis=1, keepdims=True))))
    dX = half(half(a * unit) @ Wq.astype(np.float64) / unit)
    assert ffn.check(dX, r["dX"], "dX") is None
    assert np.linalg.norm(dX - r["dX"][0]) < 1.2 * r["dX_norm"]
    # mistakes: gate and up exchanged, a dropped row of the weight, no slope, scales left out of one row
    swapped = np.concatenate([a[:, F:], a[:, :F]], axis=1)
    for wrong in (swapped, np.where(np.arange(2 * F) == 7, 0, a), a + np.where(np.arange(2 * F) == 3, 0.03 * a, 0)):
        assert np.linalg.norm(wrong @ Wq.astype(np.float64) - r["dX"][0]) > 1.5 * r["dX_norm"]

    X = rng.standard_normal((T, K)).astype(np.float16)
    X[:, 5] *= 20
    b = rng.standard_normal(2 * F).astype(np.float16)
    (h, eh), (p, ep) = ffn.gated_linear(X, Wq, sW, 6.0, b, "gelu")
    assert ffn.check(half(h), (h, eh), "H") is None and ffn.check(half(p), (p, ep), "pre") is None
    assert ffn.check(half(h * 1.002), (h, eh), "H") is not None
    assert ffn.check(half(ffn.gated_linear(X, Wq, sW, 6.0, None, "gelu")[0][0]), (h, eh), "H") is not None
