"""The feed-forward operators of the int8 linear layer in 64 bits, with the worst
that the roundings of a 16-bit implementation can do to each value.

Written from the definitions, on the oracle's codes, scales and int32 sums:

    Z = acc sX sW + sum_O X (Wq sW) + bias
    Y = act(Z) + residual                      H = act(G) U, [G | U] = Z
    dZ = dY act'(Z)  or  [dH U act'(G) | dH act(G)]
    dX = dZ (Wq sW),  dbias = sum_t dZ

Every function returns (value, bound) pairs.  With u = 2^-24, half a step of
fp32, and h = 2^-11, half a step of fp16 (2^-25 below its normal range):

* Z: the int32 sum's conversion, the scales' products and the bias' addition
  round once each, and every outlier term once as it is added, to a partial sum of at
  most |main| + S, S the sum of the terms' magnitudes (twice, for the matrix
  unit's own alignment): u ((3 + 2 nO) (|main| + S) + 2 |Z|).
* act, relative: the exponent of the exponential is rounded three times, which
  costs 3 u |exponent| (below 2^-18 up to an exponent of 2^30 ~ e^20; beyond that
  the value is below 2^-25), then a few units: 2^-17 |act|, and 2^-32 |z| for
  what lies beyond.  Its slope is at most 1.13: 1.2 times Z's bound comes through.
* act': s + z s (1 - s) x' or P + z p; 1 - s is off by u while s < 1, and z x' is at
  most 2^5 as long as s < 1 in fp32; with the terms' own 2^-17: 2^-17 (1 + terms).
* dX: an element A = dZ sW of a row is rounded to fp16 in units of the row's largest:
  h |A|, at least 2^-25 2^-14 of the largest; the sum of N products in fp32:
  (N + 2) u sum |A q|; then the fp16 result.
"""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erfc, expit

import oracle

U, H = 2.0 ** -24, 2.0 ** -11
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _gelu_tanh_x(z):
    k = 2 * math.sqrt(2 / math.pi)
    return k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z ** 2)


def act(z, name):
    """(value, bound) of the activation at exact z."""
    if name == "none":
        return z, np.zeros_like(z)
    if name == "relu":
        return np.maximum(z, 0), np.zeros_like(z)
    if name == "silu":
        v = z * expit(z)
    elif name == "gelu":
        v = z * 0.5 * erfc(-z * math.sqrt(0.5))
    else:
        v = z * expit(_gelu_tanh_x(z)[0])
    return v, 2.0 ** -17 * np.abs(v) + 2.0 ** -32 * np.abs(z)


def slope(z, name):
    """(value, bound) of the activation's derivative (0 for relu at 0)."""
    if name == "none":
        return np.ones_like(z), np.zeros_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64), np.zeros_like(z)
    if name == "gelu":
        a, b = 0.5 * erfc(-z * math.sqrt(0.5)), z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    else:
        x, x1 = (z, np.ones_like(z)) if name == "silu" else _gelu_tanh_x(z)
        a, b = expit(x), z * expit(x) * expit(-x) * x1
    return a + b, 2.0 ** -17 * (1 + np.abs(a) + np.abs(b))


def rounded(v, e):
    """The bound after one rounding to fp16 of a value that is off by e at most."""
    return e + H * (np.abs(v) + e) + 2.0 ** -25


def product(X, Wq, sW, threshold, bias=None):
    """(Z, bound)."""
    flags, idx = oracle.detect_outliers(X, threshold)
    Xq, sX = oracle.quantize_rows(X, flags)
    T, K = X.shape
    if K:
        main = oracle.int8_gemm(Xq, Wq).astype(np.float64)
    else:
        main = np.zeros((T, Wq.shape[0]))
    s = sW.astype(np.float64)
    main *= sX[:T].astype(np.float64)[:, None] * s
    xo, wo = X[:, idx].astype(np.float64), Wq[:, idx].astype(np.float64) * s[:, None]
    z = main + xo @ wo.T
    mag = np.abs(main) + np.abs(xo) @ np.abs(wo).T
    if bias is not None:
        z = z + bias.astype(np.float64)
    return z, U * ((3 + 2 * len(idx)) * mag + 2 * np.abs(z))


def linear_epilogue(X, Wq, sW, threshold, bias=None, activation="none", residual=None):
    """((Y, bound), (pre, bound)), both after their rounding to fp16."""
    z, ez = product(X, Wq, sW, threshold, bias)
    y, ey = act(z, activation)
    ey = ey + 1.2 * ez
    if residual is not None:
        y = y + residual.astype(np.float64)
        ey = ey + U * (np.abs(y) + ey)
    return (y, rounded(y, ey)), (z, rounded(z, ez))


def gated_linear(X, Wq, sW, threshold, bias=None, activation="silu"):
    z, ez = product(X, Wq, sW, threshold, bias)
    F = Wq.shape[0] // 2
    a, ea = act(z[:, :F], activation)
    ea = ea + 1.2 * ez[:, :F]
    u, eu = z[:, F:], ez[:, F:]
    h = a * u
    eh = np.abs(u) * ea + np.abs(a) * eu + ea * eu + U * np.abs(h)
    return (h, rounded(h, eh)), (z, rounded(z, ez))


def grad_pre(dY, pre, activation, gated):
    """(dZ, bound) in fp32, before any rounding to fp16."""
    d = dY.astype(np.float64)
    if not gated:
        if activation == "none":
            return d, np.zeros_like(d)
        s, es = slope(pre.astype(np.float64), activation)
        z = d * s
        return z, np.abs(d) * es + 2 * U * np.abs(z)
    z = pre.astype(np.float64)
    F = z.shape[1] // 2
    g, u = z[:, :F], z[:, F:]
    v, ev = act(g, activation)
    s, es = slope(g, activation)
    dg, du = d * u * s, d * v
    return (np.concatenate([dg, du], axis=1),
            np.concatenate([np.abs(d * u) * es + 3 * U * np.abs(dg), np.abs(d) * ev + 2 * U * np.abs(du)], axis=1))


def backward(dY, pre, Wq, sW, activation="none", gated=False):
    """dict of (value, bound): dX, grad_pre (both after their rounding to fp16) and
    dbias; and dX_norm, the norm that dX's errors have as independent ones, each
    uniform within its rounding's half step."""
    z, ez = grad_pre(dY, pre, activation, gated)
    T, N = z.shape
    s, q = sW.astype(np.float64), Wq.astype(np.float64)
    a = z * s
    ea = ez * s + 2 * U * np.abs(a)
    top = np.abs(a).max(axis=1, initial=0)[:, None]
    aq = np.abs(q)
    dX = a @ q
    worst = (ea + H * (np.abs(a) + ea) + 2.0 ** -39 * top) @ aq + (N + 2) * U * (np.abs(a) @ aq)
    # the sum over tokens: T additions, whatever their order
    dbias = z.sum(axis=0)
    return dict(dX=(dX, rounded(dX, worst)), grad_pre=(z, rounded(z, ez)),
                dbias=(dbias, ez.sum(axis=0) + (T + 2) * U * (np.abs(z) + ez).sum(axis=0)),
                dX_norm=float(np.sqrt((((H * a) ** 2 @ q ** 2 + (H * dX) ** 2) / 3).sum())))


def check(got, want, what):
    """None, or the first element that is off by more than its bound.  An fp16 value
    is an infinity from 65520 on (half way from the largest, 65504, to 2^16)."""
    v, e = want
    half = np.asarray(got).dtype == np.float16
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == v.shape, (what, got.shape, v.shape)
    with np.errstate(invalid="ignore"):
        d = np.abs(got - v)
    over = half & np.isinf(got) & (np.sign(got) == np.sign(v)) & (np.abs(v) + e >= 65520)
    bad = ~((d <= e) | over)
    if not bad.any():
        return None
    i = tuple(int(x) for x in np.argwhere(bad)[0])
    return f"{what}{list(i)}: {got[i]!r}, exact {v[i]!r}, off by {d[i]:.3e}, bound {e[i]:.3e}; {int(bad.sum())} of {bad.size}"
