"""How far the attention over the int8 key/value cache may be off, row by row,
from what its kernels round.  For tests; fp64, nothing shared with the HIP path.

With z the scores, w = softmax(z), v the values, O = w v, all from the codes:

* A query is rounded to integers of 1/16256 of its largest value: each of its D
  values is off by at most d = max|q| / 32512, independently of the others, so
  dz[t] = scale sum_j k[t, j] e[j], |e[j]| <= d.  To first order
  dO = sum_t w[t] (v[t] - O) dz[t].
* A probability p is rounded to fp16: by at most 2^-11 of itself (in two parts
  2^-22), or by 2^-25 where it is subnormal.  In the units of p the sum over
  the row is at least S = sum_t exp(z[t] - max z), as the maximum that p is
  taken against is at most the row's, and a value is its code times at most the
  largest value scale of the sequence: dO <= 2^-25 sum_t |code[t]| vmax / S.
* The result is rounded to 16 bits: half a step.
* fp32: z is off by 2^-22 of the row's largest |z| and the exponential by 2^-22
  (three roundings each), and a sum of n terms by n 2^-24 of the terms' sizes.

``worst`` adds the bounds up.  ``spread`` takes the roundings as the independent
errors that they are: e[j] uniform in +-d (variance d^2 / 3), the relative error
of a number rounded to 11 bits of variance 2^-22 / 3 * mean(1 / m^2) = 0.1803 2^-22
over mantissas m in [1, 2) of density 1 / (m ln 2), subnormal ones 2^-50 / 3; the
result's own rounding is known.
"""
from __future__ import annotations

import numpy as np

from . import kv as okv


class Rows:
    """Per (token, query head): O, worst, own (error of O's rounding), variance of
    what is before it, fp32 (what is not random): [tokens, q_heads, dim]; lse,
    worst_lse [tokens, q_heads].  NaN in rows of no sequence."""

    def __init__(self, T, Hq, D):
        for n in ("O", "worst", "own", "variance", "fp32"):
            setattr(self, n, np.full((T, Hq, D), np.nan))
        self.lse, self.worst_lse = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)


def rounded(x, eps):
    """x to the 16-bit type of this eps (2^-10: fp16, 2^-7: bf16), nearest even."""
    if eps == 2.0**-10:
        return x.astype(np.float16).astype(np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def values(c: okv.Cache, row, n):
    """Codes, scales and presence of the first n tokens of a table row."""
    t = np.arange(n)
    p = np.asarray(row)[t // c.page].astype(np.int64)
    there = (p >= 0) & (p < c.pages)
    p = np.where(there, p, 0)
    k, v = (x[p, :, t % c.page].astype(np.float64) for x in (c.k, c.v))
    ks, vs = (np.where(there[:, None], x[p], 0).astype(np.float64) for x in (c.ks, c.vs))
    k[~there], v[~there] = 0, 0
    return k, v, ks, vs, there


def rows(c: okv.Cache, Q, scale, q_start, kv_len, table, rope=None, causal=True, window=0, eps=2.0**-10, two=False):
    """Q fp32 [tokens, q_heads, dim]; two: probabilities in two fp16 parts."""
    T, Hq, D = Q.shape
    G = Hq // c.heads
    r = Rows(T, Hq, D)
    relative = 2.0**-22 if two else 2.0**-11
    spread = 0.1803 * relative**2
    for s in range(len(kv_len)):
        q0, n, L = int(q_start[s]), int(q_start[s + 1] - q_start[s]), int(kv_len[s])
        kc, vc, ks, vs, there = values(c, table[s], L)
        t = np.arange(L)
        for i in range(n):
            p = L - n + i
            see = there.copy()
            if causal:
                see &= t <= p
            if window:
                see &= t > p - window
            for x in (r.O, r.worst, r.own, r.variance, r.fp32, r.worst_lse):
                x[q0 + i] = 0
            r.lse[q0 + i] = -np.inf
            if not see.any():
                continue
            q = okv.rotate(Q[q0 + i].astype(np.float32), max(p, 0), rope).astype(np.float64)
            for h in range(c.heads):
                k, v = kc[see, h] * ks[see, h][:, None], vc[see, h] * vs[see, h][:, None]
                code = np.abs(vc[see, h])
                vmax = vs[there, h].max()
                for j in range(h * G, (h + 1) * G):
                    z = scale * (k @ q[j])
                    e = np.exp(z - z.max())
                    S = e.sum()
                    w = e / S
                    O = w @ v
                    d = np.abs(q[j]).max() / 32512
                    away = np.abs(v - O)
                    A, W = w @ np.abs(v), w @ away
                    fp = (np.abs(z).max() + 1) * 2.0**-22
                    Z = scale * d * np.abs(k).sum(1).max()
                    inner = (1 + Z) * Z * W + fp * W + relative * A + 2.0**-25 * code.sum(0) * vmax / S + len(z) * 2.0**-24 * A
                    at = q0 + i, j
                    r.O[at], r.lse[at] = O, z.max() + np.log(S)
                    r.worst[at] = inner + (np.abs(O) + inner) * eps / 2 + 2.0**-25
                    r.own[at] = rounded(O, eps) - O
                    M = (k * w[:, None]).T @ (v - O)                # [j, dim]: what an error of q[j] gives
                    r.variance[at] = ((scale * d) ** 2 / 3 * (M**2).sum(0) + spread * (w**2 @ v**2)
                                      + (2.0**-25 * vmax / S) ** 2 / 3 * (code**2).sum(0))
                    # (fp32 sums: a term's roundings go both ways, sqrt(n) of them)
                    r.fp32[at] = fp * W + np.sqrt(len(z)) * 2.0**-24 * A + 2.0**-25
                    r.worst_lse[at] = Z + fp + len(z) * 2.0**-24 + 2.0**-22 * abs(r.lse[at])
    return r


def limit(r: Rows):
    """The limit of the norm of all rows' errors own + e.  |e|^2 of a row has a
    deviation of at most sqrt(2) of its mean (that of a single normal number), and
    2 own e one of at most 2 |own| times that of e: the sum over the rows stays
    within five deviations."""
    live = np.isfinite(r.lse)
    own, var = (r.own[live] ** 2).sum(1), r.variance[live].sum(1)
    dev = np.sqrt((2 * var**2 + 4 * own * var).sum())
    return np.sqrt(own.sum() + var.sum() + 5 * dev) + np.sqrt((r.fp32[live] ** 2).sum())


def check(r: Rows, got, lse=None):
    """None, or what is wrong with got [tokens, q_heads, dim] (fp64)."""
    seq = ~np.isnan(r.lse)
    live = np.isfinite(r.lse)
    if got[seq & ~live].any():
        return "a row that sees nothing is not 0"
    err = np.abs(got - r.O)[live]
    if not (err <= r.worst[live]).all():
        return f"an element is off by {(err / r.worst[live]).max():.3g} of its bound"
    norm, most = np.sqrt((err**2).sum()), limit(r)
    if not norm <= most:
        return f"the error's norm is {norm:.4g}, its limit {most:.4g}, the output's norm {np.sqrt((r.O[live]**2).sum()):.4g}"
    if lse is not None:
        if not np.isneginf(lse[seq & ~live]).all():
            return "lse of a row that sees nothing is not -inf"
        err = np.abs(lse[live] - r.lse[live])
        if not (err <= r.worst_lse[live]).all():
            return f"lse is off by {(err / r.worst_lse[live]).max():.3g} of its bound"
    return None
