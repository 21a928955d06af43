"""Plain numpy forms of the int8 key/value cache operators, for tests.

Written from their definitions, one sequence, page and head after another:

* append: x' = rotated x, s = max(fl32(max|x'| / 127), old scale if the page
  has older rows), code = clamp(rne(fl32(x' * r)), -127, 127) with
  r = min(fl32(1 / s), FLT_MAX); older rows are coded again under a larger
  scale.  In fp32, each operation rounded, so codes and scales are exact
  (lowentro.cn "model quantization" notes, Q2 and Q11: symmetric absmax).
* read: fl32(code * scale).
* attention: softmax(scale * q . k) . v in fp64 over the keys a row sees.

Nothing here is shared with the HIP path.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32


class Cache:
    """k, v int8 [pages, heads, page, dim]; ks, vs fp32 [pages, heads]."""

    def __init__(self, k, v, ks, vs):
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.pages, self.heads, self.page, self.dim = k.shape


def rotate(x, pos, rope):
    """x fp32 [heads, dim] at position pos; rope = (cos, sin, interleaved) or None."""
    if rope is None:
        return x
    cos, sin, inter = rope
    R = 2 * cos.shape[1]
    c, s = cos[pos].astype(F32), sin[pos].astype(F32)
    y = x.copy()
    if inter:
        a, b = x[:, 0:R:2], x[:, 1:R:2]
        y[:, 0:R:2] = a * c - b * s
        y[:, 1:R:2] = b * c + a * s
    else:
        a, b = x[:, :R // 2], x[:, R // 2:R]
        y[:, :R // 2] = a * c - b * s
        y[:, R // 2:R] = b * c + a * s
    return y


def codes(x, s):
    if s == 0:
        r = F32(0)
    else:
        with np.errstate(over="ignore"):
            r = min(F32(1) / s, np.finfo(F32).max)
    return np.clip(np.rint((x * F32(r)).astype(F32)), -127, 127).astype(np.int8)


def append(c: Cache, K, V, q_start, kv_len, table, rope=None):
    """K, V fp32 [tokens, heads, dim]; c changes in place."""
    for s in range(len(kv_len)):
        q0, n, L = int(q_start[s]), int(q_start[s + 1] - q_start[s]), int(kv_len[s])
        begin = L - n
        first = max(begin, 0)
        for b in range(first // c.page, -(-L // c.page)):
            lo, hi = max(first, b * c.page), min(L, (b + 1) * c.page)
            p = int(table[s][b])
            if lo >= hi or not 0 <= p < c.pages:
                continue
            off = lo - b * c.page
            for src, q, sc, rot in ((K, c.k, c.ks, rope), (V, c.v, c.vs, None)):
                rows = np.stack([rotate(src[q0 + t - begin].astype(F32), t, rot) for t in range(lo, hi)])
                for h in range(c.heads):
                    old = sc[p, h] if off else F32(0)
                    new = max(F32(np.abs(rows[:, h]).max() / F32(127)), old)
                    if off and new > old:
                        q[p, h, :off] = codes((q[p, h, :off].astype(F32) * old).astype(F32), new)
                    q[p, h, off:off + hi - lo] = codes(rows[:, h], new)
                    sc[p, h] = new


def held(c: Cache, row, t0, t1):
    """(k, v, there) of tokens t0 .. t1 - 1 of a table row: fp32 values [t, heads, dim]."""
    k = np.zeros((t1 - t0, c.heads, c.dim), F32)
    v = np.zeros_like(k)
    there = np.zeros(t1 - t0, bool)
    for t in range(t0, t1):
        p = int(row[t // c.page])
        if t < 0 or not 0 <= p < c.pages:
            continue
        there[t - t0] = True
        k[t - t0] = c.k[p, :, t % c.page].astype(F32) * c.ks[p][:, None]
        v[t - t0] = c.v[p, :, t % c.page].astype(F32) * c.vs[p][:, None]
    return k, v, there


def read(c: Cache, q_start, kv_len, table, tokens):
    """fp32 (K, V) [tokens, heads, dim]; NaN in rows of no sequence."""
    K = np.full((tokens, c.heads, c.dim), np.nan, F32)
    V = K.copy()
    for s in range(len(kv_len)):
        q0, n, L = int(q_start[s]), int(q_start[s + 1] - q_start[s]), int(kv_len[s])
        K[q0:q0 + n] = V[q0:q0 + n] = 0
        lo = max(L - n, 0)
        if L > lo:
            k, v, _ = held(c, table[s], lo, L)
            K[q0 + lo - (L - n):q0 + n], V[q0 + lo - (L - n):q0 + n] = k, v
    return K, V


def attention(c: Cache, Q, scale, q_start, kv_len, table, rope=None, causal=True, window=0):
    """fp64 (O [tokens, q_heads, dim], lse [tokens, q_heads], A, Z): A = sum of the
    weights times |v|, Z = the largest |z| error of a query rounded to 1/32512 of
    its largest value (both for error bounds).  NaN in rows of no sequence."""
    T, Hq, D = Q.shape
    G = Hq // c.heads
    O = np.full((T, Hq, D), np.nan)
    A = O.copy()
    lse = np.full((T, Hq), np.nan)
    Z = np.zeros((T, Hq))
    for s in range(len(kv_len)):
        q0, n, L = int(q_start[s]), int(q_start[s + 1] - q_start[s]), int(kv_len[s])
        k, v, there = held(c, table[s], 0, L)
        k, v = k.astype(np.float64), v.astype(np.float64)
        t = np.arange(L)
        for i in range(n):
            p = L - n + i
            see = there.copy()
            if causal:
                see &= t <= p
            if window:
                see &= t > p - window
            q = rotate(Q[q0 + i].astype(F32), max(p, 0), rope).astype(np.float64) if L else Q[q0 + i].astype(np.float64)
            O[q0 + i] = A[q0 + i] = 0
            lse[q0 + i] = -np.inf
            if not see.any():
                continue
            kk, vv = k[see], v[see]
            for j in range(Hq):
                z = scale * (kk[:, j // G] @ q[j])
                m = z.max()
                e = np.exp(z - m)
                w = e / e.sum()
                O[q0 + i, j] = w @ vv[:, j // G]
                A[q0 + i, j] = w @ np.abs(vv[:, j // G])
                lse[q0 + i, j] = m + np.log(e.sum())
                Z[q0 + i, j] = scale * np.abs(kk[:, j // G]).sum(1).max() * np.abs(q[j]).max() / 32512
    return O, lse, A, Z
