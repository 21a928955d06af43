"""The error bounds of oracle/kv_error.py tried out on the host: a simulation of
what the attention kernels round passes, and mistakes planted in it do not."""
import numpy as np
import pytest

from oracle import kv as okv
from oracle import kv_error

F32 = np.float32


def a_cache(rng, pages, heads, page, dim, spread=(0.3, 3.0)):
    x = rng.standard_normal((2, pages, heads, page, dim)).astype(F32) * rng.uniform(*spread, (2, pages, heads, 1, 1)).astype(F32)
    s = (np.abs(x).max((3, 4)) / F32(127)).astype(F32)
    q = np.rint(x / s[..., None, None]).astype(np.int8)
    return okv.Cache(q[0], q[1], s[0], s[1])


def half(x):
    return x.astype(np.float16).astype(np.float64)


def simulated(c, Q, scale, q_start, kv_len, table, rope=None, causal=True, window=0, eps=2.0**-10, two=False, parts=1,
              mistake=None):
    """The kernels' roundings in numpy: queries as 15-bit integers, probabilities
    in fp16 relative to a part's maximum and largest value scale, parts merged,
    the result rounded.  ``mistake`` is planted in the merge."""
    T, Hq, D = Q.shape
    G = Hq // c.heads
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    for s in range(len(kv_len)):
        q0, n, L = int(q_start[s]), int(q_start[s + 1] - q_start[s]), int(kv_len[s])
        kc, vc, ks, vs, there = kv_error.values(c, table[s], L)
        t = np.arange(L)
        for i in range(n):
            p = L - n + i
            see = there.copy()
            if causal:
                see &= t <= p
            if window:
                see &= t > p - window
            out[q0 + i], lse[q0 + i] = 0, -np.inf
            if not see.any():
                continue
            q = okv.rotate(Q[q0 + i].astype(F32), max(p, 0), rope).astype(np.float64)
            cuts = np.array_split(np.flatnonzero(see), parts)
            for j in range(Hq):
                h = j // G
                step = np.abs(q[j]).max() / 16256
                qi = np.rint(q[j] / step) if step else q[j]
                ms, ls, os_ = [], [], []
                for cut in cuts:
                    if not len(cut):
                        continue
                    z = (kc[cut, h] @ qi) * (step * scale * ks[cut, h])
                    m, vref = z.max(), vs[cut, h].max()
                    pe = np.exp(z - m)
                    f = pe * (vs[cut, h] / vref if vref else 0)
                    ph = half(f) + (half(f - half(f)) if two else 0)
                    ms.append(m)
                    ls.append(pe.sum())
                    os_.append(ph @ vc[cut, h] * vref)
                ms, ls, os_ = np.array(ms), np.array(ls), np.array(os_)
                g = np.exp(ms - ms.max())
                bad = len(g) // 2
                if mistake == "part dropped":
                    os_[bad] = 0
                elif mistake == "weight off":
                    g[bad] *= 1.03
                elif mistake == "parts swapped":
                    os_[[0, bad]] = os_[[bad, 0]]
                out[q0 + i, j] = kv_error.rounded((g @ os_) / (g @ ls), eps)
                lse[q0 + i, j] = ms.max() + np.log(g @ ls)
    if mistake == "zero":
        out[~np.isnan(out)] = 0
    return out, lse


def setup(seed, ns, ls, heads, group, dim, page, q_scale=1.0):
    rng = np.random.default_rng(seed)
    used = [-(-l // page) for l in ls]
    table = np.full((len(ls), max(used)), -1)
    order, at = rng.permutation(sum(used)), 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    c = a_cache(rng, sum(used), heads, page, dim)
    q_start = np.concatenate([[0], np.cumsum(ns)])
    Q = rng.standard_normal((q_start[-1], heads * group, dim)).astype(np.float16).astype(F32) * F32(q_scale)
    return c, Q, dim ** -0.5, q_start, ls, table


CASES = [
    # ns, ls, heads, group, dim, page, q_scale, causal, window, parts
    ([1], [20000], 1, 8, 128, 128, 1.0, True, 0, 79),
    ([4, 2, 9], [5000, 100, 1300], 2, 3, 64, 64, 1.0, True, 1400, 20),
    ([1] * 16, [100 + 37 * i for i in range(16)], 2, 4, 64, 16, 2.0, True, 0, 3),
    ([65, 1, 40], [65, 400, 300], 2, 1, 128, 16, 2.0, True, 0, 1),
    ([40, 30], [900, 64], 1, 3, 64, 128, 2.0, False, 70, 2),
]


@pytest.mark.parametrize("ns, ls, heads, group, dim, page, q_scale, causal, window, parts", CASES)
def test_bounds_hold_what_the_kernels_round(ns, ls, heads, group, dim, page, q_scale, causal, window, parts):
    args = setup(1, ns, ls, heads, group, dim, page, q_scale)
    for eps in (2.0**-10, 2.0**-7):
        for two in (False, True):
            kw = dict(causal=causal, window=window, eps=eps, two=two)
            r = kv_error.rows(*args, **kw)
            got, lse = simulated(*args, parts=parts, **kw)
            assert kv_error.check(r, got, lse) is None
    # the same as the plain form, which rounds keys and values to fp32 (2^-24):
    # 32512 Z bounds scale sum |k| |q|
    O, L, A, Z = okv.attention(*args, causal=causal, window=window)
    z = 2.0**-24 * 32512 * Z
    assert (np.abs(r.O - O) <= (2.0**-24 + 2 * z[..., None]) * A + 1e-14).all()
    assert (np.abs(r.lse - L) <= z + 1e-13 * np.abs(L)).all()


@pytest.mark.parametrize("mistake", ["zero", "part dropped", "weight off", "parts swapped"])
@pytest.mark.parametrize("eps", [2.0**-10, 2.0**-7])
@pytest.mark.parametrize("case", CASES[:3])
def test_bounds_find_planted_mistakes(case, eps, mistake):
    ns, ls, heads, group, dim, page, q_scale, causal, window, parts = case
    args = setup(2, ns, ls, heads, group, dim, page, q_scale)
    kw = dict(causal=causal, window=window, eps=eps)
    few = min(parts, 4)                                   # (of 79 parts one is little)
    assert kv_error.check(kv_error.rows(*args, **kw), simulated(*args, parts=few, mistake=mistake, **kw)[0]) is not None


def test_bounds_find_a_missing_second_part():
    """Probabilities in one fp16 part where two are due, with many rows."""
    args = setup(3, [1] * 40, [150 + 13 * i for i in range(40)], 4, 4, 64, 16, 2.0)
    r = kv_error.rows(*args, two=True)
    assert kv_error.check(r, simulated(*args, two=True)[0]) is None
    got = simulated(*args, two=False)[0]
    assert kv_error.check(r, got) is not None
    assert np.sqrt(((got - r.O)**2).sum()) > 1.1 * kv_error.limit(r)


def test_rounded():
    x = np.random.default_rng(0).standard_normal(1000) * 10.0 ** np.random.default_rng(1).integers(-3, 4, 1000)
    import torch
    assert (kv_error.rounded(x, 2.0**-7) == torch.from_numpy(x).bfloat16().double().numpy()).all()
    assert (kv_error.rounded(x, 2.0**-10) == torch.from_numpy(x).half().double().numpy()).all()
