"""GPU tests of the int8 key/value cache against the plain forms of
oracle/kv.py: codes and scales bit for bit, values read back bit for bit,
attention within a bound derived from what the kernel rounds."""
import functools

import numpy as np
import pytest
import torch

import int8_matmul_amd as li8
from oracle import kv as okv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@functools.lru_cache
def rope_tables(rows, dims):
    ang = np.arange(rows)[:, None] * (10000.0 ** (-2.0 * np.arange(dims // 2) / dims))
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


class Setup:
    """A cache with random contents, a table of distinct pages, and a batch."""

    def __init__(self, ns, ls, heads, dim, page, dtype=F16, seed=0, rot=0, inter=False, spare=3, max_kv=None, max_q=None, lead=0, tail=0, group=1):
        self.rng = rng = np.random.default_rng(seed)
        self.ns, self.ls, self.heads, self.dim, self.page, self.dtype = ns, ls, heads, dim, page, dtype
        self.group = group
        used = [-(-l // page) for l in ls]
        pages = sum(used) + spare
        order = rng.permutation(pages)
        self.width = max(max(used), 1, -(-(max_kv or 0) // page))
        # table entries past a sequence's pages lead nowhere
        self.table = rng.choice([-1, -7, pages, 2**31 - 1], (len(ls), self.width)).astype(np.int32)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = order[at:at + u]
            at += u
        self.unused = order[at:]
        x = rng.standard_normal((2, pages, heads, page, dim)).astype(np.float32) * rng.uniform(0.3, 3, (2, pages, heads, 1, 1)).astype(np.float32)
        sc = (np.abs(x).max((3, 4)) / np.float32(127)).astype(np.float32)
        q = np.rint(x / sc[..., None, None]).astype(np.int8)
        sc[:, self.unused] = np.nan                       # pages of nobody may hold anything
        self.ref = okv.Cache(q[0].copy(), q[1].copy(), sc[0].copy(), sc[1].copy())
        self.cache = li8.KVCache(*(torch.from_numpy(a).to(DEV) for a in (q[0], q[1], sc[0], sc[1])))
        self.q_start = np.concatenate([[lead], lead + np.cumsum(ns)]).astype(np.int32)
        self.tokens = int(self.q_start[-1]) + tail
        self.max_kv = max(ls) if max_kv is None else max_kv
        self.batch = li8.KVBatch(i32(self.q_start.tolist()), i32(ls), torch.from_numpy(self.table).to(DEV),
                                 self.tokens, max(ns) if max_q is None else max_q, self.max_kv)
        self.rope = self.oracle_rope = None
        if rot:
            c, s = rope_tables(max(self.max_kv, 1), rot)
            self.rope = li8.Rope(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), inter)
            self.oracle_rope = (c, s, inter)

    def rows(self, heads, scale=1.0, pad=0):
        """A [tokens, heads, dim] tensor of self.dtype; with pad, a slice of wider rows."""
        x = torch.from_numpy(self.rng.standard_normal((self.tokens, heads * self.dim + pad)).astype(np.float32) * scale)
        x = x.to(self.dtype).to(DEV)
        lo = pad // 2 // 8 * 8
        return x[:, lo:lo + heads * self.dim].unflatten(1, (heads, self.dim))

    def same_cache(self):
        for got, want in ((self.cache.k, self.ref.k), (self.cache.v, self.ref.v), (self.cache.k_scale, self.ref.ks),
                          (self.cache.v_scale, self.ref.vs)):
            assert np.array_equal(got.cpu().numpy(), want, equal_nan=want.dtype == np.float32)


def f32(t):
    return t.float().cpu().numpy()


APPENDS = [
    # ns, ls, heads, dim, page, rot, inter
    ([1], [1], 1, 64, 16, 0, False),
    ([1, 1, 1], [1, 16, 17], 2, 128, 16, 128, False),
    ([1, 1, 1, 1], [64, 65, 63, 200], 3, 128, 64, 64, True),
    ([1, 1], [128, 130], 5, 64, 128, 64, False),
    ([5, 3, 9], [5, 20, 137], 2, 64, 32, 32, True),
    ([129, 1, 64, 0, 33], [129, 7, 100, 11, 33], 2, 128, 128, 128, False),
    ([40, 300], [41, 333], 3, 64, 64, 48, False),
    ([17, 31], [17, 500], 1, 128, 32, 96, True),
    ([200], [1000], 2, 128, 16, 16, False),
    ([7, 4], [3, 0], 2, 64, 16, 64, False),               # more rows than tokens
]


@pytest.mark.parametrize("ns, ls, heads, dim, page, rot, inter", APPENDS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append(ns, ls, heads, dim, page, rot, inter, dtype):
    t = Setup(ns, ls, heads, dim, page, dtype, seed=len(ns) + page, rot=rot, inter=inter, lead=2, tail=3)
    for scale in (0.5, 4.0):                              # the second time every scale grows
        K, V = t.rows(heads, scale, pad=80), t.rows(heads, scale, pad=24)
        before = K.clone(), V.clone()
        li8.kv_append(K, V, t.cache, t.batch, rope=t.rope)
        okv.append(t.ref, f32(K), f32(V), t.q_start, t.ls, t.table, t.oracle_rope)
        t.same_cache()
        assert torch.equal(K, before[0]) and torch.equal(V, before[1])


def test_append_special_values():
    """All-zero rows, subnormal rows, the largest finite values."""
    t = Setup([4, 4, 4], [4, 20, 9], 2, 64, 16, F16)
    for fill in (0.0, 6e-8, 65504.0):
        K = torch.full((12, 2, 64), fill, dtype=F16, device=DEV)
        K[::2, :, ::3] *= -1
        li8.kv_append(K, K, t.cache, t.batch)
        okv.append(t.ref, f32(K), f32(K), t.q_start, t.ls, t.table)
        t.same_cache()
    b = Setup([3], [3], 1, 64, 16, BF16)
    for fill in (1e-38, 9.2e-41, 3e38):                   # (9.2e-41 is a bf16 subnormal)
        K = torch.full((3, 1, 64), fill, dtype=BF16, device=DEV)
        li8.kv_append(K, K, b.cache, b.batch)
        okv.append(b.ref, f32(K), f32(K), b.q_start, b.ls, b.table)
        b.same_cache()


def test_append_token_by_token_and_again():
    """One token at a time through three pages; the last one twice."""
    n, heads, dim, page = 40, 2, 128, 16
    t = Setup([1], [n], heads, dim, page, rot=128)
    for i in range(n):
        K, V = t.rows(heads), t.rows(heads, 0.2)
        t.batch.kv_len.fill_(i + 1)
        for _ in range(2 if i == n - 1 else 1):
            li8.kv_append(K, V, t.cache, t.batch, rope=t.rope)
            okv.append(t.ref, f32(K), f32(V), t.q_start, [i + 1], t.table, t.oracle_rope)
            t.same_cache()


@pytest.mark.parametrize("dim, page, dtype", [(64, 16, F16), (128, 64, BF16), (128, 128, F16), (64, 32, BF16)])
def test_read(dim, page, dtype):
    t = Setup([1, 70, 0, 129, 64, 6], [50, 70, 9, 300, 64, 4], 3, dim, page, dtype, lead=1, tail=2)
    out = tuple(torch.full((t.tokens, 3 * dim + 16), 7.0, dtype=dtype, device=DEV)[:, 8:8 + 3 * dim].unflatten(1, (3, dim))
                for _ in range(2))
    got = li8.kv_read(t.cache, t.batch, dtype, out=out)
    for g, w in zip(got, okv.read(t.ref, t.q_start, t.ls, t.table, t.tokens)):
        want = torch.from_numpy(np.nan_to_num(w, nan=7.0)).to(dtype)   # rows of no sequence stay
        assert torch.equal(g.cpu(), want)
    assert torch.equal(li8.kv_read(t.cache, t.batch, dtype)[0][1:-2].cpu(), got[0][1:-2].cpu())


def tolerance(O, A, Z, n_keys, vmax, dtype):
    """What the kernel may be off by, element by element:
    * scores: queries are integers of 1/16256 of their largest value, off by
      half a step: |dz| <= Z, plus fp32 rounding of z (2^-16 covers |z| < 64);
      a weight, and the sum it is divided by, change by 1 + |dz| each;
    * probabilities: half a step of fp16, 2^-11 relative, or 2^-25 absolute
      where the value is subnormal (the largest is at least 1 in its units,
      so relative to the sum; value scales in these tests differ by less
      than 2^5 within a sequence, which the factor 32 covers);
    * the result: half a step of its type.
    """
    dz = (Z + 2.0**-16)[..., None]
    inner = A * (2.0**-11 + 2.02 * dz) + n_keys * 2.0**-25 * 32 * vmax
    return inner + (np.abs(O) + inner) * torch.finfo(dtype).eps / 2 + 2.0**-25


def check_attention(t, Hq, scale=None, causal=True, window=0, q_scale=1.0, expect=None, pad=0):
    Q = t.rows(Hq, q_scale, pad)
    sc = t.dim ** -0.5 if scale is None else scale
    out = torch.full((t.tokens, Hq, t.dim), 7.0, dtype=t.dtype, device=DEV)
    lse = torch.full((t.tokens, Hq), 7.0, dtype=torch.float32, device=DEV)
    if expect is not None:
        p = li8.kv_attention_plan(t.batch, t.cache, Hq, causal, window)
        assert (p["path"], p["splits"] > 1) == expect, p
    ws = li8.new_kv_attention_workspace(t.batch, t.cache, Hq).fill_(255)
    li8.kv_attention(Q, t.cache, t.batch, scale=sc, rope=t.rope, causal=causal, window=window, out=out, lse=lse,
                     workspace=ws)
    O, L, A, Z = okv.attention(t.ref, f32(Q), sc, t.q_start, t.ls, t.table, t.oracle_rope, causal, window)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    none = np.isnan(L)
    assert (got[none] == 7).all() and (gl[none] == 7).all()             # rows of no sequence
    got, gl, O, L, A, Z = got[~none], gl[~none], O[~none], L[~none], A[~none], Z[~none]
    empty = np.isneginf(L)
    assert (got[empty] == 0).all() and np.isneginf(gl[empty]).all()     # rows that see nothing
    live = t.ref.vs[np.unique(t.table[(t.table >= 0) & (t.table < t.ref.pages)])]
    tol = tolerance(O, A, Z, max(t.ls + [1]), float(live.max(initial=0)) * 127, t.dtype)
    err = np.abs(got - O)
    assert (err <= tol).all(), (err / tol).max()
    # lse: the scores' error, and fp32 sums of up to max_kv numbers
    bound = Z + 2.0**-16 + max(t.ls + [1]) * 2.0**-24 + 2.0**-22 * np.abs(np.where(empty, 0, L))
    with np.errstate(invalid="ignore"):
        assert (np.abs(gl - L)[~empty] <= bound[~empty]).all()
    # the same again, bit for bit, without lse, into a fresh tensor
    again = li8.kv_attention(Q, t.cache, t.batch, scale=sc, rope=t.rope, causal=causal, window=window)
    rows = ~none.any(1)
    assert torch.equal(again.cpu()[torch.from_numpy(rows)], out.cpu()[torch.from_numpy(rows)])
    return out


FEW = [
    # ns, ls, heads, group, dim, page, rot, causal, window
    ([1], [1], 1, 1, 64, 16, 0, True, 0),
    ([1], [1], 1, 1, 128, 128, 128, True, 0),
    ([1] * 9, [2, 15, 16, 17, 31, 32, 33, 63, 65], 2, 3, 64, 16, 64, True, 0),
    ([1] * 8, [64, 127, 128, 129, 255, 256, 257, 700], 2, 8, 128, 32, 128, True, 0),
    ([1] * 3, [1279, 1280, 5], 1, 16, 128, 64, 0, True, 0),
    ([1, 1], [0, 40], 2, 1, 64, 16, 64, True, 0),                       # no tokens at all
    ([1] * 4, [100, 300, 7, 31], 2, 4, 64, 16, 64, True, 1),
    ([1] * 4, [100, 300, 7, 31], 2, 4, 128, 64, 0, True, 33),
    ([2, 5, 1, 0, 3], [2, 90, 1, 8, 300], 1, 4, 64, 16, 64, True, 0),   # 20 columns
    ([2, 5, 1, 0, 3], [2, 90, 1, 8, 300], 2, 4, 128, 32, 128, True, 17),
    ([5, 3], [2, 0], 2, 1, 64, 16, 64, True, 0),                        # rows before the first token
    ([5, 3], [2, 0], 2, 1, 64, 16, 64, False, 0),
    ([7, 4], [50, 200], 1, 5, 64, 16, 0, False, 0),
    ([7, 4], [50, 200], 1, 5, 128, 16, 32, False, 9),
    ([1, 1], [77, 500], 1, 20, 128, 64, 0, True, 0),                    # a group past 16
    ([3], [400], 1, 21, 64, 64, 64, True, 100),                         # 63 columns: two blocks
]


@pytest.mark.parametrize("ns, ls, heads, group, dim, page, rot, causal, window", FEW)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_few(ns, ls, heads, group, dim, page, rot, causal, window, dtype):
    t = Setup(ns, ls, heads, dim, page, dtype, seed=page + group, rot=rot, inter=group % 2 == 0, lead=1, tail=2)
    check_attention(t, heads * group, causal=causal, window=window, expect=("few", False), q_scale=2.0, pad=16)


def test_attention_many_blocks():
    """More blocks than the wide workgroups are used for."""
    t = Setup([1] * 70, [(37 * i) % 90 for i in range(70)], 8, 64, 16)
    check_attention(t, 8, expect=("few", False))


SHARED = [
    # ns, ls, heads, group, dim, page, rot, causal, window
    ([1], [1281], 1, 1, 64, 16, 64, True, 0),
    ([1], [20000], 1, 8, 128, 128, 0, True, 0),
    ([1] * 5, [3000, 1, 1500, 0, 2999], 2, 4, 128, 64, 128, True, 0),
    ([1] * 70, [2000] + [(97 * i) % 1500 for i in range(69)], 1, 2, 64, 32, 0, True, 0),   # past 64 sequences
    ([1] * 130, [(531 * i) % 1800 for i in range(130)], 3, 1, 64, 16, 0, True, 0),
    ([4, 2, 0, 9], [5000, 100, 0, 1300], 2, 3, 64, 64, 64, True, 1400),
    ([4, 2, 0, 9], [5000, 100, 0, 1300], 1, 3, 128, 16, 0, False, 0),
    ([9, 9], [4000, 3000], 1, 7, 64, 64, 0, False, 2000),
    ([7, 1], [2000, 3], 1, 9, 64, 16, 64, True, 0),                     # 63 columns: two blocks
]


@pytest.mark.parametrize("ns, ls, heads, group, dim, page, rot, causal, window", SHARED)
def test_attention_shared(ns, ls, heads, group, dim, page, rot, causal, window):
    for dtype in (F16, BF16):
        t = Setup(ns, ls, heads, dim, page, dtype, seed=page + group, rot=rot, lead=1, tail=1)
        check_attention(t, heads * group, causal=causal, window=window, expect=("few", True))


TILED = [
    # ns, ls, heads, group, dim, page, rot, causal, window
    ([1], [1], 1, 1, 64, 16, 64, True, 0),
    ([64], [64], 1, 1, 128, 16, 128, True, 0),
    ([65, 1, 130], [65, 400, 1000], 2, 1, 64, 16, 64, True, 0),
    ([257, 300], [257, 777], 1, 1, 128, 64, 0, True, 0),
    ([33, 100, 0, 7], [500, 100, 5, 3], 2, 8, 128, 32, 64, True, 0),
    ([100, 64], [900, 64], 1, 3, 64, 128, 64, True, 70),
    ([100, 64], [900, 64], 1, 3, 128, 16, 0, True, 1),
    ([100, 70], [130, 64], 2, 1, 128, 64, 32, False, 0),
    ([90, 200], [900, 210], 1, 2, 64, 32, 0, False, 50),
    ([70, 80], [30, 0], 1, 1, 64, 16, 64, True, 0),                     # rows before the first token
    ([70, 80], [30, 0], 1, 1, 128, 16, 0, False, 0),
    ([64, 3], [3000, 2100], 1, 2, 128, 64, 128, True, 0),
    ([20, 30], [5000, 70], 1, 5, 64, 16, 0, True, 0),
    ([64, 100], [2500, 1200], 1, 1, 64, 128, 0, True, 1500),
    ([64, 100], [2500, 1200], 1, 1, 128, 32, 0, False, 1100),
    ([1100], [1100], 1, 1, 64, 64, 0, False, 0),
    ([700, 0, 300], [700, 0, 310], 3, 1, 128, 16, 128, True, 0),        # prompts
    ([9] * 70, [600 + (61 * i) % 400 for i in range(70)], 1, 8, 64, 16, 0, True, 0),   # past 64 sequences
    ([150, 9], [90, 1500], 2, 2, 64, 64, 64, True, 0),
]


def tiled_blocks(ns, heads, group, window, shared):
    """Blocks of each pair of a sequence and a head that the bounds have to allow."""
    pairs = len(ns) * heads
    span = min(1 << 14, window + 256 + 31) if window else 1 << 14
    blocks = max(-(-4096 // (span // 64)), 1 if shared else 256, -(-max(ns) * group // 256) * pairs)
    return -(-blocks // pairs)


# (under a short window as many blocks as the tiled kernel takes go unshared)
TILED_RUNS = [(*c, shared) for shared in (True, False) for c in TILED
              if not shared or len(c[0]) * c[2] * tiled_blocks(c[0], c[2], c[3], c[8], True) < 256]


@pytest.mark.parametrize("ns, ls, heads, group, dim, page, rot, causal, window, shared", TILED_RUNS)
def test_attention_tiled(ns, ls, heads, group, dim, page, rot, causal, window, shared):
    """Small chunks with bounds that call for the tiled kernel: many rows and
    keys allowed, of which there are few.  It takes 4096 blocks x steps of 64
    keys, and 256 blocks or more go unshared."""
    rows = tiled_blocks(ns, heads, group, window, shared) * 256 // group
    for dtype in (F16, BF16):
        t = Setup(ns, ls, heads, dim, page, dtype, seed=page + group, rot=rot, inter=page == 32, lead=1,
                  max_kv=1 << 14, max_q=rows, tail=max(0, rows - sum(ns)))
        check_attention(t, heads * group, causal=causal, window=window, q_scale=2.0, expect=("tiled", shared))


def tiled_setup(ns, ls, heads, group, dim, shared, dtype=F16):
    rows = tiled_blocks(ns, heads, group, 0, shared) * 256 // group
    return Setup(ns, ls, heads, dim, 16, dtype, max_kv=1 << 14, max_q=rows, tail=max(0, rows - sum(ns)))


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_tiled_extremes(dim, shared):
    """The tiled kernel: peaked scores, a zero query, scale 0, zero scales,
    page numbers that do not exist, no page at all."""
    t = tiled_setup([70, 64], [700, 90], 1, 2, dim, shared)
    expect = ("tiled", shared)
    check_attention(t, 2, q_scale=30.0, scale=0.2, expect=expect)
    check_attention(t, 2, q_scale=0.0, expect=expect)
    check_attention(t, 2, scale=0.0, expect=expect)
    for c, r in ((t.cache.k_scale, t.ref.ks), (t.cache.v_scale, t.ref.vs)):
        c[t.table[0, 1]] = 0.0
        r[t.table[0, 1]] = 0.0
    check_attention(t, 2, expect=expect)
    for s, b, bad in ((0, 1, -1), (0, 2, t.ref.pages), (1, 0, 2**31 - 1), (1, 2, -2**31), (1, 5, -5)):
        t.table[s, b] = bad
    t.batch.table.copy_(torch.from_numpy(t.table))
    check_attention(t, 2, expect=expect)
    t.cache.v_scale.zero_()
    t.ref.vs[:] = 0
    assert not check_attention(t, 2, expect=expect)[:134].any()
    t.table[:] = -1
    t.batch.table.fill_(-1)
    assert not check_attention(t, 2, expect=expect)[:134].any()


@pytest.mark.parametrize("case", ["few", "few shared", "tiled"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_least_value_scales(case, dtype):
    """Value scales below fp32's normal range count as 0: what they would give,
    at most 127 * 2^-126, is below the tolerance's absolute part."""
    if case == "tiled":
        t = tiled_setup([70, 64], [700, 90], 1, 2, 64, False, dtype)
    else:
        t = Setup([1, 1], [90, 300] if case == "few" else [3000, 1500], 1, 64, 16, dtype)
    for first, least in ((1, 1.0e-39), (0, 1.0e-45)):
        for s in range(2):                                # one page of each sequence, then all
            at = t.table[s, first:first + 1] if first else t.table[s, :-(-t.ls[s] // 16)]
            t.cache.v_scale[torch.from_numpy(at.astype(np.int64)).to(DEV)] = least
            t.ref.vs[at] = np.float32(least)
        check_attention(t, 2, expect=(case.split()[0], case == "few shared"))


def test_attention_tiled_many_blocks():
    """A prompt with two rounds of blocks for the chip: unshared, longest first."""
    t = Setup([530], [530], 172, 64, 64)
    check_attention(t, 172, expect=("tiled", False))


@pytest.mark.parametrize("ns, ls, group", [([1, 1], [90, 300], 2), ([1], [3000], 4), ([70, 64], [700, 90], 2)])
def test_attention_extremes(ns, ls, group):
    """Peaked scores, a zero query, zero keys and values, scale 0, page scales
    far apart."""
    for dim in (64, 128):
        t = Setup(ns, ls, 1, dim, 16, F16)
        check_attention(t, group, q_scale=30.0, scale=0.2)
        check_attention(t, group, q_scale=0.0)
        check_attention(t, group, scale=0.0)
        p = t.table[0, 1]
        for c, r in ((t.cache.k_scale, t.ref.ks), (t.cache.v_scale, t.ref.vs)):
            c[p] = 0.0
            r[p] = 0.0
        check_attention(t, group)
        t.cache.v_scale.zero_()
        t.ref.vs[:] = 0
        out = check_attention(t, group)
        assert not out[torch.from_numpy(np.arange(t.tokens) < t.q_start[-1])].any()


@pytest.mark.parametrize("ns, ls, group", [([1, 1], [90, 300], 2), ([1, 1], [3000, 1500], 4), ([70, 64], [700, 90], 2)])
def test_bad_pages(ns, ls, group):
    """Page numbers that do not exist inside a sequence: masked, read as zeros,
    not written."""
    t = Setup(ns, ls, 2, 64, 16, F16, rot=64)
    for s, b, bad in ((0, 1, -1), (0, 3, t.ref.pages), (1, 0, 2**31 - 1), (1, 2, -2**31)):
        t.table[s, b] = bad
    t.table[1, -(-ls[1] // 16) - 1] = -5                  # the page of the last token too
    t.batch.table.copy_(torch.from_numpy(t.table))
    check_attention(t, 2 * group)
    got = li8.kv_read(t.cache, t.batch, F16)
    for g, w in zip(got, okv.read(t.ref, t.q_start, t.ls, t.table, t.tokens)):
        assert torch.equal(g.cpu(), torch.from_numpy(w).to(F16))
    K = t.rows(2)
    li8.kv_append(K, K, t.cache, t.batch, rope=t.rope)
    okv.append(t.ref, f32(K), f32(K), t.q_start, t.ls, t.table, t.oracle_rope)
    t.same_cache()
    # a sequence with no page at all
    t.table[:] = -1
    t.batch.table.fill_(-1)
    out = check_attention(t, 2 * group)
    assert not out.any()


def test_lengths_past_the_bounds():
    """Lengths on the GPU that the host's bounds do not allow are cut: rows
    past the packed tensors, tokens past max_kv, chunks past max_q."""
    t = Setup([3, 2], [20, 30], 1, 64, 16)
    Q, K = t.rows(1), t.rows(1)
    for q_start, kv_len in (([0, 3, 2**31 - 1], [20, 2**31 - 1]), ([-5, 2, 1], [-3, 30]), ([4, 1, 5], [31, 99]),
                            ([0, 5, 5], [2**31 - 1, -2**31])):
        t.batch.q_start.copy_(i32(q_start))
        t.batch.kv_len.copy_(i32(kv_len))
        li8.kv_append(K, K, t.cache, t.batch)
        li8.kv_read(t.cache, t.batch)
        li8.kv_attention(Q, t.cache, t.batch)
        torch.cuda.synchronize()
    t.batch.q_start.copy_(i32(t.q_start.tolist()))
    t.batch.kv_len.copy_(i32(t.ls))
    for a, b in ((t.ref.k, t.cache.k), (t.ref.v, t.cache.v), (t.ref.ks, t.cache.k_scale), (t.ref.vs, t.cache.v_scale)):
        a[:] = b.cpu().numpy()
    check_attention(t, 1)


def test_large_offsets():
    """Pages whose codes lie past 2^32 bytes, rows past 2^31 elements."""
    page, heads, dim, pages = 128, 8, 128, 34000          # 4.46e9 bytes of keys
    k = torch.zeros((pages, heads, page, dim), dtype=torch.int8, device=DEV)
    s = torch.zeros((pages, heads), dtype=torch.float32, device=DEV)
    cache = li8.KVCache(k, torch.zeros_like(k), s, torch.zeros_like(s))
    tokens, stride = 1100000, 2048                        # 2.25e9 elements
    big = torch.empty((tokens, stride), dtype=F16, device=DEV)
    n = 150
    x = torch.randn((n, heads, dim), device=DEV).to(F16)
    big[-n:, 1024:] = x.flatten(1)
    K = big[:, 1024:].unflatten(1, (heads, dim))
    table = i32([[pages - 1, pages - 3]])
    batch = li8.KVBatch(i32([tokens - n, tokens]), i32([n]), table, tokens, n, n)
    li8.kv_append(K, K, cache, batch)
    small = li8.KVBatch(i32([0, n]), i32([n]), table, n, n, n)
    near = li8.new_kv_cache(4, heads, dim, page, DEV)
    close = li8.KVBatch(i32([0, n]), i32([n]), i32([[1, 3]]), n, n, n)
    li8.kv_append(x, x, near, close)
    assert torch.equal(cache.k[pages - 1], near.k[1]) and torch.equal(cache.v[pages - 3], near.v[3])
    assert not cache.k[:pages - 3].any() and not cache.k[pages - 2].any()
    for a, b in zip(li8.kv_read(cache, small), li8.kv_read(near, close)):
        assert torch.equal(a, b)
    li8.kv_read(cache, batch, out=(K, K))
    assert torch.equal(K[-n:], li8.kv_read(near, close)[1])
    K[-n:] = x
    want = li8.kv_attention(x, near, close)
    out = big[:, :1024].unflatten(1, (heads, dim))
    li8.kv_attention(K, cache, batch, out=out)
    assert torch.equal(out[-n:], want)
    one = li8.KVBatch(i32([tokens - 1, tokens]), i32([n]), table, tokens, 1, n)
    li8.kv_attention(K, cache, one, out=out)
    assert torch.equal(out[-1:], li8.kv_attention(x[-1:], near, li8.KVBatch(i32([0, 1]), i32([n]), i32([[1, 3]]), 1, 1, n)))


def test_other_stream_and_two_at_once():
    t = Setup([1, 1, 1], [3000, 2000, 40], 4, 128, 64, BF16, rot=128)
    u = Setup([90, 70], [200, 3000], 2, 128, 64, BF16, rot=64, seed=5)
    Qt, Qu = t.rows(16), u.rows(8)
    want = li8.kv_attention(Qt, t.cache, t.batch, rope=t.rope), li8.kv_attention(Qu, u.cache, u.batch, rope=u.rope)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(a):
            x = li8.kv_attention(Qt, t.cache, t.batch, rope=t.rope)
        with torch.cuda.stream(b):
            y = li8.kv_attention(Qu, u.cache, u.batch, rope=u.rope)
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_graph_replay():
    """A decode step captured once and replayed for the following tokens: the
    lengths, tables and rows change in place between replays."""
    heads, group, dim, page, S = 2, 4, 128, 16, 3
    t = Setup([1] * S, [2000, 30, 100], heads, dim, page, F16, rot=128)
    e = Setup([1] * S, [2000, 30, 100], heads, dim, page, F16, rot=128)     # the same, run eagerly
    K, V, Q = t.rows(heads), t.rows(heads), t.rows(heads * group)
    ws = li8.new_kv_attention_workspace(t.batch, t.cache, heads * group)
    out = torch.empty_like(Q)

    def step(x, o):
        li8.kv_append(K, V, x.cache, x.batch, rope=x.rope)
        li8.kv_attention(Q, x.cache, x.batch, rope=x.rope, out=o, workspace=ws)

    lens = t.batch.kv_len.clone() - 8
    t.batch.kv_len.copy_(lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(t, out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(t, out)
    for a, b in ((t.cache.k, e.cache.k), (t.cache.v, e.cache.v), (t.cache.k_scale, e.cache.k_scale),
                 (t.cache.v_scale, e.cache.v_scale)):
        a.copy_(b)
    for i in range(8):
        K.copy_(t.rows(heads, 1 + i % 3))
        V.copy_(t.rows(heads))
        Q.copy_(t.rows(heads * group))
        t.batch.kv_len.copy_(lens + i)
        e.batch.kv_len.copy_(lens + i)
        g.replay()
        got = out.clone()
        want = torch.empty_like(Q)
        torch.cuda.synchronize()
        step(e, want)
        assert torch.equal(got, want)
        same = torch.equal(t.cache.k, e.cache.k) and torch.equal(t.cache.v, e.cache.v)
        scales = torch.equal(t.cache.v_scale.nan_to_num(-1), e.cache.v_scale.nan_to_num(-1))   # (NaN: nobody's pages)
        assert same and scales


def test_layer_prompt_then_steps():
    """The operators as a layer uses them: the int8 qkv projection, append,
    attention, the int8 output projection; a ragged prompt in two chunks, then
    single tokens.  The cache is bit for bit the plain form's, every attention
    within its bound."""
    heads, group, dim, page, hidden = 2, 4, 64, 16, 256
    Hq = heads * group
    rng = np.random.default_rng(3)
    W = torch.from_numpy(rng.standard_normal(((Hq + 2 * heads) * dim, hidden)).astype(np.float32) * 0.1).half().to(DEV)
    Wo = torch.from_numpy(rng.standard_normal((hidden, Hq * dim)).astype(np.float32) * 0.05).half().to(DEV)
    (Wq, sW), (Woq, sWo) = li8.quantize_weight(W), li8.quantize_weight(Wo)
    total = [90, 33]
    t = Setup([1, 1], total, heads, dim, page, F16, rot=64)
    chunks = [([60, 20], [60, 20]), ([25, 10], [85, 30])] + [([1, 1], [86 + i, 31 + i]) for i in range(3)]
    for ns, ls in chunks:
        t.ns, t.ls = ns, ls
        t.q_start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        t.tokens = int(t.q_start[-1])
        t.batch = li8.KVBatch(i32(t.q_start.tolist()), i32(ls), t.batch.table, t.tokens, max(ns), t.max_kv)
        X = torch.from_numpy(rng.standard_normal((t.tokens, hidden)).astype(np.float32)).half().to(DEV)
        qkv = li8.linear(X, Wq, sW).unflatten(1, (Hq + 2 * heads, dim))
        q, k, v = qkv.split([Hq, heads, heads], dim=1)
        li8.kv_append(k, v, t.cache, t.batch, rope=t.rope)
        okv.append(t.ref, f32(k), f32(v), t.q_start, ls, t.table, t.oracle_rope)
        t.same_cache()
        o = li8.kv_attention(q, t.cache, t.batch, rope=t.rope)
        O, L, A, Z = okv.attention(t.ref, f32(q), dim ** -0.5, t.q_start, ls, t.table, t.oracle_rope)
        tol = tolerance(O, A, Z, max(ls), float(t.ref.vs[t.table[t.table >= 0][t.table[t.table >= 0] < t.ref.pages]].max()) * 127, F16)
        assert (np.abs(o.double().cpu().numpy() - O) <= tol).all()
        y = li8.linear(o.flatten(1), Woq, sWo)
        assert y.shape == (t.tokens, hidden) and torch.isfinite(y).all()


def test_binding_refusals():
    t = Setup([2, 1], [20, 5], 2, 64, 16, F16, rot=64)
    K, Q = t.rows(2), t.rows(4)
    with pytest.raises(TypeError):
        li8.kv_append(K.float(), K.float(), t.cache, t.batch)
    with pytest.raises(TypeError):
        li8.kv_append(K, K.bfloat16(), t.cache, t.batch)
    with pytest.raises(ValueError):
        li8.kv_append(K[:2], K[:2], t.cache, t.batch)                   # rows of another batch
    with pytest.raises(ValueError):
        li8.kv_append(K.transpose(0, 1).contiguous().transpose(0, 1), K, t.cache, t.batch)
    with pytest.raises(ValueError):
        li8.kv_attention(Q.cpu(), t.cache, t.batch)
    with pytest.raises(TypeError):
        li8.kv_attention(Q, t.batch, t.cache)
    with pytest.raises(TypeError):
        li8.kv_read(t.cache, t.batch, torch.float32)
    with pytest.raises(li8.Int8MatmulError):
        li8.kv_attention(t.rows(3), t.cache, t.batch)                   # 3 heads over 2
    with pytest.raises(li8.Int8MatmulError):
        li8.kv_attention(Q, t.cache, t.batch, rope=li8.Rope(t.rope.cos[:10].contiguous(), t.rope.sin[:10].contiguous()))
    with pytest.raises(li8.Int8MatmulError):
        li8.kv_attention(Q, t.cache, t.batch, scale=float("nan"))
    odd = torch.zeros(3 * (2 * 64 + 4), dtype=F16, device=DEV).as_strided((3, 2, 64), (132, 64, 1))
    with pytest.raises(li8.Int8MatmulError):
        li8.kv_append(odd, odd, t.cache, t.batch)                       # row stride not a multiple of 8
    with pytest.raises(ValueError):
        li8.KVBatch(t.batch.q_start, t.batch.kv_len[:1], t.batch.table, 3, 2, 20)
    with pytest.raises(ValueError):
        li8.KVBatch(t.batch.q_start, t.batch.kv_len, t.batch.table, -1, 2, 20)
    with pytest.raises(TypeError):
        li8.KVBatch(t.batch.q_start, t.batch.kv_len, t.batch.table.long(), 3, 2, 20)
    with pytest.raises(ValueError):
        li8.KVCache(t.cache.k, t.cache.v[:1], t.cache.k_scale, t.cache.v_scale)
    big = li8.KVBatch(t.batch.q_start, t.batch.kv_len, torch.zeros((2, 4096), dtype=torch.int32, device=DEV), 3, 2, 65536)
    need = li8.kv_attention_workspace_bytes(big, t.cache, 4)
    assert need > 0
    with pytest.raises(li8.Int8MatmulError):
        li8.kv_attention(Q, t.cache, big, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    e = li8.KVBatch(i32([0]), i32([]), torch.zeros((0, 2), dtype=torch.int32, device=DEV), 0, 0, 0)
    empty = torch.empty((0, 4, 64), dtype=F16, device=DEV)
    assert li8.kv_attention(empty, t.cache, e).shape == (0, 4, 64)      # an empty batch is fine
    li8.kv_append(empty[:, :2], empty[:, :2], t.cache, e)
