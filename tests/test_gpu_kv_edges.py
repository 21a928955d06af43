"""GPU tests of the int8 key/value cache at its edges, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import int8_matmul_amd as li8
import test_gpu_kv as base
from oracle import kv as okv
from oracle import kv_error

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("least", [0.0, 2.0**-99, 2.0**-110])
def test_sum_over_pages_without_values(least):
    """Pages whose value scale is (almost) 0 count in the softmax's sum with
    their full weight: one key at z = 0 in a page with values, 16383 at
    2^-26.125 of its weight, all but 15 of them in pages without.  They are
    2.2e-4 of the sum together.

    Bound: scores are exact to 2^-16 of a weight (queries of one value,
    integer codes), and a lane adds 2 numbers for each of 512 subtiles of 32
    keys in fp32, each sum off by half a step: 1024 * 2^-24."""
    heads, dim, page, n, rows = 256, 64, 128, 16384, 128
    pages = n // page
    k = torch.zeros((pages, heads, page, dim), dtype=torch.int8, device=DEV)
    k[..., 0] = -26
    k[3, :, 5, 0] = 0
    v = torch.ones_like(k)
    ks = torch.ones((pages, heads), dtype=torch.float32, device=DEV)
    vs = torch.full_like(ks, least)
    vs[3] = 1.0
    cache = li8.KVCache(k, v, ks, vs)
    batch = li8.KVBatch(i32([0, rows]), i32([n]), torch.arange(pages, dtype=torch.int32, device=DEV)[None], rows, rows, n)
    assert li8.kv_attention_plan(batch, cache, heads, causal=False) == dict(path="tiled", splits=1)
    Q = torch.zeros((rows, heads, dim), dtype=F16, device=DEV)
    Q[..., 0] = 1.0
    lse = torch.empty((rows, heads), dtype=torch.float32, device=DEV)
    scale = 26.125 / 26 * math.log(2)
    out = li8.kv_attention(Q, cache, batch, scale=scale, causal=False, lse=lse)
    w = 2.0**-26.125
    total = 1 + (n - 1) * w
    bound = 1024 * 2.0**-24 + n * w * 2.0**-16
    got = lse.double().cpu().numpy()
    assert np.abs(got - math.log(total)).max() <= bound, (got.min(), got.max(), math.log(total))
    want = (1 + 15 * w + (n - 16) * w * least) / total
    assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0**-11 + bound + 2.0**-24


def small(seqs=1, tokens=1, kv=20):
    cache = li8.new_kv_cache(4, 2, 64, 16, DEV)
    return cache, li8.KVBatch(i32([0] + [tokens] * seqs), i32([kv] * seqs), i32([[1, 2]] * seqs), tokens, tokens, kv)


def test_numbers_past_32_bits():
    """Refused, not cut to their low bits."""
    cache, batch = small()
    Q = torch.zeros((1, 4, 64), dtype=F16, device=DEV)
    for window in (2**32 + 1, 2**31, 2**64):
        with pytest.raises(ValueError):
            li8.kv_attention(Q, cache, batch, window=window)
    li8.kv_attention(Q, cache, batch, window=2**31 - 1)
    none = dict(dtype=torch.int8, device=DEV), dict(dtype=torch.float32, device=DEV)
    for shape in ((0, 2**32 + 4, 16, 64), (0, 4, 2**32 + 16, 64), (0, 4, 16, 2**32 + 64)):
        k, s = torch.empty(shape, **none[0]), torch.empty(shape[:2], **none[1])
        with pytest.raises(ValueError):
            li8.KVCache(k, k, s, s)
    for shape in ((2**32 + 20, 0), (0, 2**31 + 32)):
        with pytest.raises(ValueError):
            li8.Rope(torch.empty(shape, **none[1]), torch.empty(shape, **none[1]))
    with pytest.raises(ValueError):
        li8.KVBatch(i32([0]), i32([]), torch.empty((0, 2**32 + 2), dtype=torch.int32, device=DEV), 0, 0, 0)


def test_descriptions_are_fixed():
    """The library reads what was described at construction: a name bound anew
    would pass the checks and leave the old bounds and pointers in use."""
    cache, batch = small(tokens=2)
    rope = li8.Rope(torch.zeros((20, 32), device=DEV), torch.zeros((20, 32), device=DEV))
    for thing, names in ((cache, ("k", "v", "k_scale", "v_scale", "pages", "heads", "page_size", "head_dim", "device")),
                         (batch, ("q_start", "kv_len", "table", "seqs", "tokens", "max_q", "max_kv", "device")),
                         (rope, ("cos", "sin", "interleaved", "device"))):
        for name in names:
            was = getattr(thing, name)
            with pytest.raises(AttributeError):
                setattr(thing, name, was)
            with pytest.raises(AttributeError):
                delattr(thing, name)
            assert getattr(thing, name) is was
    with pytest.raises(ValueError):                       # rows of a batch with more of them
        li8.kv_append(torch.zeros((3, 2, 64), dtype=F16, device=DEV), torch.zeros((3, 2, 64), dtype=F16, device=DEV), cache, batch)


def test_largest_grids():
    """The most workgroups that the checks let through (2^32 work-items less a
    few), nearly all of them without a row: the last sequence's tokens are
    stored, read and attended to."""
    cache = li8.new_kv_cache(3, 16, 64, 16, DEV)
    x = torch.randn((8192, 16, 64), device=DEV).to(F16)

    def last(seqs, n, max_q):
        q_start, kv_len = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV), torch.zeros(seqs, dtype=torch.int32, device=DEV)
        q_start[-1], kv_len[-1] = n, n
        return li8.KVBatch(q_start, kv_len, i32([[1, 2]]).expand(seqs, 2).contiguous(), max_q, max_q, 32)

    near, one = li8.new_kv_cache(3, 16, 64, 16, DEV), li8.KVBatch(i32([0, 17]), i32([17]), i32([[1, 2]]), 17, 17, 32)
    li8.kv_append(x[:17], x[:17], near, one)
    big = last((1 << 23) - 1, 17, 17)
    li8.kv_append(x[:17], x[:17], cache, big)
    assert torch.equal(cache.k, near.k) and torch.equal(cache.v, near.v) and torch.equal(cache.k_scale, near.k_scale)
    del big
    big = last((1 << 17) - 1, 17, 8192)
    K, V = li8.kv_read(cache, big)
    want = li8.kv_read(near, one)
    assert torch.equal(K[:17], want[0]) and torch.equal(V[:17], want[1])
    del big
    big = last((1 << 20) - 1, 1, 1)
    assert li8.kv_attention_plan(big, cache, 16) == dict(path="few", splits=1)
    out = li8.kv_attention(x[:1], cache, big)
    first = li8.KVBatch(i32([0, 1]), i32([1]), i32([[1, 2]]), 1, 1, 32)
    assert torch.equal(out, li8.kv_attention(x[:1], near, first))


def cut(t, q_start, kv_len):
    """(first row, rows, rows that count, tokens) of each sequence, from the
    header: rows lie in the packed tensors, a sequence is cut to max_kv tokens,
    of which its rows are the last, and rows past max_q are left out."""
    out = []
    for s, length in enumerate(kv_len):
        q0 = min(max(q_start[s], 0), t.tokens)
        rows = min(max(q_start[s + 1], q0), t.tokens) - q0
        out.append((q0, rows, min(rows, t.batch.max_q), min(max(length, 0), t.max_kv)))
    return out


CUTS = [
    # ns, ls, heads, group, dim, page, max_q, max_kv, what the GPU finds: q_start, kv_len
    ([3, 2], [20, 30], 1, 1, 64, 16, None, None, [0, 3, 2**31 - 1], [20, 2**31 - 1]),
    ([3, 2], [20, 30], 1, 1, 64, 16, None, None, [-5, 2, 1], [-3, 30]),
    ([3, 2], [20, 30], 1, 1, 64, 16, None, None, [4, 1, 5], [31, 99]),
    ([3, 2], [20, 30], 1, 1, 64, 16, None, None, [0, 5, 5], [2**31 - 1, -2**31]),
    ([40, 9, 7], [60, 41, 33], 2, 3, 128, 16, 25, 50, [0, 40, 49, 56], [60, 41, 33]),       # chunks past max_q, tokens past max_kv
    ([40, 9, 7], [60, 41, 33], 2, 3, 128, 16, 25, 50, [0, 40, 49, 56], [10, 2**30, 3]),
    ([40, 9, 7], [60, 41, 33], 2, 3, 64, 64, 5, 64, [2, 51, 51, 2**31 - 1], [64, 41, 63]),
    ([1, 6], [3000, 2000], 1, 4, 64, 64, 3, 2500, [0, 1, 7], [2600, 2000]),                  # keys shared
    ([200, 300], [210, 400], 8, 1, 64, 16, 150, 1 << 14, [0, 200, 500], [210, 2**31 - 1]),   # tiled
    ([200, 300], [210, 400], 8, 1, 128, 64, 150, 1 << 14, [-9, 180, 400], [90, 390]),
]


@pytest.mark.parametrize("ns, ls, heads, group, dim, page, max_q, max_kv, q_start, kv_len", CUTS)
@pytest.mark.parametrize("causal", [True, False])
def test_numbers_past_the_bounds(ns, ls, heads, group, dim, page, max_q, max_kv, q_start, kv_len, causal):
    """Lengths on the GPU that the host's bounds do not allow are cut as the
    header says: codes, scales, values, outputs and the rows left as they were."""
    t = base.Setup(ns, ls, heads, dim, page, F16, seed=dim, rot=64, max_kv=max_kv, max_q=max_q)
    t.batch.q_start.copy_(i32(q_start))
    t.batch.kv_len.copy_(i32(kv_len))
    seqs = cut(t, q_start, kv_len)
    K, V, Q = t.rows(heads), t.rows(heads, 2.0), t.rows(heads * group)
    li8.kv_append(K, V, t.cache, t.batch, rope=t.rope)
    for s, (q0, rows, n, L) in enumerate(seqs):
        okv.append(t.ref, base.f32(K), base.f32(V), [q0, q0 + n], [L - rows + n], t.table[s:s + 1], t.oracle_rope)
    t.same_cache()

    got = tuple(torch.full((t.tokens, heads, dim), 7.0, dtype=F16, device=DEV) for _ in range(2))
    li8.kv_read(t.cache, t.batch, out=got)
    want = np.full((2, t.tokens, heads, dim), 7.0, np.float32)
    for s, (q0, rows, n, L) in enumerate(seqs):
        kv = okv.read(t.ref, [q0, q0 + n], [L - rows + n], t.table[s:s + 1], t.tokens)
        want[:, q0:q0 + n] = [x[q0:q0 + n] for x in kv]
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), torch.from_numpy(w).to(F16))

    out = torch.full((t.tokens, heads * group, dim), 7.0, dtype=F16, device=DEV)
    lse = torch.full((t.tokens, heads * group), 7.0, dtype=torch.float32, device=DEV)
    li8.kv_attention(Q, t.cache, t.batch, rope=t.rope, causal=causal, out=out, lse=lse)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    left = np.ones(t.tokens, bool)
    for s, (q0, rows, n, L) in enumerate(seqs):
        r = kv_error.rows(t.ref, base.f32(Q), dim ** -0.5, [q0, q0 + rows], [L], t.table[s:s + 1], t.oracle_rope, causal)
        r.lse[q0 + n:] = np.nan                           # rows past max_q
        wrong = kv_error.check(r, out, lse)
        assert wrong is None, (s, wrong)
        left[q0:q0 + n] = False
    assert (out[left] == 7).all() and (lse[left] == 7).all()


def plain(Q, cache, table, kv, scale):
    """fp64 (O, bound) of one sequence's last rows without a rotation: the bound
    of a kernel with probabilities in one fp16 part (oracle/kv_error.py, with
    sum w |v - O| <= 2 sum w |v|)."""
    rows, Hq, D = Q.shape
    H, page = cache.heads, cache.page_size
    at = torch.arange(kv, device=DEV)
    p, i = table.long()[at // page], at % page
    kc, vc = cache.k[p, :, i].double(), cache.v[p, :, i].double()
    k, vs = kc * cache.k_scale[p].double()[..., None], cache.v_scale[p].double()
    v = vc * vs[..., None]
    O, B = torch.empty((rows, Hq, D), dtype=torch.float64, device=DEV), torch.empty((rows, Hq, D), dtype=torch.float64, device=DEV)
    G = Hq // H
    for r in range(rows):
        n = kv - rows + r + 1
        for h in range(H):
            q = Q[r, h * G:(h + 1) * G].double()
            kk, vv = k[:n, h].contiguous(), v[:n, h].contiguous()
            z = scale * (q @ kk.T.contiguous())
            e = (z - z.amax(1, keepdim=True)).exp()
            S = e.sum(1, keepdim=True)
            w = e / S
            A = w @ vv.abs()
            O[r, h * G:(h + 1) * G] = o = w @ vv
            Z = scale * q.abs().amax(1, keepdim=True) / 32512 * kk.abs().sum(1).max()
            inner = A * (2.0**-11 + 2 * (1 + Z) * Z + 2.0**-21 * (z.abs().amax(1, keepdim=True) + 1) + n * 2.0**-24)
            inner = inner + 2.0**-25 * vc[:n, h].abs().sum(0) * vs[:, h].max() / S
            B[r, h * G:(h + 1) * G] = inner + (o.abs() + inner) * 2.0**-11 + 2.0**-25
    return O, B


@pytest.mark.parametrize("heads, group, rows, kv, path", [
    (1, 1 << 20, 1, 64, "tiled"),          # the most query heads: one row is 4096 blocks
    (1, 1000003, 2, 20, "tiled"),
    (1, 1048573, 1, 33, "tiled"),
    (2, 300, 3, 100, "few"),               # a row of more columns than a block
    (65535, 1, 1, 40, "few"),              # the most heads
    (65535, 5, 2, 17, "few"),
])
def test_many_heads(heads, group, rows, kv, path):
    dim, page = 64, 16
    torch.manual_seed(group)
    cache = li8.new_kv_cache(8, heads, dim, page, DEV)
    whole = li8.KVBatch(i32([0, kv]), i32([kv]), i32([[4, 1, 3, 2, 7, 5, 6]]), kv, kv, kv)
    K, V = (torch.randn((kv, heads, dim), device=DEV).to(F16) for _ in range(2))
    li8.kv_append(K, V, cache, whole)
    for x, got in zip((K, V), li8.kv_read(cache, whole)):
        # half a step of the page's scale, again where a page grew; one append: once
        half = x.abs().float().amax(dim=(0, 2)) / 127 / 2 + 2.0**-9
        assert ((x.float() - got.float()).abs() <= half[None, :, None] * 1.001).all()
    Q = (torch.randn((rows, heads * group, dim), device=DEV) * 2).to(F16)
    batch = li8.KVBatch(i32([0, rows]), i32([kv]), whole.table, rows, rows, kv)
    assert li8.kv_attention_plan(batch, cache, heads * group) == dict(path=path, splits=1)
    out = li8.kv_attention(Q, cache, batch).double()
    if heads == 1 or heads == 2:
        O, B = plain(Q, cache, whole.table[0], kv, dim ** -0.5)
        assert ((out - O).abs() <= B).all(), ((out - O).abs() / B).max()
    else:
        for h in (0, 1, 4095, 4096, 32768, 65534):
            one = li8.KVCache(*(c[:, h:h + 1].contiguous() for c in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
            O, B = plain(Q[:, h * group:(h + 1) * group], one, whole.table[0], kv, dim ** -0.5)
            assert ((out[:, h * group:(h + 1) * group] - O).abs() <= B).all(), h
        # (every head: its own, not its neighbour's)
        first = out[0, ::group] if group > 1 else out[0]
        assert (first[1:] != first[:-1]).any(1).all()


def test_strided_tables():
    """Rows of a wider table, as a server's slots are."""
    ns, ls, heads, dim, page = [3, 1, 40], [50, 2000, 90], 2, 64, 16
    t = base.Setup(ns, ls, heads, dim, page, F16, rot=64)
    wide = torch.full((7, t.width + 9), -3, dtype=torch.int32, device=DEV)
    wide[1::2, 4:4 + t.width] = t.batch.table
    strided = li8.KVBatch(t.batch.q_start, t.batch.kv_len, wide[1::2, 4:4 + t.width], t.tokens, max(ns), t.max_kv)
    assert strided.table.stride(0) == 2 * (t.width + 9)
    Q, K = t.rows(6), t.rows(heads)
    copy = li8.KVCache(*(c.clone() for c in (t.cache.k, t.cache.v, t.cache.k_scale, t.cache.v_scale)))
    for batch, cache in ((t.batch, t.cache), (strided, copy)):
        li8.kv_append(K, K, cache, batch, rope=t.rope)
    assert torch.equal(copy.k, t.cache.k) and torch.equal(copy.v, t.cache.v)
    assert torch.equal(li8.kv_attention(Q, copy, strided, rope=t.rope), li8.kv_attention(Q, t.cache, t.batch, rope=t.rope))
    for a, b in zip(li8.kv_read(copy, strided), li8.kv_read(t.cache, t.batch)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shared", [True, False])
def test_graph_of_a_chunk(shared):
    """The tiled kernel, its merge and a read captured, the workspace made inside
    the capture; replayed with other lengths, rows and pages, eager calls in between."""
    group = 2
    rows = base.tiled_blocks([70, 64], 1, group, 0, shared) * 256 // group
    t = base.Setup([70, 64], [700, 300], 1, 64, 16, F16, rot=64, max_kv=1 << 14, max_q=rows, tail=rows - 134)
    Q, K = t.rows(group), t.rows(1)
    out = torch.zeros_like(Q)
    back = torch.zeros_like(K), torch.zeros_like(K)

    def step():
        li8.kv_append(K, K, t.cache, t.batch, rope=t.rope)
        li8.kv_attention(Q, t.cache, t.batch, rope=t.rope, out=out)
        li8.kv_read(t.cache, t.batch, out=back)

    assert (li8.kv_attention_plan(t.batch, t.cache, group)["splits"] > 1) == shared
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i, (lens, starts) in enumerate((([700, 300], [0, 70, 134]), ([90, 299], [3, 20, 100]), ([650, 64], [0, 1, 65]), ([0, 7], [0, 0, 7]),
                                        ([700, 300], [0, 70, 134]))):
        Q.copy_(t.rows(group))
        K.copy_(t.rows(1, 1 + i))
        t.batch.kv_len.copy_(i32(lens))
        t.batch.q_start.copy_(i32(starts))
        before = tuple(c.clone() for c in (t.cache.k, t.cache.v, t.cache.k_scale, t.cache.v_scale))
        out.zero_()
        g.replay()
        got = out.clone(), back[0].clone(), back[1].clone(), t.cache.k.clone(), t.cache.v_scale.clone()
        torch.cuda.synchronize()
        for c, b in zip((t.cache.k, t.cache.v, t.cache.k_scale, t.cache.v_scale), before):
            c.copy_(b)
        out.zero_()
        step()
        for a, b in zip(got, (out, *back, t.cache.k, t.cache.v_scale)):
            assert torch.equal(a.nan_to_num(-1) if a.is_floating_point() else a, b.nan_to_num(-1) if b.is_floating_point() else b), i
        torch.cuda.synchronize()
