"""The key/value cache's C ABI: exported symbols, refusals on the host before
anything is launched, the plan, the index arithmetic, and the plain forms
that the GPU tests compare with.  Runs without a GPU."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

import int8_matmul_amd as li8
from oracle import kv as okv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "llm_int8_kv.h")

OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
# fake, never-dereferenced device addresses
P = 0x7F0000000000
P2 = 0x7F0000100000
MIS = 0x7F0000000008   # 8-byte aligned only
MIS2 = 0x7F0000000002  # 2-byte aligned only


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(li8.library_path()):
        import int8_matmul_amd.build as b
        b.build()
    return li8.load_library()


def cache(**kw):
    c = dict(k=P, v=P, k_scale=P, v_scale=P, pages=100, heads=4, page_size=16, head_dim=64)
    c.update(kw)
    return li8._CKVCache(*(c[n] for n, _ in li8._CKVCache._fields_))


def batch(**kw):
    b = dict(q_start=P, kv_len=P, table=P, table_stride=8, table_width=8, seqs=3, tokens=10, max_q=5,
             max_kv=100)
    b.update(kw)
    return li8._CKVBatch(*(b[n] for n, _ in li8._CKVBatch._fields_))


def rope(**kw):
    r = dict(cos=P, sin=P, rows=100, dims=64, interleaved=0)
    r.update(kw)
    return li8._CRope(*(r[n] for n, _ in li8._CRope._fields_))


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_header_functions_are_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(int8_kv_[a-z0-9_]*)\s*\(", src))
    assert names == {"int8_kv_append", "int8_kv_read", "int8_kv_attention",
                     "int8_kv_attention_workspace_bytes", "int8_kv_attention_plan"}
    raw = ctypes.CDLL(li8.library_path())
    for n in names:
        ctypes.cast(getattr(raw, n), ctypes.c_void_p)


def append(lib, c=None, b=None, r=None, K=P, ks=256, V=P, vs=256, dt=0):
    return lib.int8_kv_append(K, ks, V, vs, dt, ref(r), ref(b or batch()), ref(c or cache()), None)


def read(lib, c=None, b=None, K=P, ks=256, V=P, vs=256, dt=0):
    return lib.int8_kv_read(ref(c or cache()), ref(b or batch()), dt, K, ks, V, vs, None)


def attend(lib, c=None, b=None, r=None, Q=P, qs=512, dt=0, heads=8, scale=0.125, causal=1, window=0, O=P2,
           os_=512, lse=None, ws=P, wsb=1 << 40):
    return lib.int8_kv_attention(Q, qs, dt, heads, scale, ref(r), causal, window, ref(b or batch()),
                                 ref(c or cache()), O, os_, lse, ws, wsb, None)


@pytest.mark.parametrize("bad, status", [
    (dict(head_dim=80), SHAPE), (dict(head_dim=0), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=48), SHAPE), (dict(page_size=256), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=65536), SHAPE), (dict(pages=-1), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(pages=0), SHAPE), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID), (dict(k=MIS), ALIGN),
    (dict(v=MIS), ALIGN), (dict(k_scale=MIS2), ALIGN), (dict(v_scale=MIS2), ALIGN)])
def test_bad_cache(lib, bad, status):
    c = cache(**bad)
    assert append(lib, c=c) == status
    assert read(lib, c=c) == status
    assert attend(lib, c=c, heads=8 * max(1, c.heads) if c.heads < 100 else c.heads) == status


@pytest.mark.parametrize("bad, status", [
    (dict(seqs=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(max_q=-1), SHAPE), (dict(max_kv=-1), SHAPE),
    (dict(max_kv=129), SHAPE), (dict(table_width=-1), SHAPE), (dict(table_stride=7), SHAPE),
    (dict(table_width=1 << 27, table_stride=1 << 27, max_kv=(1 << 30) + 1), SHAPE),
    (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID), (dict(table=None), INVALID),
    (dict(q_start=MIS2), ALIGN), (dict(kv_len=MIS2), ALIGN), (dict(table=MIS2), ALIGN)])
def test_bad_batch(lib, bad, status):
    b = batch(**bad)
    assert append(lib, b=b) == status
    assert read(lib, b=b) == status
    assert attend(lib, b=b) == status


def test_null_descriptions(lib):
    assert lib.int8_kv_append(P, 256, P, 256, 0, None, None, ref(cache()), None) == INVALID
    assert lib.int8_kv_append(P, 256, P, 256, 0, None, ref(batch()), None, None) == INVALID
    assert lib.int8_kv_read(None, ref(batch()), 0, P, 256, P, 256, None) == INVALID
    assert lib.int8_kv_attention_workspace_bytes(None, ref(cache()), 8) == 0


@pytest.mark.parametrize("bad, status", [
    (dict(dims=0), SHAPE), (dict(dims=24), SHAPE), (dict(dims=80), SHAPE), (dict(dims=-16), SHAPE),
    (dict(rows=99), SHAPE), (dict(interleaved=2), INVALID), (dict(cos=None), INVALID),
    (dict(sin=None), INVALID), (dict(cos=MIS), ALIGN), (dict(sin=MIS), ALIGN)])
def test_bad_rope(lib, bad, status):
    assert append(lib, r=rope(**bad)) == status
    assert attend(lib, r=rope(**bad)) == status


def test_bad_tokens(lib):
    for f in (append, read):
        assert f(lib, K=None) == INVALID and f(lib, V=None) == INVALID
        assert f(lib, K=MIS) == ALIGN and f(lib, V=MIS) == ALIGN
        assert f(lib, ks=255) == ALIGN and f(lib, vs=260) == ALIGN     # not a multiple of 8
        assert f(lib, ks=248) == SHAPE and f(lib, vs=0) == SHAPE       # rows overlap
        assert f(lib, dt=2) == INVALID and f(lib, dt=-1) == INVALID
        assert f(lib, ks=(1 << 31) + 8) == SHAPE


def test_bad_attention(lib):
    assert attend(lib, Q=None) == INVALID and attend(lib, O=None) == INVALID
    assert attend(lib, Q=MIS) == ALIGN and attend(lib, O=MIS) == ALIGN
    assert attend(lib, qs=504) == SHAPE and attend(lib, os_=504) == SHAPE
    assert attend(lib, heads=6) == SHAPE and attend(lib, heads=0) == SHAPE and attend(lib, heads=-4) == SHAPE
    assert attend(lib, heads=(1 << 20) + 4) == SHAPE
    for s in (math.nan, math.inf, -0.5):
        assert attend(lib, scale=s) == INVALID
    assert attend(lib, causal=2) == INVALID and attend(lib, window=-1) == INVALID
    assert attend(lib, dt=7) == INVALID
    assert attend(lib, lse=MIS2) == ALIGN and attend(lib, ws=MIS) == ALIGN
    # a batch whose keys are shared between workgroups needs its workspace
    b = batch(table_width=4096, table_stride=4096, max_kv=65536, max_q=1)
    need = lib.int8_kv_attention_workspace_bytes(ref(b), ref(cache()), 8)
    assert need > 0
    assert attend(lib, b=b, ws=None, wsb=0) == WORKSPACE
    assert attend(lib, b=b, wsb=need - 1) == WORKSPACE


def test_output_over_the_queries(lib):
    """Workgroups that share a row's keys read its query at different times."""
    assert attend(lib, Q=P, O=P) == INVALID


def test_empty_calls(lib):
    for kw in (dict(seqs=0), dict(tokens=0), dict(max_q=0)):
        b = batch(**kw, q_start=None, kv_len=None, table=None)
        assert append(lib, b=b, K=None, V=None) == OK
        assert read(lib, b=b, K=None, V=None) == OK
        assert attend(lib, b=b, Q=None, O=None, ws=None, wsb=0) == OK
    # no tokens at all: nothing to store
    assert append(lib, b=batch(max_kv=0), K=None, V=None) == OK


def plan(lib, b, c, heads, causal=1, window=0):
    path, splits = ctypes.c_int32(), ctypes.c_int32()
    st = lib.int8_kv_attention_plan(ref(b), ref(c), heads, causal, window, ctypes.byref(path), ctypes.byref(splits))
    assert st == OK
    return path.value, splits.value


def test_plan(lib):
    c = cache(heads=8, head_dim=128, page_size=64)
    wide = dict(table_width=1 << 16, table_stride=1 << 16)
    assert plan(lib, batch(seqs=0), c, 8) == (0, 1)
    assert plan(lib, batch(max_q=1), c, 64) == (1, 1)                       # short: one launch
    assert plan(lib, batch(max_q=1, seqs=1, max_kv=131072, **wide), c, 64)[0] == 1
    assert plan(lib, batch(max_q=1, seqs=1, max_kv=131072, **wide), c, 64)[1] > 100
    assert plan(lib, batch(max_q=1, seqs=1, max_kv=131072, **wide), c, 64, 1, 256) == (1, 1)
    assert plan(lib, batch(max_q=512, tokens=512, max_kv=8192, **wide), c, 64) == (2, 1)
    assert plan(lib, batch(max_q=512, tokens=4, max_kv=8192, **wide), c, 8)[0] == 1     # 4 rows at most
    assert plan(lib, batch(max_q=64, tokens=512, max_kv=512, **wide), c, 64)[0] == 1    # little work
    assert plan(lib, batch(max_q=256, tokens=512, seqs=1, max_kv=8192, **wide), c, 64) == (2, 128)
    assert lib.int8_kv_attention_plan(ref(batch()), ref(c), 64, 1, 0, None, None) == INVALID
    # the workspace covers every window and both masks
    for q in (1, 5, 40, 700):
        for kv in (1, 100, 3000, 70000, 1 << 20):
            for s in (1, 7, 300):
                b = batch(max_q=q, tokens=q * s, seqs=s, max_kv=max(kv, q), **wide)
                need = lib.int8_kv_attention_workspace_bytes(ref(b), ref(c), 64)
                for w in (0, 1, 100, 5000, 1 << 30):
                    for causal in (0, 1):
                        if plan(lib, b, c, 64, causal, w)[1] > 1:
                            assert need > 0, (q, kv, s, w, causal)


def test_workspace_of_the_largest_batches(lib):
    """Past 2^30 steps nothing is shared, under a window neither: the
    workspace is asked for without one."""
    wide = dict(table_width=1 << 20, table_stride=1 << 20)
    for heads, rows, seqs, kv in ((4, 1, 512, 1 << 24), (4, 4, 512, 1 << 24), (4, 128, 32, 1 << 30),
                                  (4, 128, 16, 1 << 26), (8, 300, 2, 1 << 30)):
        c = cache(heads=heads, head_dim=128, page_size=128, pages=1 << 30)
        b = batch(max_q=rows, tokens=rows * seqs, seqs=seqs, max_kv=kv, **{**wide, "table_width": kv // 128,
                                                                           "table_stride": kv // 128})
        need = lib.int8_kv_attention_workspace_bytes(ref(b), ref(c), heads)
        for w in (0, 1, 4096, 1 << 20, 1 << 28):
            for causal in (0, 1):
                path, splits = plan(lib, b, c, heads, causal, w)
                # two slots of fp32 rows and a number for each workgroup that shares
                slots = 2 * 256 * min(rows, 256) if path == 2 else 2 * min(rows, 16)
                assert splits == 1 or need >= slots * (4 * 128 + 4), (heads, rows, seqs, kv, w, causal)


def test_index_arithmetic(tmp_path):
    exe = tmp_path / "kv_index_check"
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "int8_matmul_amd", "csrc"),
                        os.path.join(ROOT, "tests", "native", "kv_index_check.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_python_binding_rejects_cpu_tensors(lib):
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        li8.KVCache(z(2, 1, 16, 64, dtype=torch.int8), z(2, 1, 16, 64, dtype=torch.int8), z(2, 1), z(2, 1))
    with pytest.raises(ValueError):
        li8.KVBatch(z(2, dtype=torch.int32), z(1, dtype=torch.int32), z(1, 1, dtype=torch.int32), 1, 1, 16)
    with pytest.raises(ValueError):
        li8.Rope(z(4, 8), z(4, 8))


# ---- the plain forms themselves ----

def empty_cache(pages, heads, page, dim):
    return okv.Cache(np.zeros((pages, heads, page, dim), np.int8), np.zeros((pages, heads, page, dim), np.int8),
                     np.zeros((pages, heads), np.float32), np.zeros((pages, heads), np.float32))


def test_oracle_append_pins():
    """The absmax maps to +-127, values come back within half a step, a page's
    second chunk raises the scale and codes the first again."""
    c = empty_cache(3, 1, 16, 64)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 1, 64)).astype(np.float32)
    okv.append(c, x, -x, [0, 5], [5], [[2]])
    s = np.abs(x).max() / np.float32(127)
    assert c.ks[2, 0] == s and np.abs(c.k[2, 0, :5]).max() == 127 and (c.k[2] == -c.v[2]).all()
    assert np.abs(c.k[2, 0, :5] * s - x[:, 0]).max() <= s * 0.5001
    assert not c.k[:2].any() and not c.k[2, 0, 5:].any()
    before = c.k[2, 0, :5].astype(np.float32) * s
    big = np.full((1, 1, 64), 10.0, np.float32)
    okv.append(c, big, big, [0, 1], [6], [[2]])
    assert c.ks[2, 0] == np.float32(10) / np.float32(127) and (c.k[2, 0, 5] == 127).all()
    assert np.abs(c.k[2, 0, :5] * c.ks[2, 0] - before).max() <= c.ks[2, 0] * 0.5001
    okv.append(c, x[:1], x[:1], [0, 1], [1], [[2]])       # position 0 again: the page forgets
    assert c.ks[2, 0] == np.abs(x[0]).max() / np.float32(127)


def test_oracle_rotation_pins():
    pos, half = 7, 32
    ang = np.arange(16)[:, None] * (10000.0 ** (-np.arange(half) / half))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    x = np.random.default_rng(1).standard_normal((2, 128)).astype(np.float32)
    for inter in (False, True):
        y = okv.rotate(x, pos, (cos, sin, inter))
        assert (y[:, 64:] == x[:, 64:]).all()
        z = x[:, 0:64:2] + 1j * x[:, 1:64:2] if inter else x[:, :32] + 1j * x[:, 32:64]
        w = y[:, 0:64:2] + 1j * y[:, 1:64:2] if inter else y[:, :32] + 1j * y[:, 32:64]
        assert np.abs(w - z * np.exp(1j * ang[pos])).max() < 1e-5
    # scores depend on the distance alone
    a, b = np.random.default_rng(2).standard_normal((2, 1, 64)).astype(np.float32)
    r = (cos, sin, False)
    assert abs((okv.rotate(a, 9, r) @ okv.rotate(b, 4, r).T - okv.rotate(a, 14, r) @ okv.rotate(b, 9, r).T)[0, 0]) < 1e-4


def test_oracle_attention_pins():
    rng = np.random.default_rng(3)
    c = empty_cache(2, 1, 16, 64)
    x = rng.standard_normal((20, 1, 64)).astype(np.float32)
    okv.append(c, x, 2 * x, [0, 20], [20], [[1, 0]])
    K, V = okv.read(c, [0, 20], [20], [[1, 0]], 20)
    q = rng.standard_normal((20, 3, 64)).astype(np.float32)
    O, lse, _, _ = okv.attention(c, q, 0.1, [0, 20], [20], [[1, 0]])
    assert np.allclose(O[0], V[0])                                      # one key: its value
    assert np.allclose(lse[0], 0.1 * q[0] @ K[0, 0])
    O0, l0, _, _ = okv.attention(c, q, 0.0, [0, 20], [20], [[1, 0]], causal=False)
    assert np.allclose(O0, V[:, 0].mean(0)) and np.allclose(l0, np.log(20))
    O1, _, _, _ = okv.attention(c, q, 0.1, [0, 20], [20], [[1, 0]], window=1)
    assert np.allclose(O1, np.repeat(V, 3, 1))
    O2, l2, _, _ = okv.attention(c, q, 0.1, [0, 20], [12], [[1, 0]])    # 8 rows before the first token
    assert (O2[:8] == 0).all() and np.isneginf(l2[:8]).all() and np.isfinite(l2[8:]).all()


def test_more_work_items_than_a_launch_has(lib):
    """Workgroups x their size stay below 2^32 along a grid's x: sizes past it
    are refused by the checks, not by the launch."""
    wide = dict(table_width=1 << 12, table_stride=1 << 12)
    # read: 64 tokens for each of 2^24 workgroups of 256
    for seqs, q in ((1 << 17, 8192), (1 << 24, 64), (1 << 30, 1), ((1 << 31) - 1, (1 << 31) - 1)):
        assert read(lib, b=batch(seqs=seqs, tokens=(1 << 31) - 1, max_q=q)) == SHAPE
    # append: one wave for a page while its rows fit it, else four
    for seqs, q in ((1 << 26, 1), (1 << 26, 8), (1 << 22, 64), (1 << 23, 17), ((1 << 31) - 1, (1 << 31) - 1)):
        assert append(lib, b=batch(seqs=seqs, tokens=(1 << 31) - 1, max_q=q)) == SHAPE
    # attention: few columns in workgroups of 256, tiled ones of 512
    for seqs, heads, group, q, kv, path in ((1 << 20, 16, 1, 1, 16, 1), (1 << 22, 4, 9, 2, 100, 1),
                                            (1 << 15, 256, 16, 10, 100, 2), (1 << 13, 256, 1, 1000, 4096, 2),
                                            ((1 << 31) - 1, 65535, 1, (1 << 31) - 1, 16, 2)):
        c = cache(heads=heads)
        sizes = dict(tokens=(1 << 31) - 1, max_q=q, max_kv=kv, **wide)
        b = batch(seqs=seqs, **sizes)
        stride = heads * group * 64
        p, s = ctypes.c_int32(), ctypes.c_int32()
        out = ctypes.byref(p), ctypes.byref(s)
        assert lib.int8_kv_attention_plan(ref(b), ref(c), heads * group, 1, 0, *out) == SHAPE
        assert attend(lib, c=c, b=b, heads=heads * group, qs=stride, os_=stride) == SHAPE
        assert lib.int8_kv_attention_workspace_bytes(ref(b), ref(c), heads * group) == 0
        if seqs < 1 << 30:                                # one (sequence, head) fewer, or eight, is fine
            assert lib.int8_kv_attention_plan(ref(batch(seqs=seqs - 1, **sizes)), ref(c), heads * group, 1, 0, *out) == OK
            assert p.value == path


def test_scales_past_the_scores(lib):
    """From 2.4e38 on scale * log2(e) was infinite, and a query of zeros gave NaN."""
    for s in (1.0e29, 3.0e38):
        assert attend(lib, scale=s) == INVALID
    b = batch(tokens=0, q_start=None, kv_len=None, table=None)
    assert attend(lib, b=b, scale=9.9e28) == OK
