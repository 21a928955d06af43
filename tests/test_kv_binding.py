"""The key/value cache's Python binding on the host: what it hands to the
library.  Runs without a GPU."""
import ctypes
import os
import types

import pytest

import int8_matmul_amd as li8


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(li8.library_path()):
        import int8_matmul_amd.build as b
        b.build()
    return li8.load_library()


def described(c):
    """Stands for a KVBatch or a KVCache whose description the library reads."""
    return types.SimpleNamespace(_ref=ctypes.addressof(c), _c=c)


P = 0x7F0000000000       # never dereferenced


def cache():
    return described(li8._CKVCache(P, P, P, P, 1 << 20, 8, 64, 128))


def batch(seqs=1, tokens=512, max_q=512, max_kv=131072):
    return described(li8._CKVBatch(P, P, P, 2048, 2048, seqs, tokens, max_q, max_kv))


@pytest.mark.parametrize("window", [1 << 31, 2**32 + 256, 2**63, -(1 << 31) - 1, 2**32])
def test_windows_past_32_bits(window):
    """2^32 + 256 would reach the library as 256."""
    with pytest.raises(ValueError):
        li8.kv_attention_plan(batch(), cache(), 64, window=window)


@pytest.mark.parametrize("heads", [1 << 31, 2**32 + 64])
def test_heads_past_32_bits(heads):
    with pytest.raises(ValueError):
        li8.kv_attention_plan(batch(), cache(), heads)
    with pytest.raises(ValueError):
        li8.kv_attention_workspace_bytes(batch(), cache(), heads)


def test_numbers_within_32_bits():
    wide = li8.kv_attention_plan(batch(), cache(), 64, window=(1 << 31) - 1)
    assert wide == li8.kv_attention_plan(batch(), cache(), 64)
    assert li8.kv_attention_plan(batch(tokens=1, max_q=1), cache(), 64, window=256)["splits"] == 1
    with pytest.raises(TypeError):
        li8.kv_attention_plan(batch(), cache(), 64, window=256.0)
    with pytest.raises(li8.Int8MatmulError):
        li8.kv_attention_plan(batch(), cache(), 64, window=-1)


def test_described_objects_are_fixed(monkeypatch):
    """KVCache and Rope once more without a GPU."""
    import torch
    monkeypatch.setattr(li8, "_require", lambda *a: None)
    k, s = torch.zeros((2, 1, 16, 64), dtype=torch.int8), torch.zeros((2, 1))
    cache, rope = li8.KVCache(k, k, s, s), li8.Rope(torch.zeros(4, 8), torch.zeros(4, 8))
    for thing, name in ((cache, "k"), (cache, "pages"), (rope, "cos"), (rope, "extra")):
        with pytest.raises(AttributeError):
            setattr(thing, name, None)
    with pytest.raises(AttributeError):
        del cache.k
    assert cache._c.k == cache.k.data_ptr() and rope._c.cos == rope.cos.data_ptr()
