"""The C ABI of the feed-forward operators: every declared symbol is exported, and
bad arguments are refused on the host before anything is launched.

These run without a GPU: every call here either fails validation or is empty,
and neither makes a HIP call.
"""
import ctypes
import os
import re

import pytest
import torch

import int8_matmul_amd as li8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "llm_int8_ffn.h")
OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
P, MIS = 0x7F0000000000, 0x7F0000000008   # never dereferenced; 8-byte aligned only
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(li8.library_path()):
        import int8_matmul_amd.build as b
        b.build()
    return li8.load_library()


def declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(llm_int8_[a-z0-9_]*)\s*\(", src)))


def test_every_declared_symbol_is_exported(lib):
    assert declared() == sorted(["llm_int8_linear_epilogue", "llm_int8_gated_linear", "llm_int8_backward_workspace_bytes",
                                 "llm_int8_linear_backward", "llm_int8_gated_backward"])
    raw = ctypes.CDLL(li8.library_path())
    for name in declared():
        ctypes.cast(getattr(raw, name), ctypes.c_void_p)


def test_the_header_compiles_as_c(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "llm_int8_ffn.h"\nint main(void) { return LI8_ACT_GELU_TANH == 4 ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", "-c", str(src), "-o", str(tmp_path / "t.o")], check=True)


def test_activations_are_the_headers():
    src = open(HEADER).read()
    got = {m[0].lower(): int(m[1]) for m in re.findall(r"LI8_ACT_([A-Z_]+) = (\d+)", src)}
    assert got == li8.ACTIVATIONS


EPILOGUE = dict(X=P, Wq=P, sW=P, threshold=6.0, T=40, K=64, N=24, bias=P, act=2, residual=P, Y=P, pre=P, ws=P, size=BIG)
GATED = dict(X=P, Wq=P, sW=P, threshold=6.0, T=40, K=64, F=24, bias=P, act=2, H=P, pre=P, ws=P, size=BIG)
BACK = dict(dY=P, pre=P, act=2, Wq=P, sW=P, T=40, K=64, N=24, dX=P, grad_pre=P, dbias=P, ws=P, size=BIG)
FORWARD_CALLS = [("llm_int8_linear_epilogue", EPILOGUE, "N", "Y"), ("llm_int8_gated_linear", GATED, "F", "H")]
BACK_CALLS = ["llm_int8_linear_backward", "llm_int8_gated_backward"]


def call(lib, name, base, **changes):
    assert not set(changes) - set(base)
    return getattr(lib, name)(*{**base, **changes}.values(), None)


@pytest.mark.parametrize("name, base, wide, out", FORWARD_CALLS)
def test_forward_refusals(lib, name, base, wide, out):
    def st(**kw):
        return call(lib, name, base, **kw)

    for kw in (dict(T=-1), dict(K=-16), {wide: -1}, dict(K=24), dict(K=133152), dict(T=1 << 31, K=0), {wide: 1 << 31},
               dict(T=1 << 27, K=64), {wide: 1 << 27, "K": 64}, {wide: (1 << 63) - 1}, {wide: 1 << 62}):
        assert st(**kw) == SHAPE, kw
    # grids of 2^32 work-items and more
    assert st(T=1 << 25, K=16, **{wide: 1 << 13}) == SHAPE
    for kw in (dict(threshold=float("nan")), dict(threshold=-0.5), dict(act=-1), dict(act=5), dict(X=None), dict(Wq=None),
               dict(sW=None), {out: None}):
        assert st(**kw) == INVALID, kw
    for p in [k for k, v in base.items() if v == P]:
        assert st(**{p: MIS}) == ALIGN, p
    need = lib.llm_int8_linear_workspace_bytes(40, 64, 24 if wide == "N" else 48)
    assert need > 0 and st(size=need - 1) == WORKSPACE and st(ws=None) == WORKSPACE
    # an empty call is valid whatever its pointers are
    assert st(T=0, X=None, ws=None, size=0, **{out: None}) == OK
    assert st(**{wide: 0, "Wq": None, "sW": None, out: None, "ws": None, "size": 0}) == OK


@pytest.mark.parametrize("name", BACK_CALLS)
def test_backward_refusals(lib, name):
    gated = "gated" in name

    def st(**kw):
        return call(lib, name, BACK, **kw)

    for kw in (dict(T=-1), dict(K=-16), dict(N=-1), dict(K=24), dict(K=133152), dict(T=1 << 31, K=0), dict(N=1 << 31),
               dict(T=1 << 27), dict(N=1 << 27), dict(N=(1 << 63) - 1), dict(N=(1 << 21) + 1, K=16),
               dict(N=(1 << 20) + 1, K=16) if gated else dict(N=1 << 22, K=16)):
        assert st(**kw) == SHAPE, kw
    for kw in (dict(act=-1), dict(act=5), dict(dY=None), dict(pre=None), dict(Wq=None), dict(sW=None), dict(dX=None)):
        assert st(**kw) == INVALID, kw
    if gated:   # the pair's values are read whatever the activation is
        assert st(act=0, pre=None) == INVALID
    for p in [k for k, v in BACK.items() if v == P]:
        assert st(**{p: MIS}) == ALIGN, p
    need = lib.llm_int8_backward_workspace_bytes(100, 64, 48 if gated else 24)
    assert need > 0 and st(T=100, size=need - 1) == WORKSPACE and st(T=100, ws=None) == WORKSPACE
    # nothing to write: no tokens and no bias gradient, or no features
    assert st(T=0, dY=None, pre=None, dX=None, dbias=None, ws=None, size=0) == OK
    assert st(T=0, N=0, dbias=None) == OK and st(N=0, K=0, dX=None) == OK and st(N=0, T=0, dbias=P) == OK


def test_backward_workspace_bytes(lib):
    ws = lib.llm_int8_backward_workspace_bytes
    assert ws(0, 64, 24) == ws(40, 64, 0) == ws(-1, 64, 24) == ws(40, 24, 24) == ws(40, 64, (1 << 21) + 1) == 0
    assert ws(40, 64, 24) == 0   # few rows, one range of the weight's rows: none needed
    # many rows: the fp16 operand of the product, and no partial sums
    assert 2 * 4096 * 22016 <= ws(4096, 4096, 22016) < 2 * 4096 * 22016 + (8 << 20)
    # few rows: partial sums only
    assert ws(8, 1024, 1024) == 8 * 4 * 8 * 1024
    for T in (1, 16, 17, 32, 33, 64, 65, 128, 129, 300, 4096):
        for K in (16, 256, 1040, 11008):
            for N in (1, 63, 64, 65, 4096, 9000):
                assert ws(T, K, N) % 256 == 0
    assert ws(40, 0, 24) > 0     # (no product, but dbias and grad_pre)


def test_the_binding_refuses_on_the_host():
    """What needs no GPU: tensors that are not on one."""
    x = torch.zeros((4, 16), dtype=torch.float16)
    w, s = torch.zeros((8, 16), dtype=torch.int8), torch.zeros(8)
    y = torch.zeros((4, 8), dtype=torch.float16)
    for f in (lambda: li8.linear_epilogue(x, w, s), lambda: li8.gated_linear(x, w, s), lambda: li8.linear_backward(y, w, s),
              lambda: li8.gated_backward(y[:, :4], y, w, s)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    for f in (lambda: li8.linear_epilogue(None, w, s), lambda: li8.gated_backward([1], y, w, s)):
        with pytest.raises(TypeError):
            f()


def test_backward_refuses_more_rows_than_the_column_sums_count(lib):
    """K = 0 allows rows past 2^30, where stepping past the last row would leave 32 bits."""
    for name in BACK_CALLS:
        for T in ((1 << 30) + 1, (1 << 31) - 1):
            assert call(lib, name, BACK, T=T, K=0, N=1) == SHAPE
            assert lib.llm_int8_backward_workspace_bytes(T, 0, 2) == 0
    assert lib.llm_int8_backward_workspace_bytes(1 << 30, 0, 2) > 0
