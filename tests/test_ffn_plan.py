"""Which kernels the feed-forward operators run (include/llm_int8_ffn_plan.h): symbols,
refusals and the rules' limits, on the host."""
import ctypes
import os
import re
import subprocess

import pytest

import int8_matmul_amd as li8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "llm_int8_ffn_plan.h")
OK, INVALID, SHAPE = 0, 1, 2
NAMES = ["llm_int8_backward_plan", "llm_int8_epilogue_plan"]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(li8.library_path()):
        import int8_matmul_amd.build as b
        b.build()
    return li8.load_library()


def test_every_declared_symbol_is_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(llm_int8_[a-z0-9_]*)\s*\(", src))) == NAMES
    raw = ctypes.CDLL(li8.library_path())
    for name in NAMES:
        ctypes.cast(getattr(raw, name), ctypes.c_void_p)


def test_the_header_compiles_as_c_and_holds_what_the_binding_reads(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "llm_int8_ffn_plan.h"\n'
                   "_Static_assert(sizeof(li8_epilogue_plan) == 28 && sizeof(li8_backward_plan) == 24, \"sizes\");\n"
                   "int main(void) { return LI8_BACKWARD_ROWS == 3 ? 0 : 1; }\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", "-c", str(src), "-o", str(tmp_path / "t.o")], check=True)
    text = open(HEADER).read()
    for name, keys in (("epilogue", li8.epilogue_plan(17, 16, 16)), ("backward", li8.backward_plan(17, 16, 16))):
        fields = re.search(r"typedef struct li8_%s_plan \{\s*int32_t ([^;]*);" % name, text)[1]
        assert [f.strip() for f in fields.split(",")] == list(keys)


@pytest.mark.parametrize("name", NAMES)
def test_refusals(lib, name):
    out = (ctypes.c_int32 * 8)()

    def st(T, K, N, gated=0, p=out):
        return getattr(lib, name)(T, K, N, gated, p)

    for shape in ((-1, 16, 2), (4, -16, 2), (4, 16, -2), (4, 24, 2), (4, 133152, 2), (1 << 31, 0, 2), (4, 0, 1 << 31),
                  (1 << 27, 64, 2), (4, 64, 1 << 27)):
        assert st(*shape) == SHAPE, shape
    assert st(4, 16, 3, 1) == INVALID and st(4, 16, 3, 0) == OK
    assert st(4, 16, 2, 0, None) == INVALID
    over = (1 << 25, 16, 1 << 13) if "epilogue" in name else (4, 0, (1 << 21) + 2)
    assert st(*over) == SHAPE
    with pytest.raises(li8.Int8MatmulError, match="SHAPE"):
        (li8.epilogue_plan if "epilogue" in name else li8.backward_plan)(4, 24, 2)


def test_empty_calls():
    for T, K, N in ((0, 64, 24), (40, 64, 0), (0, 0, 0)):
        assert li8.epilogue_plan(T, K, N)["path"] == li8.backward_plan(T, K, N)["path"] == "empty"
    assert li8.backward_plan(40, 0, 24)["path"] == "rows"


def test_few_tokens_go_the_layers_way():
    for T, K in ((1, 16), (16, 8192), (16, 8208), (3, 16384), (17, 16), (4096, 4096)):
        assert li8.epilogue_plan(T, K, 4096)["path"] == li8.plan(T, K, 4096)["path"]


def cd(a, b):
    return -(-a // b)


@pytest.mark.parametrize("gated", [False, True])
def test_every_grid_is_below_2_32_work_items(gated):
    """The largest N that each T allows (K = 0 bounds nothing else), and N below it: the tiles of the plan times their
    threads (512, or 256 of a pair's 64 x 128 tile)."""
    most = 0
    for T in [*range(17, 700), 1023, 1024, 1025, 4096, 4097, 65536, 1 << 20, (1 << 20) + 1, 1 << 26, (1 << 31) - 1]:
        top = min((((1 << 23) - 1) // cd(T, 256)) * 128, (1 << 31) - 2)
        for N in {top, top - 2, top // 2, top // 3, top - 126, 1 << 15, 40000, 66000}:
            N -= N % 2
            if not 0 < N <= top:
                continue
            p = li8.epilogue_plan(T, 0, N, gated)
            tiles = cd(T, p["tile_m"]) * (cd(N // 2, p["tile_n"] // 2) if gated else cd(N, p["tile_n"])) * p["ranges"]
            items = tiles * (256 if gated and p["tile_m"] == 64 else 512)
            assert items < 1 << 32, (T, N, p)
            most = max(most, items)
    assert most > 1 << 31                                  # (the limit is not far above what is reached)


def test_ranges_of_k_fit_where_the_sums_go():
    """Ranges only while all their workgroups run at once and their sums fit the gathered columns' place."""
    for T in (17, 33, 64, 65, 100, 200, 256, 300):
        for K in (256, 2048, 4096, 8208, 28672):
            for N in (2, 8, 34, 66, 130, 258, 1000, 4096, 8192):
                for gated in (False, True):
                    p = li8.epilogue_plan(T, K, N, gated)
                    if p["ranges"] > 1:
                        tiles = cd(T, 64) * (cd(N // 2, 64) if gated else cd(N, 128))
                        blocks = 2 * cd(N // 2, 32) if gated else cd(N, 32)
                        assert p["tile_m"] == 64 and tiles * p["ranges"] <= 256 and p["ranges"] <= cd(K, 128)
                        assert p["ranges"] * cd(T, 32) * blocks * 4096 <= N * K


def test_the_backward_workspace_holds_what_a_call_uses(lib):
    """The operand, its rows' factors, the strips of dbias where there are several, the ranges' sums; no more."""
    def up(n):
        return cd(n, 256) * 256

    for T in (1, 65, 300, 768, 769, 1300, 4096, 1 << 20):
        for K in (0, 16, 1040, 4096):
            for N in (1, 2, 64, 4098, 22016, 1 << 18, 1 << 21):
                if T * K >= 1 << 31 or N * K >= 1 << 31:
                    continue
                got = lib.llm_int8_backward_workspace_bytes(T, K, N)
                plans = [li8.backward_plan(T, K, N, g) for g in ([False, True] if N % 2 == 0 else [False])]
                part = up(4 * plans[0]["ranges"] * T * K) if plans[0]["ranges"] > 1 else 0
                if plans[0]["path"] == "few":
                    assert got == part
                    continue
                strips = max(p["strips"] for p in plans)
                least = up(2 * T * cd(N, 64) * 64) + up(4 * T) + part + (up(4 * strips * N) if strips > 1 else 0)
                assert got == least or (N == 1 and got >= least), (T, K, N)
