"""GPU tests of the feed-forward operators' kernel variants, each with its plan asserted, so
that a change of the rules cannot leave one without a test; bounds as in test_gpu_ffn.py."""
import numpy as np
import pytest
import torch

import int8_matmul_amd as li8
import oracle
import test_gpu_ffn as base
from oracle import ffn

pytestmark = pytest.mark.gpu
DEV, F16 = base.DEV, base.F16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu tests must run on an MI355X")
    li8.load_library()


# T, K, N, the tile's rows, whether the weight's rows are split, whether dbias has several strips
TILES = [
    (385, 11024, 62, 128, False, False), (390, 11024, 450, 128, False, False), (3000, 1296, 386, 128, False, True),
    (601, 2064, 4110, 128, True, False), (2050, 272, 4098, 128, True, True),
    (700, 11024, 578, 256, False, False), (4001, 2064, 450, 256, False, True),
    (130, 11024, 4098, 256, True, False), (1500, 272, 16386, 256, True, True),
    (769, 1040, 770, 64, False, True), (770, 256, 770, 64, True, True),
]


@pytest.mark.parametrize("T, K, N, tile, split, strips", TILES)
@pytest.mark.parametrize("gated", [False, True])
def test_gradient_tiles(T, K, N, tile, split, strips, gated):
    """All elements, ragged rows too, the sums of ranges and strips in one launch among them."""
    act = ffn.ACTS[(T + N) % 5]
    for n in (N, N - 2 if gated else N - 1):
        print(f"case gradient tile {T}x{K}x{n} {gated} {act}", flush=True)
        p = li8.backward_plan(T, K, n, gated)
        assert (p["path"], p["tile"], p["ranges"] > 1, p["strips"] > 1) == ("tiled", tile, split, strips), p
        base.Backward(T, K, n, gated, seed=T + n).check(act, save=n == N, bias=True)


# training sizes: T, K, N, gated, the plan's tile, whether split, rounds of the row kernel
TRAINING = [(4096, 4096, 22016, True, 256, False, 3), (512, 5120, 27648, True, 256, True, 4),
            (4096, 11008, 4096, False, 256, False, 1), (512, 5120, 27648, False, 256, True, 0)]


@pytest.mark.parametrize("T, K, N, gated, tile, split, rounds", TRAINING)
def test_gradients_of_training_sizes(T, K, N, gated, tile, split, rounds):
    """Rows of every tile of 256, and the bias' gradient of features in several column blocks."""
    print(f"case training {T}x{K}x{N} {gated}", flush=True)
    p = li8.backward_plan(T, K, N, gated)
    assert (p["tile"], p["ranges"] > 1, p["row_rounds"]) == (tile, split, rounds), p
    F = N // 2 if gated else N
    rng = np.random.default_rng(31)
    Wq, sW = rng.integers(-127, 128, (N, K)).astype(np.int8), (rng.random(N) * 1e-3 + 1e-4).astype(np.float32)
    dY, pre = base._big((T, F), 5), base._big((T, N), 6)
    ws = base.dirty(li8.backward_workspace_bytes(T, K, N))
    g, db = torch.empty((T, N), dtype=F16, device=DEV), torch.empty(N, device=DEV)
    kw = dict(activation="silu", grad_pre=g, dbias=db, workspace=ws)
    if gated:
        dX = li8.gated_backward(dY, pre, base.dev(Wq), base.dev(sW), **kw)
    else:
        dX = li8.linear_backward(dY, base.dev(Wq), base.dev(sW), pre=pre, **kw)
    rows = sorted({0, T - 1, *(int(i) for i in np.arange(0, T, 256) + rng.integers(0, 256, T // 256))})
    want = ffn.backward(base._rows(dY, rows), base._rows(pre, rows), Wq, sW, "silu", gated)
    for t, k in ((dX, "dX"), (g, "grad_pre")):
        assert ffn.check(base._rows(t, rows), want[k], k) is None, ffn.check(base._rows(t, rows), want[k], k)
    for f in (0, 127, 128, F // 2 + 5, F - 1):
        cols = [f, F + f] if gated else [f]
        z, ez = ffn.grad_pre(base.host(dY[:, f:f + 1]), base.host(pre[:, cols]), "silu", gated)
        w = (z.sum(0), ez.sum(0) + (T + 2) * ffn.U * (np.abs(z) + ez).sum(0))
        assert ffn.check(base.host(db[cols]), w, "dbias") is None, ffn.check(base.host(db[cols]), w, "dbias")


# features of a row, and the rounds of 512 x 8 that stay in registers
ROUNDS = [(4096, 1), (4104, 2), (8192, 2), (8200, 3), (11008, 3), (12288, 3), (12296, 4), (13824, 4), (16384, 4), (16392, 0),
          (1032, 1), (2050, 1), (4098, 2), (8190, 2), (8194, 0)]


@pytest.mark.parametrize("F, rounds", ROUNDS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])   # every form of the kernel
def test_rounds_of_long_rows(F, rounds, gated, act):
    print(f"case rounds {F} {gated} {act}", flush=True)
    N, T = F * (1 + gated), 67
    p = li8.backward_plan(T, 32, N, gated)
    assert (p["path"], p["row_threads"], p["row_rounds"]) == ("tiled", 512, rounds), p
    base.Backward(T, 32, N, gated, seed=F).check(act)


@pytest.mark.parametrize("F, rounds", [(5, 1), (8, 1), (510, 1), (512, 1), (514, 2), (1016, 2), (1022, 2), (1024, 2)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_rounds_of_short_rows(F, rounds, gated, act):
    """A wave for each row."""
    print(f"case short rows {F} {gated} {act}", flush=True)
    N, T = F * (1 + gated), 131
    p = li8.backward_plan(T, 48, N, gated)
    assert (p["path"], p["row_threads"], p["row_rounds"]) == ("tiled", 64, rounds), p
    base.Backward(T, 48, N, gated, seed=F).check(act)


@pytest.mark.parametrize("T, tile", [(20, 32), (50, 64)])
@pytest.mark.parametrize("N", [512, 510])                 # whole groups of eight, and ragged ones
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_forms_of_the_kernel_for_few_rows(T, tile, N, gated, act):
    print(f"case few rows {T} {N} {gated} {act}", flush=True)
    p = li8.backward_plan(T, 272, N, gated)
    assert (p["path"], p["tile"]) == ("few", tile), p
    base.Backward(T, 272, N, gated, seed=T).check(act)
