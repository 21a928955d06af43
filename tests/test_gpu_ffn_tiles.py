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


FOLD = [(400, 272, 12546, 256, 128), (64, 272, 12546, 64, 128), (400, 528, 13826, 256, 128)]


@pytest.mark.parametrize("T, K, N, tile_m, tile_n", FOLD)
@pytest.mark.parametrize("outliers", [3, 64, 65, 150, 256, 257])
def test_outlier_columns_copied_from_the_stages(T, K, N, tile_m, tile_n, outliers):
    """Both sides of the counts at which the product copies them and the prepare kernel does not gather, in a workspace
    that holds no codes."""
    print(f"case fold {T}x{K}x{N} {outliers}", flush=True)
    for gated in (False, True):
        p = li8.epilogue_plan(T, K, N, gated)
        assert (p["tile_m"], p["tile_n"], p["fold_lo"], p["fold_hi"]) == (tile_m, tile_n, 64, 256), p
    f = base.Forward(T, K, N, seed=16, fixed=outliers, residual=True)
    assert len(oracle.detect_outliers(f.X, 6.0)[1]) == outliers
    f.epilogue(activation="gelu", save=True)
    f.ws = base.dirty(f.ws.numel())
    f.gated(activation="silu", save=False)
    x, w, s = f.d["X"], f.d["Wq"], f.d["sW"]
    Y = li8.linear(x, w, s).view(torch.int16)
    pre = torch.empty((T, N), dtype=F16, device=DEV)
    assert torch.equal(li8.linear_epilogue(x, w, s, workspace=base.dirty(f.ws.numel())).view(torch.int16), Y)
    li8.gated_linear(x, w, s, pre=pre, workspace=base.dirty(f.ws.numel()))
    assert torch.equal(pre.view(torch.int16), Y)


@pytest.mark.parametrize("outliers", [6, 100, 250])
def test_a_chunk_through_an_up_projection_is_the_linear_layer(outliers):
    """512 x 5120 x 13824, whose 40 stages pass the ring many times: bit for bit the plain layer's product."""
    T, K, N = 512, 5120, 13824
    print(f"case fold {T}x{K}x{N} {outliers}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(outliers)
    x = torch.randn((T, K), generator=g, device=DEV).clamp(-5.9, 5.9).half()
    x[:, torch.randperm(K, generator=g, device=DEV)[:outliers]] *= 40
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    s = torch.rand(N, generator=g, device=DEV) * 1e-3 + 1e-4
    assert int((x.abs() > 6).any(0).sum()) == outliers and li8.epilogue_plan(T, K, N)["fold_hi"] == 256
    Y = li8.linear(x, w, s).view(torch.int16)
    ws, pre = base.dirty(li8.linear_workspace_bytes(T, K, N)), torch.empty((T, N), dtype=F16, device=DEV)
    assert torch.equal(li8.linear_epilogue(x, w, s, workspace=ws).view(torch.int16), Y)
    li8.gated_linear(x, w, s, pre=pre, workspace=base.dirty(ws.numel()))
    assert torch.equal(pre.view(torch.int16), Y)


# T, K, tile (rows 64 x 128, ranges of K), N: every tile of the epilogue variants by its plan
VARIANTS = [
    (64, 272, 12546, dict(tile_m=64, tile_n=128, ranges=1, per_cu=1), dict(tile_m=64, tile_n=128, ranges=1, per_cu=1)),
    (1024, 272, 2178, dict(tile_m=64, tile_n=128, ranges=1, per_cu=2), dict(tile_m=64, tile_n=128, ranges=1, per_cu=2)),
    (100, 4112, 258, dict(tile_m=64, tile_n=128, per_cu=1), dict(tile_m=64, tile_n=128, per_cu=1)),
    (1100, 272, 6000, dict(tile_m=256, tile_n=128, ranges=1), dict(tile_m=256, tile_n=128, ranges=1)),
    (2048, 80, 11008, dict(tile_m=256, tile_n=192, ranges=1), dict(tile_m=256, tile_n=256, ranges=1)),
    (2500, 80, 5002, dict(tile_m=256, tile_n=256, ranges=1), dict(tile_m=256, tile_n=256, ranges=1)),
]


@pytest.mark.parametrize("T, K, N, linear, gated", VARIANTS)
def test_epilogue_tiles(T, K, N, linear, gated):
    print(f"case epilogue tile {T}x{K}x{N}", flush=True)
    for want, pair in ((linear, False), (gated, True)):
        p = li8.epilogue_plan(T, K, N, pair)
        assert want.items() <= p.items() and (p["ranges"] > 1) == (T == 100), p
    f = base.Forward(T, K, N, seed=17, residual=True, sparse=1e-3)
    f.epilogue(activation="gelu_tanh")
    f.gated(activation="silu")


@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("T, K", [(5, 64), (6, 8224), (40, 64), (40, 4112)])
def test_gates_over_their_range(act, T, K):
    """Gates from -60000 to 60000, densest where the exponentials leave fp32, times up values from 2^-6 to 300: products
    past fp16's range and in the underflowed tails."""
    print(f"case gates {act} {T}x{K}", flush=True)
    F = 264
    f = base.Forward(T, K, 2 * F, seed=18, fixed=0)
    gate = np.concatenate([np.linspace(-110, 110, 200), np.exp(np.linspace(4.8, 11, 32)), -np.exp(np.linspace(4.8, 11, 32))])
    up = 2.0 ** np.random.default_rng(19).uniform(-6, 8.2, F) * (1 - 2 * (np.arange(F) % 2))
    f.bias = np.concatenate([gate, up]).astype(np.float16)
    f.d["bias"] = base.dev(f.bias)
    Hh, _ = f.gated(activation=act)
    h = base.host(Hh)
    assert np.isinf(h).any() and not np.isnan(h).any()
    assert act == "none" or (np.abs(h[:, gate < -105]) <= 2.0 ** -24).all()


@pytest.mark.parametrize("T, K, N", [(8, 11008, 4096), (16, 11008, 4096), (3, 9216, 13826), (16, 9216, 13826)])
@pytest.mark.parametrize("kw", [{}, dict(sparse=1e-3)])
def test_few_tokens_in_long_slices(T, K, N, kw):
    """Slices of K past 4096 columns (many weight rows): twice the weight loads of shorter ones in flight."""
    print(f"case long slices {T}x{K}x{N} {kw}", flush=True)
    assert li8.epilogue_plan(T, K, N, True)["path"] == "few_tokens_split"
    f = base.Forward(T, K, N, seed=23, residual=True, **kw)
    f.epilogue(activation="silu")
    f.gated(activation="gelu")
    x, w, s = f.d["X"], f.d["Wq"], f.d["sW"]
    Y = li8.linear(x, w, s).view(torch.int16)
    pre = torch.empty((T, N), dtype=F16, device=DEV)
    assert torch.equal(li8.linear_epilogue(x, w, s).view(torch.int16), Y)
    li8.gated_linear(x, w, s, pre=pre)
    assert torch.equal(pre.view(torch.int16), Y)


@pytest.mark.parametrize("T, K, N", [(50, 272, 512), (300, 272, 4098), (2050, 272, 4098), (1300, 0, 6002), (70, 48, 8202)])
@pytest.mark.parametrize("gated", [False, True])
def test_the_backward_workspace_is_enough(T, K, N, gated):
    """A workspace of exactly the bytes asked for, between others that stay as they are."""
    print(f"case workspace {T}x{K}x{N} {gated}", flush=True)
    n = li8.backward_workspace_bytes(T, K, N)
    buf = torch.full((n + (1 << 17),), 7, dtype=torch.uint8, device=DEV)
    b = base.Backward(T, K, N, gated, seed=25)
    got = b.run("silu", workspace=buf[1 << 16:(1 << 16) + n])
    assert (buf[:1 << 16] == 7).all() and (buf[(1 << 16) + n:] == 7).all()
    want = ffn.backward(b.dY, b.pre, b.Wq, b.sW, "silu", gated)
    for k, t in got.items():
        assert ffn.check(base.host(t), want[k], k) is None, ffn.check(base.host(t), want[k], k)
