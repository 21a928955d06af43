"""GPU tests of the feed-forward operators against their 64-bit forms: every element
within the bound of its own roundings (oracle/ffn.py), at the edges of sizes and values.
(test_gpu_ffn_tiles.py goes through the kernel variants by their plans.)"""
import dataclasses

import numpy as np
import pytest
import torch

import int8_matmul_amd as li8
import oracle
import workloads
from oracle import ffn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu tests must run on an MI355X")
    li8.load_library()


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def guarded(shape, dtype=F16, rows=3):
    """A tensor inside a larger buffer of a marker value; check with `intact`."""
    n = int(np.prod(shape))
    pad = 64 * rows
    buf = torch.full((n + 2 * pad,), 7.75, dtype=dtype, device=DEV)
    return buf, buf[pad:pad + n].view(shape)


def intact(buf, view):
    pad = (buf.numel() - view.numel()) // 2
    return bool((buf[:pad] == 7.75).all()) and bool((buf[pad + view.numel():] == 7.75).all())


def dirty(n):
    """A workspace full of NaN patterns, of exactly n bytes."""
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)


class Forward:
    def __init__(self, T, K, N, seed=0, sparse=0.0, fixed=2, bias=True, residual=False):
        rng = np.random.default_rng(seed)
        w = dataclasses.replace(workloads.WORKLOADS["ffn_13b"], T=T, K=K, N=N, sparse_rate=sparse, n_fixed=min(fixed, K))
        self.T, self.K, self.N = T, K, N
        self.X, _ = workloads.make_activation(w, seed=seed)
        self.W = (rng.standard_normal((N, K)) * 0.05 * np.exp(0.3 * rng.standard_normal((N, 1)))).astype(np.float16)
        self.Wq, self.sW = oracle.quantize_weight(self.W)
        self.bias = (rng.standard_normal(N) * 0.7).astype(np.float16) if bias else None
        self.residual = (rng.standard_normal((T, N)) * 3).astype(np.float16) if residual else None
        self.d = {k: dev(getattr(self, k)) for k in ("X", "Wq", "sW", "bias", "residual")}
        self.ws = dirty(li8.linear_workspace_bytes(T, K, N))

    def epilogue(self, threshold=6.0, activation="none", save=True, in_place=False):
        yb, Y = guarded((self.T, self.N))
        pb, pre = guarded((self.T, self.N))
        res = self.d["residual"]
        if in_place:
            Y.copy_(res)
            res = Y
        li8.linear_epilogue(self.d["X"], self.d["Wq"], self.d["sW"], threshold, bias=self.d["bias"], activation=activation,
                            residual=res, out=Y, pre=pre if save else None, workspace=self.ws)
        want, wpre = ffn.linear_epilogue(self.X, self.Wq, self.sW, threshold, self.bias, activation, self.residual)
        assert ffn.check(host(Y), want, "Y") is None, ffn.check(host(Y), want, "Y")
        if save:
            assert ffn.check(host(pre), wpre, "pre") is None, ffn.check(host(pre), wpre, "pre")
        assert intact(yb, Y) and intact(pb, pre)
        return Y, pre

    def gated(self, threshold=6.0, activation="silu", save=True):
        hb, Hh = guarded((self.T, self.N // 2))
        pb, pre = guarded((self.T, self.N))
        li8.gated_linear(self.d["X"], self.d["Wq"], self.d["sW"], threshold, bias=self.d["bias"], activation=activation, out=Hh,
                         pre=pre if save else None, workspace=self.ws)
        want, wpre = ffn.gated_linear(self.X, self.Wq, self.sW, threshold, self.bias, activation)
        assert ffn.check(host(Hh), want, "H") is None, ffn.check(host(Hh), want, "H")
        if save:
            assert ffn.check(host(pre), wpre, "pre") is None, ffn.check(host(pre), wpre, "pre")
        assert intact(hb, Hh) and intact(pb, pre)
        return Hh, pre


# T, K, N of the weight's rows (2F of a pair), further options; by kernel
FEW = [
    (1, 16, 2, {}), (1, 4096, 34, {}), (2, 272, 100, {}), (8, 1024, 520, {}), (7, 4096, 46, dict(sparse=4e-3)),
    (3, 512, 4230, {}),                                    # more row groups than workgroups, 8 token slots
    (16, 512, 4186, dict(sparse=1e-2)), (12, 48, 130, {}),  # 16 token slots
    (4, 4112, 70, {}), (16, 8192, 90, dict(sparse=1e-3)), (9, 5120, 4110, {}),   # K past 4096
    (5, 640, 66, dict(fixed=300)),                         # more outlier columns than the LDS list holds
]
SPLIT = [(1, 8208, 40, {}), (16, 11008, 74, dict(sparse=5e-4)), (8, 9216, 4106, {}), (3, 16384, 18, {})]
TILED = [
    (17, 16, 8, {}), (40, 64, 6, {}), (64, 272, 130, dict(sparse=1e-2)), (300, 1040, 520, dict(sparse=2e-3)),
    (257, 512, 1002, {}), (129, 4096, 258, {}), (513, 256, 2730, {}), (33, 8208, 100, {}),
    (100, 528, 384, dict(fixed=400)),                      # every second column an outlier, gathered by the prepare kernel
]
# the larger tiles, which few rows do not take (outlier columns gathered)
WIDE = [(2048, 64, 11008, 192, {}), (2500, 64, 5000, 256, {}), (1100, 272, 6000, 128, dict(sparse=2e-3)),
        (1100, 272, 5998, 128, {}), (1100, 528, 6010, 128, dict(fixed=400))]


@pytest.mark.parametrize("T, K, N, kw", FEW + SPLIT + TILED)
@pytest.mark.parametrize("i", [0, 1])
def test_epilogue(T, K, N, kw, i):
    act = ffn.ACTS[(T + K + 2 * i) % 5]
    print(f"case epilogue {T}x{K}x{N} {act} {i}", flush=True)
    path = li8.plan(T, K, N)["path"]
    assert path == ("few_tokens" if T <= 16 and K <= 8192 else "few_tokens_split" if T <= 16 else "tiled")
    N -= i                                                 # odd widths too
    f = Forward(T, K, N, seed=T + N, residual=i == 0, bias=i == 1 or T % 2 == 0, **kw)
    f.epilogue(activation=act, save=i == 1)
    f.epilogue(activation=act, save=i == 0)


@pytest.mark.parametrize("T, K, N, kw", FEW + SPLIT + TILED)
@pytest.mark.parametrize("i", [0, 1])
def test_gated(T, K, N, kw, i):
    act = ffn.ACTS[(T + K + 2 * i + 1) % 5]
    print(f"case gated {T}x{K}x{N} {act} {i}", flush=True)
    N = max(2, N - 2 * i * (1 + T % 3))                    # F odd, and not a multiple of 8
    f = Forward(T, K, N, seed=T + N, bias=i == 1, **kw)
    f.gated(activation=act, save=True)
    f.gated(activation=act, save=False)


@pytest.mark.parametrize("T, K, N, tile, kw", WIDE)
def test_wide_tiles(T, K, N, tile, kw):
    print(f"case wide {T}x{K}x{N}", flush=True)
    assert li8.plan(T, K, N)["tile_n"] == tile
    f = Forward(T, K, N, seed=3, residual=True, **kw)
    f.epilogue(activation="gelu", save=False)
    f.epilogue(activation="none", save=True)
    f.gated(activation="silu", save=tile != 192)


@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("T", [5, 40])
def test_every_activation_over_its_range(act, T):
    """Arguments from far below to far above, through a weight of one row pair: every
    act at arguments past where it saturates, products included."""
    print(f"case range {act} {T}", flush=True)
    f = Forward(T, 64, 128, seed=9, fixed=0)
    f.bias = (np.sign(np.arange(128) - 31.5) * np.exp(np.linspace(-9, 10.8, 128))).astype(np.float16)
    f.bias[64:] = np.linspace(-60000, 60000, 64).astype(np.float16)
    f.d["bias"] = dev(f.bias)
    f.epilogue(activation=act)
    f.gated(activation=act) if act in ("relu", "none") else None


@pytest.mark.parametrize("threshold", [0.0, 6.0, float("inf")])
@pytest.mark.parametrize("T, K, N", [(6, 256, 66), (6, 8224, 34), (50, 256, 66)])
def test_thresholds(T, K, N, threshold):
    print(f"case threshold {T}x{K}x{N} {threshold}", flush=True)
    f = Forward(T, K, N, seed=1, residual=True, sparse=1e-2)
    f.epilogue(threshold, "silu")
    f.gated(threshold, "gelu_tanh")


@pytest.mark.parametrize("T, K, N", [(1, 64, 40), (8, 8208, 33), (70, 64, 40), (300, 128, 131), (2048, 64, 11008), (1100, 64, 6001)])
@pytest.mark.parametrize("save", [False, True])
def test_residual_in_place(T, K, N, save):
    print(f"case in place {T}x{K}x{N} {save}", flush=True)
    f = Forward(T, K, N, seed=2, residual=True)
    f.epilogue(activation="gelu", save=save, in_place=True)


@pytest.mark.parametrize("T, K, N", [(1, 4096, 520), (8, 512, 4200), (12, 512, 4200), (16, 8192, 64), (7, 11008, 72), (300, 1040, 520),
                                     (2048, 64, 11008), (2500, 64, 5000), (1100, 272, 6000)])
def test_without_extras_it_is_the_linear_layer(T, K, N):
    """Bit for bit: the product stays fp32 up to the same single rounding."""
    print(f"case plain {T}x{K}x{N}", flush=True)
    f = Forward(T, K, N, seed=4, bias=False, sparse=2e-3)
    x, w, s = f.d["X"], f.d["Wq"], f.d["sW"]
    Y = li8.linear(x, w, s)
    pre, pre2 = torch.empty_like(Y), torch.empty_like(Y)
    assert torch.equal(li8.linear_epilogue(x, w, s, pre=pre).view(torch.int16), Y.view(torch.int16))
    li8.gated_linear(x, w, s, pre=pre2)
    assert torch.equal(pre.view(torch.int16), Y.view(torch.int16)) and torch.equal(pre2.view(torch.int16), Y.view(torch.int16))


def test_no_features_of_the_input():
    """K = 0: Z is the bias."""
    for T in (3, 40):
        x, w, s = (torch.empty(sh, dtype=d, device=DEV) for sh, d in (((T, 0), F16), ((20, 0), torch.int8), ((20,), torch.float32)))
        s.fill_(1)
        b = torch.randn(20, device=DEV).half()
        r = torch.randn(T, 20, device=DEV).half()
        y = li8.linear_epilogue(x, w, s, bias=b, activation="relu", residual=r)
        assert torch.equal(y, (b.float().clamp(min=0) + r.float()).half())
        h = li8.gated_linear(x, w, s, bias=b, activation="relu")
        assert torch.equal(h, (b[:10].float().clamp(min=0) * b[10:].float()).half().expand(T, 10))


class Backward:
    def __init__(self, T, K, N, gated, seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.T, self.K, self.N, self.is_gated = T, K, N, gated
        F = N // 2 if gated else N
        self.Wq, self.sW = oracle.quantize_weight(
            (rng.standard_normal((N, K)) * 0.05 * np.exp(0.5 * rng.standard_normal((N, 1)))).astype(np.float16))
        self.dY = (rng.standard_normal((T, F)) * 1e-2 * np.exp(spread * rng.standard_normal((T, 1)))).astype(np.float16)
        self.pre = (rng.standard_normal((T, N)) * 1.5).astype(np.float16)

    def run(self, activation, save=True, bias=True, workspace=None):
        dY, pre, w, s = (dev(a) for a in (self.dY, self.pre, self.Wq, self.sW))
        xb, dX = guarded((self.T, self.K))
        gb, g = guarded((self.T, self.N))
        bb, db = guarded((self.N,), torch.float32)
        ws = dirty(li8.backward_workspace_bytes(self.T, self.K, self.N)) if workspace is None else workspace
        kw = dict(activation=activation, out=dX, grad_pre=g if save else None, dbias=db if bias else None, workspace=ws)
        if self.is_gated:
            li8.gated_backward(dY, pre, w, s, **kw)
        else:
            li8.linear_backward(dY, w, s, pre=None if activation == "none" else pre, **kw)
        torch.cuda.synchronize()
        assert intact(xb, dX) and intact(gb, g) and intact(bb, db)
        return dict(dX=dX, grad_pre=g if save else None, dbias=db if bias else None)

    def check(self, activation, save=True, bias=True):
        got = self.run(activation, save, bias)
        want = ffn.backward(self.dY, self.pre, self.Wq, self.sW, activation, self.is_gated)
        for k, t in got.items():
            if t is not None:
                assert ffn.check(host(t), want[k], k) is None, ffn.check(host(t), want[k], k)
        # as independent errors (256 of them and more: 1.25 of the expected norm is past four deviations)
        if self.T * self.K >= 256 and want["dX_norm"] > 0:
            err = np.linalg.norm(host(got["dX"]).astype(np.float64) - want["dX"][0])
            assert err <= 1.25 * want["dX_norm"] + 2.0 ** -25 * np.sqrt(self.T * self.K), (err, want["dX_norm"])
        return got


ROWS = [
    # one kernel for few rows: one range and several, one to four stages, every chunk border
    (1, 16, 2), (1, 4096, 4096), (3, 48, 62), (16, 256, 64), (17, 272, 66), (32, 512, 256), (33, 1040, 258), (37, 304, 1000),
    (48, 256, 2050), (49, 512, 2046), (64, 1024, 514), (5, 4096, 300), (8, 64, 8190),
    # few rows, long weight
    (2, 5120, 4400), (20, 8448, 2048), (40, 11008, 1030), (64, 4096, 5002),
    # tiles of 32 and 64 rows, split and not, one stage and more
    (65, 16, 2), (100, 256, 64), (128, 272, 130), (129, 1040, 514), (256, 512, 1000), (257, 272, 4106), (300, 16, 62),
    (700, 2064, 770), (2050, 256, 66),
]


@pytest.mark.parametrize("T, K, N", ROWS)
@pytest.mark.parametrize("gated", [False, True])
def test_backward(T, K, N, gated):
    act = ffn.ACTS[(T + N) % 5]
    for i, n in enumerate((N, N - 2 if gated else N - 1)):   # ragged rows too
        if n < 1 + gated:
            continue
        print(f"case backward {T}x{K}x{n} {gated} {act} {i}", flush=True)
        Backward(T, K, n, gated, seed=T + n).check(act, save=(T + i) % 2 == 0, bias=(K // 16 + i) % 2 == 0)


@pytest.mark.parametrize("N", [4100, 8192, 8194, 12290, 16400, 33000])
@pytest.mark.parametrize("gated", [False, True])
def test_long_rows(N, gated):
    """One to four rounds of a row's features in registers, and rows past that."""
    N *= 1 + gated
    print(f"case long rows {N} {gated}", flush=True)
    Backward(66, 32, N, gated, seed=N).check("silu")


@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [20, 70])
def test_every_slope(act, gated, T):
    print(f"case slope {act} {gated} {T}", flush=True)
    b = Backward(T, 48, 512, gated, seed=8)
    b.pre = np.linspace(-14, 14, T * 512).reshape(T, 512).astype(np.float16)
    b.pre[0, :8] = [0.0, -0.0, 65504, -65504, 6e-8, -6e-8, 300, -300]
    b.check(act)


@pytest.mark.parametrize("T", [9, 70, 300])
def test_gradients_of_any_size(T):
    """Rows from below fp16's normal range to its end, rows of zeros, and one feature far
    above the others: the rows' own units keep the relative precision."""
    print(f"case sizes {T}", flush=True)
    b = Backward(T, 272, 600, False, seed=3)
    rng = np.random.default_rng(4)
    size = 2.0 ** np.linspace(-24, 13, T)[:, None]
    b.dY = (rng.standard_normal((T, 600)) * size).clip(-65504, 65504).astype(np.float16)
    b.dY[T // 2] = 0
    b.dY[T // 3, 17] = 60000
    b.check("none")


@pytest.mark.parametrize("T", [9, 70, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_with_infinities_stay_alone(T, gated):
    """A row with an infinity or NaN gives a row of infinities and NaN, and the other rows are as they were."""
    print(f"case infinities {T} {gated}", flush=True)
    b = Backward(T, 144, 520, gated, seed=5)
    act = "silu"
    clean = {k: host(v).copy() for k, v in b.run(act).items()}
    b.dY[2, 3], b.dY[T - 1, 200] = np.inf, np.nan
    got = {k: host(v) for k, v in b.run(act).items()}
    rest = [t for t in range(T) if t not in (2, T - 1)]
    assert np.array_equal(got["dX"][rest], clean["dX"][rest])
    assert not np.isfinite(got["dX"][[2, T - 1]]).any()
    assert np.array_equal(got["grad_pre"][rest], clean["grad_pre"][rest])
    wide = [n for n in range(520) if n % (260 if gated else 520) not in (3, 200)]
    assert np.array_equal(got["dbias"][wide], clean["dbias"][wide])


@pytest.mark.parametrize("T", [9, 70])
def test_weight_rows_of_zeros(T):
    b = Backward(T, 64, 130, False, seed=6)
    b.Wq[:], b.sW[:] = 0, 0
    got = b.check("gelu")
    assert not host(got["dX"]).any()


def test_empty_backward_calls():
    w, s = torch.zeros((20, 32), dtype=torch.int8, device=DEV), torch.ones(20, device=DEV)
    db = torch.full((20,), 3.0, device=DEV)
    assert li8.linear_backward(torch.empty((0, 20), dtype=F16, device=DEV), w, s, dbias=db).shape == (0, 32)
    assert not host(db).any()                               # the sum over no tokens
    for T in (5, 100):                                      # no features: a gradient of zeros
        out = torch.full((T, 32), 3.0, dtype=F16, device=DEV)
        li8.linear_backward(torch.empty((T, 0), dtype=F16, device=DEV), w[:0], s[:0], out=out)
        assert not host(out).any()
        # no columns: the bias' gradient and dZ all the same
        dY = torch.randn((T, 20), device=DEV).half()
        g, db = torch.empty_like(dY), torch.empty(20, device=DEV)
        li8.linear_backward(dY, w[:, :0].contiguous(), s, grad_pre=g, dbias=db)
        assert torch.equal(g, dY) and torch.allclose(db, dY.float().sum(0), rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T, N", [(8, 600), (64, 5002), (150, 640), (600, 600)])
def test_the_same_call_gives_the_same_bits(T, N, gated):
    b = Backward(T, 1040, N, gated, seed=7)
    first = {k: host(v).copy() for k, v in b.run("gelu").items()}
    for _ in range(3):
        again = b.run("gelu")
        for k in first:
            assert np.array_equal(first[k].view(np.uint8), host(again[k]).view(np.uint8)), k


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [11, 200])
def test_gradient_against_differences(T, gated):
    """The directional derivative of the smooth product, by central differences in 64
    bits, against the kernel's dX and dbias: off by dX's own bound along that
    direction (as independent errors, four deviations) and the differences' 1e-6."""
    rng = np.random.default_rng(12)
    K, F = 96, 70
    N = 2 * F if gated else F
    b = Backward(T, K, N, gated, seed=13)
    W = b.Wq.astype(np.float64) * b.sW.astype(np.float64)[:, None]
    X, bias = rng.standard_normal((T, K)), rng.standard_normal(N)
    b.pre = (X @ W.T + bias).astype(np.float16)
    X = np.linalg.lstsq(W, (b.pre.astype(np.float64) - bias).T, rcond=None)[0].T if not gated and K >= N else X
    base = b.pre.astype(np.float64)                         # where the forward call's values are
    dY = b.dY.astype(np.float64)

    def value(z):
        y = ffn.act(z[:, :F], "silu")[0] * z[:, F:] if gated else ffn.act(z, "silu")[0]
        return (dY * y).sum()

    got = b.run("silu")
    dX, db = host(got["dX"]).astype(np.float64), host(got["dbias"]).astype(np.float64)
    want = ffn.backward(b.dY, b.pre, b.Wq, b.sW, "silu", gated)
    h = 1e-5
    for _ in range(4):
        V, c = rng.standard_normal((T, K)), rng.standard_normal(N)
        dx = (value(base + h * (V @ W.T)) - value(base - h * (V @ W.T))) / (2 * h)
        assert abs((dX * V).sum() - dx) <= 4 * want["dX_norm"] + 1e-6 * max(1, abs(dx))
        dc = (value(base + h * c) - value(base - h * c)) / (2 * h)
        assert abs((db * c).sum() - dc) <= (want["dbias"][1] * np.abs(c)).sum() + 1e-6 * max(1, abs(dc))


@pytest.mark.parametrize("T", [3, 50, 300])
def test_a_feed_forward_block(T):
    """Gate and up, the down-projection added to the residual stream, and the way back, as a layer's training step calls
    them: each call takes what the last one stored, and is compared with the 64-bit form of the same inputs."""
    print(f"case block {T}", flush=True)
    K, F = 272, 432
    up = Forward(T, K, 2 * F, seed=20, bias=False, sparse=1e-3)
    down = Forward(T, F, K, seed=21, bias=False, residual=True)
    Hh, pre = up.gated(activation="silu")
    down.X = host(Hh)
    down.d["X"] = Hh.contiguous()
    Y, _ = down.epilogue(save=False)
    rng = np.random.default_rng(22)
    back = Backward(T, F, K, False)
    back.Wq, back.sW = down.Wq, down.sW
    back.dY = (rng.standard_normal((T, K)) * 1e-2).astype(np.float16)
    dH = back.check("none", save=False, bias=False)["dX"]
    back = Backward(T, K, 2 * F, True)
    back.Wq, back.sW, back.pre, back.dY = up.Wq, up.sW, host(pre), host(dH)
    got = back.check("silu", bias=False)
    assert got["dX"].shape == (T, K) and Y.shape == (T, K)


def calls(T, K, F, seed):
    """The four operators on one set of tensors, by name, and the tensors that change."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randint(-127, 128, (2 * F, K), generator=g, device=DEV, dtype=torch.int8)
    s = torch.rand(2 * F, generator=g, device=DEV) * 1e-3 + 1e-4
    x = torch.randn((T, K), generator=g, device=DEV).half()
    x[:, 3] *= 20
    dy, dh = (torch.randn((T, n), generator=g, device=DEV).half() for n in (2 * F, F))
    pre = torch.randn((T, 2 * F), generator=g, device=DEV).half()
    bias, res = torch.randn(2 * F, generator=g, device=DEV).half(), torch.randn((T, 2 * F), generator=g, device=DEV).half()
    o = dict(Y=torch.empty((T, 2 * F), dtype=F16, device=DEV), H=torch.empty((T, F), dtype=F16, device=DEV),
             P=torch.empty((T, 2 * F), dtype=F16, device=DEV), dX=torch.empty((T, K), dtype=F16, device=DEV),
             dX2=torch.empty((T, K), dtype=F16, device=DEV), db=torch.empty(2 * F, device=DEV),
             G=torch.empty((T, 2 * F), dtype=F16, device=DEV))
    fw = torch.empty(li8.linear_workspace_bytes(T, K, 2 * F), dtype=torch.uint8, device=DEV)
    bw = li8.new_backward_workspace(T, K, 2 * F, DEV)

    def run():
        li8.linear_epilogue(x, w, s, bias=bias, activation="gelu", residual=res, out=o["Y"], workspace=fw)
        li8.gated_linear(x, w, s, bias=bias, out=o["H"], pre=o["P"], workspace=fw)
        li8.linear_backward(dy, w, s, pre=pre, activation="gelu_tanh", out=o["dX"], dbias=o["db"], workspace=bw)
        li8.gated_backward(dh, pre, w, s, out=o["dX2"], grad_pre=o["G"], workspace=bw)

    return run, o, (x, dy, dh)


SIZES = [(5, 256, 40), (8, 8208, 20), (40, 1024, 520), (300, 528, 260), (50, 6160, 130)]


@pytest.mark.parametrize("T, K, F", SIZES)
def test_in_a_graph(T, K, F):
    """One graph of all four, replayed with other inputs in between."""
    print(f"case graph {T}x{K}x{F}", flush=True)
    run, o, inputs = calls(T, K, F, 1)
    run()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in o.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    kept = [t.clone() for t in inputs]
    for i in range(4):
        for t in inputs:
            t.mul_(0.5 + i)
        run()                                              # eager, other inputs, the same workspaces
        for t, k in zip(inputs, kept):
            t.copy_(k)
        for v in o.values():
            v.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k].view(torch.uint8), want[k].view(torch.uint8)), (i, k)


@pytest.mark.parametrize("T, K, F", SIZES)
def test_two_streams(T, K, F):
    """Calls with workspaces of their own on two streams at once."""
    print(f"case streams {T}x{K}x{F}", flush=True)
    runs = [calls(T, K, F, seed) for seed in (2, 3)]
    want = []
    for run, o, _ in runs:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in o.items()})
        for v in o.values():
            v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(10):
        for st, (run, _, _) in zip(streams, runs):
            with torch.cuda.stream(st):
                run()
    torch.cuda.synchronize()
    for w, (_, o, _) in zip(want, runs):
        for k in o:
            assert torch.equal(o[k].view(torch.uint8), w[k].view(torch.uint8)), k


def test_the_binding_refuses():
    x, w, s = torch.zeros((4, 32), dtype=F16, device=DEV), torch.zeros((8, 32), dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
    y, h = torch.zeros((4, 8), dtype=F16, device=DEV), torch.zeros((4, 4), dtype=F16, device=DEV)
    good = dict(linear_epilogue=(x, w, s), gated_linear=(x, w, s), linear_backward=(y, w, s), gated_backward=(h, y, w, s))
    for name, args in good.items():
        getattr(li8, name)(*args)
        first, wi, si = args[0], len(args) - 2, len(args) - 1

        def bad(err, match, i=None, value=None, **kw):
            a = list(args)
            if i is not None:
                a[i] = value
            with pytest.raises(err, match=match):
                getattr(li8, name)(*a, **kw)

        bad(TypeError, "float16", 0, first.float())
        bad(ValueError, "contiguous", 0, first.repeat(1, 2)[:, ::2])
        bad(ValueError, "dims", 0, first[0])
        bad(TypeError, "int8", wi, w.float())
        bad(ValueError, "GPU", wi, w.cpu())
        bad(ValueError, "sW", si, s[:7].contiguous())
        bad(TypeError, "float32", si, s.double())
        bad(ValueError, "sW", wi, w.repeat(2, 1))
        bad(ValueError, "activation", activation="swish")
        bad(ValueError, "out must be", out=torch.zeros((4, 9), dtype=F16, device=DEV))
        bad(TypeError, "float16", out=torch.zeros((4, 8), device=DEV))
        bad(TypeError, "uint8", workspace=x)
        if "backward" in name:
            bad(TypeError, "float32", dbias=y[0])
            bad(ValueError, "grad_pre", grad_pre=h)
        else:
            bad(ValueError, "bias", bias=torch.zeros(7, dtype=F16, device=DEV))
            bad(ValueError, "pre", pre=h)
    for f in (lambda: li8.gated_linear(x, w[:7].contiguous(), s[:7].contiguous()),
              lambda: li8.gated_backward(h, y, w[:7].contiguous(), s[:7].contiguous())):
        with pytest.raises(ValueError, match="even number"):
            f()
    for f in (lambda: li8.linear_epilogue(x, w[:, :16].contiguous(), s), lambda: li8.gated_linear(x, w[:, :16].contiguous(), s),
              lambda: li8.linear_backward(h, w, s), lambda: li8.gated_backward(y, y, w, s)):
        with pytest.raises(ValueError, match="mismatch"):
            f()
    with pytest.raises(TypeError, match="pre"):
        li8.linear_backward(y, w, s, activation="silu")
    with pytest.raises(ValueError, match="residual"):
        li8.linear_epilogue(x, w, s, residual=h)
    big = torch.zeros((100, 32), dtype=F16, device=DEV)
    with pytest.raises(li8.Int8MatmulError, match="WORKSPACE"):
        li8.linear_epilogue(big, w, s, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(li8.Int8MatmulError, match="SHAPE"):
        li8.linear_epilogue(big[:, :24].contiguous(), w[:, :24].contiguous(), s)


@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("T, K, N", [(5, 256, 66), (6, 8224, 34), (50, 256, 66)])
def test_nans_reach_the_outputs_that_they_enter(act, T, K, N):
    print(f"case nan {act} {T}x{K}x{N}", flush=True)
    f, F = Forward(T, K, N, seed=11, residual=True), N // 2
    x, w, s, b, r = (f.d[k] for k in ("X", "Wq", "sW", "bias", "residual"))
    clean_y = host(li8.linear_epilogue(x, w, s, bias=b, activation=act, residual=r))
    clean_h = host(li8.gated_linear(x, w, s, bias=b, activation=act))
    nb, nr = b.clone(), r.clone()
    nb[3] = nb[F + 7] = nr[1, 9] = float("nan")
    y = host(li8.linear_epilogue(x, w, s, bias=nb, activation=act, residual=nr))
    h = host(li8.gated_linear(x, w, s, bias=nb, activation=act))
    ny, nh = np.zeros_like(y, bool), np.zeros_like(h, bool)
    ny[:, [3, F + 7]] = ny[1, 9] = nh[:, [3, 7]] = True
    assert np.array_equal(np.isnan(y), ny) and np.array_equal(np.isnan(h), nh)
    assert np.array_equal(y[~ny], clean_y[~ny]) and np.array_equal(h[~nh], clean_h[~nh])


def test_a_linear_gate_passes_an_overflowed_pre():
    """act none: the slope is 1 at an infinity of the stored pre too, and the gradients are infinities where they are products with it."""
    for T in (9, 70):
        b = Backward(T, 64, 80, True, seed=12)
        b.pre[2, 5] = -np.inf                               # the gate's value of feature 5
        g = host(b.run("none")["grad_pre"])
        want = ffn.grad_pre(b.dY, b.pre, "none", True)[0]
        assert g[2, 5] == np.float16(want[2, 5]) and np.isinf(g[2, 45]) and np.isfinite(np.delete(g[2], 45)).all()


BIG = (66000, 16, 33000)   # more than 2^31 elements of [T, N]


def _big(shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, dtype=F16, device=DEV).normal_(generator=g)


def _rows(t, rows):
    return host(t[rows])


@pytest.mark.parametrize("gated", [False, True])
def test_forward_past_32_bit_offsets(gated):
    T, K, N = BIG
    print(f"case big forward {gated}", flush=True)
    rng = np.random.default_rng(21)
    Wq, sW = rng.integers(-127, 128, (N, K)).astype(np.int8), (rng.random(N) * 1e-3 + 1e-4).astype(np.float32)
    x, bias, rows = _big((T, K), 1), (rng.standard_normal(N)).astype(np.float16), [0, 1, 32541, T - 2, T - 1]
    pre = torch.empty((T, N), dtype=F16, device=DEV)
    kw = dict(threshold=float("inf"), bias=dev(bias), activation="silu", pre=pre)
    if gated:
        out = li8.gated_linear(x, dev(Wq), dev(sW), **kw)
        want = ffn.gated_linear(_rows(x, rows), Wq, sW, float("inf"), bias, "silu")
    else:
        out = _big((T, N), 2)
        res = _rows(out, rows)
        li8.linear_epilogue(x, dev(Wq), dev(sW), residual=out, out=out, **kw)
        want = ffn.linear_epilogue(_rows(x, rows), Wq, sW, float("inf"), bias, "silu", res)
    for t, w, k in ((out, want[0], "out"), (pre, want[1], "pre")):
        assert ffn.check(_rows(t, rows), w, k) is None, ffn.check(_rows(t, rows), w, k)


@pytest.mark.parametrize("gated", [False, True])
def test_backward_past_32_bit_offsets(gated):
    T, K, N = BIG
    print(f"case big backward {gated}", flush=True)
    rng = np.random.default_rng(22)
    F, rows = N // 2 if gated else N, [0, 1, 32541, T - 2, T - 1]
    Wq, sW = rng.integers(-127, 128, (N, K)).astype(np.int8), (rng.random(N) * 1e-3 + 1e-4).astype(np.float32)
    dY, pre = _big((T, F), 3), _big((T, N), 4)
    g, db = torch.empty((T, N), dtype=F16, device=DEV), torch.empty(N, device=DEV)
    if gated:
        dX = li8.gated_backward(dY, pre, dev(Wq), dev(sW), grad_pre=g, dbias=db)
    else:
        dX = li8.linear_backward(dY, dev(Wq), dev(sW), pre=pre, activation="silu", grad_pre=g, dbias=db)
    want = ffn.backward(_rows(dY, rows), _rows(pre, rows), Wq, sW, "silu", gated)
    for t, k in ((dX, "dX"), (g, "grad_pre")):
        assert ffn.check(_rows(t, rows), want[k], k) is None, ffn.check(_rows(t, rows), want[k], k)
    # the sums of some features over all rows
    for f in (0, F - 1):
        cols = [f, F + f] if gated else [f]
        z, ez = ffn.grad_pre(host(dY[:, f:f + 1]), host(pre[:, cols]), "silu", gated)
        w = (z.sum(0), ez.sum(0) + (T + 2) * ffn.U * (np.abs(z) + ez).sum(0))
        assert ffn.check(host(db[cols]), w, "dbias") is None, ffn.check(host(db[cols]), w, "dbias")


# few tiles and a long K, whose int32 sums come from several workgroups; T, K, N
RANGED = [(17, 4096, 8), (64, 4096, 258), (33, 8208, 100), (100, 11008, 74), (200, 6272, 386), (250, 16400, 66), (65, 2064, 34)]


@pytest.mark.parametrize("T, K, N", RANGED)
@pytest.mark.parametrize("kw, threshold", [({}, 6.0), (dict(sparse=2e-3), 6.0), (dict(fixed=700), 6.0), ({}, float("inf"))])
def test_ranges_of_k(T, K, N, kw, threshold):
    print(f"case ranges {T}x{K}x{N} {kw} {threshold}", flush=True)
    f = Forward(T, K, N, seed=13, residual=True, **kw)
    act = ffn.ACTS[(T + len(kw)) % 5]
    f.epilogue(threshold, act)
    f.epilogue(threshold, act, save=False, in_place=True)
    f.gated(threshold, act)
    x, w, s = f.d["X"], f.d["Wq"], f.d["sW"]
    Y = li8.linear(x, w, s, threshold).view(torch.int16)
    pre = torch.empty((T, N), dtype=F16, device=DEV)
    assert torch.equal(li8.linear_epilogue(x, w, s, threshold).view(torch.int16), Y)
    li8.gated_linear(x, w, s, threshold, pre=pre)
    assert torch.equal(pre.view(torch.int16), Y)


@pytest.mark.parametrize("T, K, N", [(17, 4096, 8), (64, 4096, 130), (100, 6160, 74)])
def test_ranges_of_k_with_every_column_an_outlier(T, K, N):
    """The gathered columns then fill the place where the ranges' sums lie."""
    print(f"case ranges all {T}x{K}x{N}", flush=True)
    f = Forward(T, K, N, seed=14)
    f.X[f.X == 0] = 1.0
    f.d["X"] = dev(f.X)
    f.epilogue(0.0, "silu")
    f.gated(0.0, "silu")
    x, w, s = f.d["X"], f.d["Wq"], f.d["sW"]
    assert torch.equal(li8.linear_epilogue(x, w, s, 0.0).view(torch.int16), li8.linear(x, w, s, 0.0).view(torch.int16))


@pytest.mark.parametrize("T, K, N", [(1024, 272, 2178), (700, 528, 4100), (64, 272, 12546), (100, 272, 16382), (64, 528, 8194)])
@pytest.mark.parametrize("fixed", [3, 70, 150, 260])
def test_small_tiles_in_rounds_and_with_many_outlier_columns(T, K, N, fixed):
    print(f"case small tiles {T}x{K}x{N} {fixed}", flush=True)
    f = Forward(T, K, N, seed=15, fixed=fixed)
    x, w, s = f.d["X"], f.d["Wq"], f.d["sW"]
    Y = li8.linear(x, w, s).view(torch.int16)
    pre = torch.empty((T, N), dtype=F16, device=DEV)
    assert torch.equal(li8.linear_epilogue(x, w, s).view(torch.int16), Y)
    li8.gated_linear(x, w, s, pre=pre)
    assert torch.equal(pre.view(torch.int16), Y)
    if fixed == 150 and T <= 100:
        f.epilogue(activation="silu")
        f.gated(activation="gelu")
