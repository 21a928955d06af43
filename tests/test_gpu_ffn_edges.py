"""GPU tests of the feed-forward operators at the ends of their ranges: infinities
and sums past fp16 in the activations."""
import numpy as np
import pytest
import torch

import int8_matmul_amd as li8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16 = torch.float16
INF = float("inf")
SMOOTH = ("silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu tests must run on an MI355X")
    li8.load_library()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


# few tokens, few tokens split over K, tiles, ranges of K
SHAPES = [(5, 256, 66), (6, 8224, 34), (50, 256, 66), (50, 8224, 66)]


@pytest.mark.parametrize("act", ("relu",) + SMOOTH)
@pytest.mark.parametrize("T, K, N", SHAPES)
def test_an_infinite_bias_gives_an_infinity(act, T, K, N):
    """act(+inf) = +inf for each of them, and the gate of a pair alike."""
    print(f"case inf {act} {T}x{K}x{N}", flush=True)
    g, F = torch.Generator(device=DEV).manual_seed(1), N // 2
    x = torch.randn((T, K), generator=g, device=DEV).half()
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    s = torch.full((N,), 1e-4, device=DEV)
    b = torch.randn(N, generator=g, device=DEV).half()
    clean_y = host(li8.linear_epilogue(x, w, s, bias=b, activation=act))
    clean_h = host(li8.gated_linear(x, w, s, bias=b, activation=act))
    b[3] = INF
    y = host(li8.linear_epilogue(x, w, s, bias=b, activation=act))
    pre = torch.empty((T, N), dtype=F16, device=DEV)
    h = host(li8.gated_linear(x, w, s, bias=b, activation=act, pre=pre))
    up = host(pre)[:, F + 3].astype(np.float64)
    assert (y[:, 3] == INF).all()
    assert (h[up > 0, 3] == INF).all() and (h[up < 0, 3] == -INF).all() and (up != 0).any()
    rest = np.arange(N) != 3
    assert np.array_equal(y[:, rest], clean_y[:, rest]) and np.array_equal(h[:, rest[:F]], clean_h[:, rest[:F]])


@pytest.mark.parametrize("act", ("relu",) + SMOOTH)
@pytest.mark.parametrize("T, K, N", SHAPES)
def test_sums_whose_squares_leave_fp32(act, T, K, N):
    """Z of 10^18 to 10^34 by its scales: an infinity of fp16 above, and zero below."""
    print(f"case large {act} {T}x{K}x{N}", flush=True)
    x = torch.ones((T, K), dtype=F16, device=DEV)
    sign = 1 - 2 * (torch.arange(N, device=DEV) % 2)
    w = (127 * sign[:, None].expand(N, K)).to(torch.int8).contiguous()
    s = 10.0 ** torch.linspace(14, 28, N, device=DEV)   # Z = +-127 K s
    y = host(li8.linear_epilogue(x, w, s, activation=act))
    assert (y[:, ::2] == INF).all() and (y[:, 1::2] == 0).all()


@pytest.mark.parametrize("act", ("relu",) + SMOOTH)
@pytest.mark.parametrize("T", [9, 70])
def test_an_overflowed_pre_has_the_slope_of_its_side(act, T):
    """Slope 1 at +inf and 0 at -inf, as at +-60000: the same gradients, bit for bit."""
    print(f"case slope at infinity {act} {T}", flush=True)
    g, K, N = torch.Generator(device=DEV).manual_seed(2), 272, 600
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    s = torch.rand(N, generator=g, device=DEV) * 1e-3 + 1e-4
    dY = torch.randn((T, N), generator=g, device=DEV).half()
    pre = torch.randn((T, N), generator=g, device=DEV).half()
    hit = torch.rand((T, N), generator=g, device=DEV) < 0.02
    got = []
    for top in (60000.0, INF):
        z = torch.where(hit, top * torch.sign(pre), pre)
        dz, db = torch.empty_like(dY), torch.empty(N, device=DEV)
        dX = li8.linear_backward(dY, w, s, pre=z, activation=act, grad_pre=dz, dbias=db)
        got.append([host(t) for t in (dX, dz, db)])
    assert int(hit.sum()) > 0 and np.isfinite(got[0][0]).all()
    for a, b in zip(*got):
        assert np.array_equal(a, b)
