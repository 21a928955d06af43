"""The feed-forward operators of the int8 linear layer as they are measured: the product with bias, activation and residual
in its epilogue, the gated pair of projections, and the gradients that pass back through both.

A weight is int8 codes [N, K] with one fp32 scale for each row, value = code * scale; it is frozen.  A gated weight is
[2 F, K], the gate's F rows first.  A forward call splits the columns of X with some |x| > threshold off; the others are
coded for each token (scale = absmax / 127, round half to even).

Case keys: kind ("epilogue", "gated", "linear_backward", "gated_backward"), T (tokens), K (input features), N (output
features; F of a gated pair), act, bias, residual, save (the forward call keeps what the backward call needs), outliers
(fixed outlier columns of X), sparse (rate of further outliers).
"""
import math

import numpy as np
import torch

own = False

THRESHOLD = 6.0
GATED = ("gated", "gated_backward")


def _case(name, kind, T, K, N, act="none", bias=False, residual=False, save=False, outliers=0, sparse=0.0):
    return dict(name=name, kind=kind, T=T, K=K, N=N, act=act, bias=bias, residual=residual, save=save, outliers=outliers,
                sparse=sparse)


def listed():
    return [
        # one user's token through a small projection with bias and activation: the call's latency
        _case("epilogue_single", "epilogue", 1, 4096, 4096, "gelu", bias=True, outliers=4),
        # a generation step of eight sequences: the 7B down-projection added to the residual stream
        _case("epilogue_down_decode_7b", "epilogue", 8, 11008, 4096, residual=True, outliers=4),
        # a chunk of a prompt through a 13B up-projection with bias, outliers on random columns too
        _case("epilogue_up_13b", "epilogue", 512, 5120, 13824, "gelu_tanh", bias=True, outliers=8, sparse=1e-4),
        # a 7B prompt's down-projection added to the residual stream
        _case("epilogue_down_prefill_7b", "epilogue", 4096, 11008, 4096, residual=True, outliers=6),
        # a generation step of eight sequences: gate and up of a 7B layer
        _case("gated_decode_7b", "gated", 8, 4096, 11008, "silu", outliers=4),
        # sixteen sequences of a 13B layer
        _case("gated_decode_13b", "gated", 16, 5120, 13824, "silu", outliers=8),
        # a ragged prompt of a small layer with odd widths and biases, kept for the backward pass
        _case("gated_ragged", "gated", 777, 1040, 2731, "gelu", bias=True, save=True, outliers=3, sparse=1e-4),
        # a 7B training batch's forward pass, kept for the backward pass
        _case("gated_train_7b", "gated", 4096, 4096, 11008, "silu", save=True, outliers=6),
        # a short sequence back through a projection with bias and activation
        _case("linear_backward_short", "linear_backward", 37, 4096, 4096, "gelu", bias=True),
        # a 7B training batch back through the down-projection
        _case("linear_backward_down_7b", "linear_backward", 4096, 11008, 4096),
        # a chunk of a 13B training batch back through gate and up
        _case("gated_backward_13b", "gated_backward", 512, 5120, 13824, "silu"),
        # a 7B training batch back through gate and up, the gradients of both kept for adapters
        _case("gated_backward_7b", "gated_backward", 4096, 4096, 11008, "silu", save=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["epilogue", "gated", "linear_backward", "gated_backward"])
    K = 16 * _log(rng, 4, 864)
    N = rng.choice([_log(rng, 33, 13824), 8 * _log(rng, 16, 1728)])
    # no more than the largest listed case
    T = min(_log(rng, 1, 4096) if rng.random() < 0.75 else rng.randint(1, 16), 4096 * 4096 * 11008 // (K * N))
    act = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"] + ([] if kind in GATED else ["none", "none"]))
    forward = kind in ("epilogue", "gated")
    save = rng.random() < 0.4 and act != "none"
    return dict(kind=kind, T=T, K=K, N=N, act=act, bias=rng.random() < 0.4, residual=kind == "epilogue" and rng.random() < 0.5,
                save=save, outliers=rng.choice([0, 1, 4, 8, 40]) if forward else 0,
                sparse=rng.choice([0.0, 0.0, 1e-4]) if forward else 0.0)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    T, K, gated = c["T"], c["K"], c["kind"] in GATED
    rows = 2 * c["N"] if gated else c["N"]
    half = torch.float16

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # rows of unlike sizes, as a trained projection has
    W = randn(rows, K) * (0.02 * torch.exp(0.3 * randn(rows, 1)))
    sW = W.abs().amax(dim=1) / 127
    Wq = torch.round(W / sW[:, None]).clamp(-127, 127).to(torch.int8)
    del W
    st = dict(case=c, Wq=Wq, sW=sW)
    if c["kind"] in ("epilogue", "gated"):
        X = randn(T, K)
        if c["outliers"]:
            cols = torch.randperm(K, generator=g, device=dev)[:c["outliers"]]
            u = torch.rand((T, c["outliers"]), generator=g, device=dev) * 80 + 20
            X[:, cols] = u * torch.sign(randn(T, c["outliers"]))
        if c["sparse"]:
            hit = torch.rand((T, K), generator=g, device=dev) < c["sparse"]
            X = torch.where(hit, torch.sign(X) * (7 + 23 * torch.rand((T, K), generator=g, device=dev)), X)
        st["X"] = X.to(half)
        st["bias"] = (randn(rows) * 0.5).to(half) if c["bias"] else None
        st["residual"] = (randn(T, c["N"]) * 3).to(half) if c["residual"] else None
        if own:
            # a serving program keeps the workspace, a training program too
            import int8_matmul_amd as li8
            st["workspace"] = torch.empty(li8.linear_workspace_bytes(T, K, rows), dtype=torch.uint8, device=dev)
    else:
        # gradients of unlike size from token to token, as a loss over some of them gives
        st["dY"] = (randn(T, c["N"]) * (1e-2 * torch.exp(randn(T, 1)))).to(half)
        st["pre"] = (randn(T, rows) * 1.5).to(half) if gated or c["act"] != "none" else None
        if own:
            import int8_matmul_amd as li8
            st["workspace"] = li8.new_backward_workspace(T, K, rows, dev)
    return st


def run(st):
    c = st["case"]
    if own:
        import int8_matmul_amd as li8
        T, N, dev = c["T"], c["N"], st["Wq"].device
        rows = st["Wq"].shape[0]
        ws = st["workspace"]
        saved = torch.empty((T, rows), dtype=torch.float16, device=dev) if c["save"] else None
        if c["kind"] == "epilogue":
            Y = li8.linear_epilogue(st["X"], st["Wq"], st["sW"], THRESHOLD, bias=st["bias"], activation=c["act"],
                                    residual=st["residual"], pre=saved, workspace=ws)
            return {"Y": Y, "pre": saved} if c["save"] else {"Y": Y}
        if c["kind"] == "gated":
            H = li8.gated_linear(st["X"], st["Wq"], st["sW"], THRESHOLD, bias=st["bias"], activation=c["act"], pre=saved,
                                 workspace=ws)
            return {"H": H, "pre": saved} if c["save"] else {"H": H}
        dbias = torch.empty((rows,), dtype=torch.float32, device=dev) if c["bias"] else None
        if c["kind"] == "linear_backward":
            dX = li8.linear_backward(st["dY"], st["Wq"], st["sW"], pre=st["pre"], activation=c["act"], grad_pre=saved,
                                     dbias=dbias, workspace=ws)
        else:
            dX = li8.gated_backward(st["dY"], st["pre"], st["Wq"], st["sW"], activation=c["act"], grad_pre=saved,
                                    dbias=dbias, workspace=ws)
        out = {"dX": dX}
        if c["save"]:
            out["grad_pre"] = saved
        if c["bias"]:
            out["dbias"] = dbias
        return out
    if c["kind"] in ("epilogue", "gated"):
        return _forward(st)
    return _backward(st)


# ---- the plain forms ----

def _act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-k * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * (k * (1 + 3 * 0.044715 * z * z))
    return torch.ones_like(z)


def _forward(st):
    c = st["case"]
    X = st["X"].float()
    out = (X.abs() > THRESHOLD).any(dim=0)
    small = X.masked_fill(out, 0.0)
    # the quotients in 64 bits and rounded once to 32: the codes are whole numbers next to a border
    scale = (small.abs().amax(dim=1, keepdim=True).double() / 127).float()
    codes = torch.round((small.double() / torch.where(scale > 0, scale, 1.0).double()).float())
    A = torch.where(out, X, codes * scale)
    z = torch.matmul(A, st["Wq"].float().t().contiguous()) * st["sW"]
    if st["bias"] is not None:
        z = z + st["bias"].float()
    res = {}
    if c["kind"] == "gated":
        F = c["N"]
        res["H"] = (_act(z[:, :F], c["act"]) * z[:, F:]).half()
    else:
        y = _act(z, c["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        res["Y"] = y.half()
    if c["save"]:
        res["pre"] = z.half()
    return res


def _backward(st):
    c = st["case"]
    d = st["dY"].float()
    if c["kind"] == "gated_backward":
        z = st["pre"].float()
        g, u = z[:, :c["N"]], z[:, c["N"]:]
        d = torch.cat([d * u * _slope(g, c["act"]), d * _act(g, c["act"])], dim=1)
    elif c["act"] != "none":
        d = d * _slope(st["pre"].float(), c["act"])
    res = {"dX": torch.matmul(d * st["sW"], st["Wq"].float()).half()}
    if c["save"]:
        res["grad_pre"] = d.half()
    if c["bias"]:
        res["dbias"] = d.double().sum(dim=0).float()
    return res


# ---- how much work ----

def work(case):
    c = case
    T, K, N = c["T"], c["K"], c["N"]
    gated = c["kind"] in GATED
    rows = 2 * N if gated else N
    b = rows * K + 4 * rows + 2 * T * K + 2 * T * N
    if c["kind"] in ("epilogue", "gated"):
        b += 2 * rows * c["bias"] + 2 * T * N * c["residual"]
    else:
        b += (2 * T * rows if gated or c["act"] != "none" else 0) + 4 * rows * c["bias"]
    b += 2 * T * rows * c["save"]
    return {"bytes": b, "flops": 2 * T * K * rows}


# ---- the same from the definitions, in 64 bits ----

def exact(case, seed):
    c = case
    st = prepare(case, seed)
    f64 = torch.float64
    W = st["Wq"].to(f64) * st["sW"].to(f64)[:, None]
    N, kind = c["N"], c["kind"]

    def phi(z):                     # the normal distribution's integral
        return torch.special.ndtr(z)

    def act(z):
        if c["act"] == "relu":
            return torch.relu(z)
        if c["act"] == "silu":
            return z * torch.sigmoid(z)
        if c["act"] == "gelu":
            return z * phi(z)
        if c["act"] == "gelu_tanh":
            return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        return z

    if kind in ("epilogue", "gated"):
        X = st["X"]
        hot = torch.nonzero((X.abs() > THRESHOLD).sum(dim=0) > 0).flatten()
        cold = torch.nonzero((X.abs() > THRESHOLD).sum(dim=0) == 0).flatten()
        rest = X[:, cold].cpu().numpy().astype("float32")
        # the scale and the quotient are defined as rounded to 32 bits, the code as the nearest whole number, ties to even
        s = (np.abs(rest).max(axis=1, initial=0).astype("float32") / np.float32(127)).astype("float32")
        q = np.rint(rest / np.where(s > 0, s, np.float32(1))[:, None])
        dev = X.device
        q, s = torch.from_numpy(q).to(dev).to(f64), torch.from_numpy(s).to(dev).to(f64)
        z = torch.matmul(q, W[:, cold].t().contiguous()) * s[:, None]
        if len(hot):
            z = z + torch.matmul(X[:, hot].to(f64), W[:, hot].t().contiguous())
        if st["bias"] is not None:
            z = z + st["bias"].to(f64)
        if kind == "gated":
            res = {"H": act(z[:, :N]) * z[:, N:]}
        else:
            res = {"Y": act(z)}
            if st["residual"] is not None:
                res["Y"] = res["Y"] + st["residual"].to(f64)
        if c["save"]:
            res["pre"] = z
        return res

    # the slopes by differentiating each activation's own definition
    def pulled(z, out_grad, value):
        z = z.detach().requires_grad_(True)
        return torch.autograd.grad(value(z), z, out_grad)[0]

    d = st["dY"].to(f64)
    if kind == "gated_backward":
        z = st["pre"].to(f64)
        d = pulled(z, d, lambda v: act(v[:, :N]) * v[:, N:])
    elif c["act"] != "none":
        d = pulled(st["pre"].to(f64), d, act)
    res = {"dX": torch.matmul(d, W)}
    if c["save"]:
        res["grad_pre"] = d
    if c["bias"]:
        res["dbias"] = d.sum(dim=0)
    return res
