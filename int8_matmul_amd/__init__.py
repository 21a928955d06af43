"""LLM.int8() mixed-precision linear layer for AMD Instinct MI355X (gfx950).

A thin ctypes binding of ``libllm_int8.so`` (HIP kernels + C ABI, declared
in ``include/llm_int8.h``).  This module only marshals arguments: every step
of the computation runs in the library's kernels.  PyTorch provides the
device memory and the stream; calls are enqueued on torch's current stream
of the tensors' device and never synchronize.

    Wq, sW = quantize_weight(W)            # once per weight, W fp16 [N,K]
    Y = linear(X, Wq, sW, threshold=6.0)   # X fp16 [T,K] -> Y fp16 [T,N]

The method (hncyxsy.com/news/230290 "LLM quantization, part 2", section
2.1; lowentro.cn "model quantization" notes, Q4; tqpw.cn/news/5683,
sections 2.1 and 3.1): feature columns of X with some |x| > threshold are
outliers and are multiplied in floating point; the other columns are
quantized to int8 with a per-token absmax scale (the weight with a
per-output-feature scale), multiplied as int8 x int8 -> int32, dequantized,
and added to the outlier product; the result is fp16.

If the library has not been built, every call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import operator
import os

import torch

__all__ = [
    "Int8MatmulError", "LibraryNotBuilt", "library_path", "load_library",
    "quantize_weight", "workspace_bytes", "linear_workspace_bytes", "plan", "new_workspace",
    "linear", "linear_noalloc", "NOALLOC_SCRATCH_BYTES", "prepare",
    "gemm", "export_stages", "stages", "few_token_path", "linear_fp16w", "prepare_fp16w",
    "gemm_fp16w", "smoothquant_column_absmax", "smoothquant_factors",
    "smoothquant_quantize_weight", "smoothquant_prepare", "smoothquant_linear",
    "cache_bytes", "new_cache", "cache_reset", "cache_stats", "linear_cached", "prepare_cached",
    "gemm_cached", "STATUS",
    "KVCache", "KVBatch", "Rope", "new_kv_cache", "kv_append", "kv_read", "kv_attention",
    "kv_attention_plan", "kv_attention_workspace_bytes", "new_kv_attention_workspace",
    "linear_epilogue", "gated_linear", "linear_backward", "gated_backward",
    "backward_workspace_bytes", "new_backward_workspace", "ACTIVATIONS", "epilogue_plan", "backward_plan",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libllm_int8.so")
_lib = None

STATUS = {
    0: "LI8_OK",
    1: "LI8_ERR_INVALID_ARG",
    2: "LI8_ERR_SHAPE",
    3: "LI8_ERR_ALIGN",
    4: "LI8_ERR_WORKSPACE",
    5: "LI8_ERR_HIP",
    6: "LI8_ERR_SCRATCH",
}


class Int8MatmulError(RuntimeError):
    """A library call returned a status other than LI8_OK."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")


class LibraryNotBuilt(ImportError):
    pass


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libllm_int8.so (raises LibraryNotBuilt if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise LibraryNotBuilt(
            f"{_LIB_PATH} is missing; build it with `python -m int8_matmul_amd.build`")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    L.li8_status_str.restype = ctypes.c_char_p
    L.li8_status_str.argtypes = [ctypes.c_int]
    L.int8_quantize_weight.restype = ctypes.c_int
    L.int8_quantize_weight.argtypes = [vp, i64, i64, vp, vp, vp]
    L.llm_int8_workspace_bytes.restype = sz
    L.llm_int8_workspace_bytes.argtypes = [i64, i64, i64]
    L.llm_int8_linear_workspace_bytes.restype = sz
    L.llm_int8_linear_workspace_bytes.argtypes = [i64, i64, i64]
    L.llm_int8_plan.restype = ctypes.c_int
    L.llm_int8_plan.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp]
    L.llm_int8_linear.restype = ctypes.c_int
    L.llm_int8_linear.argtypes = [vp, vp, vp, ctypes.c_float, i64, i64, i64, vp, vp, sz, vp]
    L.llm_int8_linear_noalloc.restype = ctypes.c_int
    L.llm_int8_linear_noalloc.argtypes = [vp, vp, vp, ctypes.c_float, i64, i64, i64, vp, vp]
    L.llm_int8_prepare.restype = ctypes.c_int
    L.llm_int8_prepare.argtypes = [vp, vp, ctypes.c_float, i64, i64, i64, vp, sz, vp]
    L.llm_int8_gemm.restype = ctypes.c_int
    L.llm_int8_gemm.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, sz, vp]
    L.llm_int8_linear_fp16w.restype = ctypes.c_int
    L.llm_int8_linear_fp16w.argtypes = [vp, vp, vp, vp, ctypes.c_float, i64, i64, i64, vp, vp,
                                        sz, vp]
    L.llm_int8_prepare_fp16w.restype = ctypes.c_int
    L.llm_int8_prepare_fp16w.argtypes = [vp, vp, ctypes.c_float, i64, i64, i64, vp, sz, vp]
    L.llm_int8_gemm_fp16w.restype = ctypes.c_int
    L.llm_int8_gemm_fp16w.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp, sz, vp]
    L.smoothquant_column_absmax.restype = ctypes.c_int
    L.smoothquant_column_absmax.argtypes = [vp, i64, i64, vp, vp]
    L.smoothquant_factors.restype = ctypes.c_int
    L.smoothquant_factors.argtypes = [vp, vp, ctypes.c_double, i64, vp, vp, vp]
    L.smoothquant_quantize_weight.restype = ctypes.c_int
    L.smoothquant_quantize_weight.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    L.smoothquant_prepare.restype = ctypes.c_int
    L.smoothquant_prepare.argtypes = [vp, vp, i64, i64, i64, vp, sz, vp]
    L.smoothquant_linear.restype = ctypes.c_int
    L.smoothquant_linear.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp, sz, vp]
    L.llm_int8_cache_bytes.restype = sz
    L.llm_int8_cache_bytes.argtypes = [i64, i64]
    L.llm_int8_cache_reset.restype = ctypes.c_int
    L.llm_int8_cache_reset.argtypes = [vp, sz, i64, i64, vp]
    L.llm_int8_linear_cached.restype = ctypes.c_int
    L.llm_int8_linear_cached.argtypes = [vp, vp, vp, ctypes.c_float, i64, i64, i64, vp, vp, sz,
                                         vp, sz, vp]
    L.llm_int8_prepare_cached.restype = ctypes.c_int
    L.llm_int8_prepare_cached.argtypes = [vp, vp, ctypes.c_float, i64, i64, i64, vp, sz, vp, sz,
                                          vp]
    L.llm_int8_gemm_cached.restype = ctypes.c_int
    L.llm_int8_gemm_cached.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, sz, vp, sz, vp]
    L.llm_int8_export_stages.restype = ctypes.c_int
    L.llm_int8_export_stages.argtypes = [vp, sz, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp]
    L.llm_int8_stages.restype = ctypes.c_int
    L.llm_int8_stages.argtypes = [vp, vp, vp, ctypes.c_float, i64, i64, i64, vp, vp, sz, vp, vp, vp,
                                  vp, vp, vp, vp, vp]
    i32 = ctypes.c_int32
    L.int8_kv_append.restype = ctypes.c_int
    L.int8_kv_append.argtypes = [vp, i64, vp, i64, ctypes.c_int, vp, vp, vp, vp]
    L.int8_kv_read.restype = ctypes.c_int
    L.int8_kv_read.argtypes = [vp, vp, ctypes.c_int, vp, i64, vp, i64, vp]
    L.int8_kv_attention_workspace_bytes.restype = sz
    L.int8_kv_attention_workspace_bytes.argtypes = [vp, vp, i32]
    L.int8_kv_attention_plan.restype = ctypes.c_int
    L.int8_kv_attention_plan.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    L.int8_kv_attention.restype = ctypes.c_int
    L.int8_kv_attention.argtypes = [vp, i64, ctypes.c_int, i32, ctypes.c_float, vp, i32, i32, vp, vp,
                                    vp, i64, vp, vp, sz, vp]
    L.llm_int8_linear_epilogue.restype = ctypes.c_int
    L.llm_int8_linear_epilogue.argtypes = [vp, vp, vp, ctypes.c_float, i64, i64, i64, vp, i32, vp, vp, vp, vp,
                                           sz, vp]
    L.llm_int8_gated_linear.restype = ctypes.c_int
    L.llm_int8_gated_linear.argtypes = [vp, vp, vp, ctypes.c_float, i64, i64, i64, vp, i32, vp, vp, vp, sz, vp]
    L.llm_int8_backward_workspace_bytes.restype = sz
    L.llm_int8_backward_workspace_bytes.argtypes = [i64, i64, i64]
    L.llm_int8_linear_backward.restype = ctypes.c_int
    L.llm_int8_linear_backward.argtypes = [vp, vp, i32, vp, vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    for plan in ("llm_int8_epilogue_plan", "llm_int8_backward_plan"):
        getattr(L, plan).restype = ctypes.c_int
        getattr(L, plan).argtypes = [i64, i64, i64, i32, vp]
    L.llm_int8_gated_backward.restype = ctypes.c_int
    L.llm_int8_gated_backward.argtypes = [vp, vp, i32, vp, vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    _lib = L
    return L


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise Int8MatmulError(fn, status)


def _stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _require(t: torch.Tensor, dtype: torch.dtype, name: str, ndim: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def quantize_weight(W: torch.Tensor, Wq: torch.Tensor | None = None,
                    sW: torch.Tensor | None = None):
    """Vector-wise int8 quantization of W fp16 [N,K]: (Wq int8 [N,K], sW fp32 [N])."""
    L = load_library()
    _require(W, torch.float16, "W", 2)
    N, K = W.shape
    if Wq is None:
        Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    if sW is None:
        sW = torch.empty((N,), dtype=torch.float32, device=W.device)
    _check("int8_quantize_weight",
           L.int8_quantize_weight(_ptr(W), N, K, _ptr(Wq), _ptr(sW), _stream(W.device)))
    return Wq, sW


def workspace_bytes(T: int, K: int, N: int) -> int:
    n = load_library().llm_int8_workspace_bytes(T, K, N)
    if n == 0:
        raise Int8MatmulError("llm_int8_workspace_bytes", 2)
    return int(n)


def new_workspace(T: int, K: int, N: int, device) -> torch.Tensor:
    return torch.empty(workspace_bytes(T, K, N), dtype=torch.uint8, device=device)


def linear_workspace_bytes(T: int, K: int, N: int) -> int:
    """Bytes llm_int8_linear needs for this shape (0 on the few-token path)."""
    return int(load_library().llm_int8_linear_workspace_bytes(T, K, N))


PATHS = {0: "empty", 1: "few_tokens", 2: "tiled", 3: "few_tokens_split"}


def plan(T: int, K: int, N: int) -> dict:
    """Which kernels a call of this shape runs: path, output tile, and the
    outlier counts (fold_lo, fold_hi] for which the tiled GEMM copies the
    weight's outlier columns itself instead of the prepare kernel."""
    out = [ctypes.c_int32() for _ in range(5)]
    _check("llm_int8_plan", load_library().llm_int8_plan(T, K, N, *(ctypes.byref(o) for o in out)))
    path, tm, tn, lo, hi = (o.value for o in out)
    return dict(path=PATHS[path], tile_m=tm, tile_n=tn, fold_lo=lo, fold_hi=hi)


def few_token_path(T: int, K: int) -> bool:
    """True if ``linear`` runs on a few-token path (fused or split) for T x K."""
    return plan(T, K, 1)["path"] in ("few_tokens", "few_tokens_split")


def _ws(workspace, T, K, N, device):
    if workspace is None:
        workspace = new_workspace(T, K, N, device)
    _require(workspace, torch.uint8, "workspace", 1)
    return workspace


def linear(X: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, threshold: float = 6.0,
           out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Y fp16 [T,N] = the LLM.int8() decomposed product of X fp16 [T,K] and W."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    T, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or sW.shape[0] != N:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Wq {tuple(Wq.shape)}, sW {tuple(sW.shape)}")
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=X.device)
    _require(out, torch.float16, "out", 2)
    if workspace is None and linear_workspace_bytes(T, K, N) == 0:
        ws = torch.empty(0, dtype=torch.uint8, device=X.device)   # the fused path uses none
    else:
        ws = _ws(workspace, T, K, N, X.device)
    _check("llm_int8_linear",
           L.llm_int8_linear(_ptr(X), _ptr(Wq), _ptr(sW), float(threshold), T, K, N,
                             _ptr(out), _ptr(ws), ws.numel(), _stream(X.device)))
    return out


# Bytes of the fixed per-GPU array llm_int8_linear_noalloc works in.
NOALLOC_SCRATCH_BYTES = 128 * 1024 * 1024


def linear_noalloc(X: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, threshold: float = 6.0,
                   out: torch.Tensor | None = None):
    """As ``linear``, with the library's fixed per-GPU scratch array as the
    workspace (llm_int8_linear_noalloc): the library allocates nothing.
    Pass ``out`` to allocate nothing here either."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    T, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or sW.shape[0] != N:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Wq {tuple(Wq.shape)}, sW {tuple(sW.shape)}")
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=X.device)
    _require(out, torch.float16, "out", 2)
    _check("llm_int8_linear_noalloc",
           L.llm_int8_linear_noalloc(_ptr(X), _ptr(Wq), _ptr(sW), float(threshold), T, K, N,
                                     _ptr(out), _stream(X.device)))
    return out


def prepare(X: torch.Tensor, Wq: torch.Tensor, threshold: float, workspace: torch.Tensor):
    """Detection, token quantization and outlier gathers into `workspace`."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(Wq, torch.int8, "Wq", 2)
    T, K = X.shape
    N = Wq.shape[0]
    ws = _ws(workspace, T, K, N, X.device)
    _check("llm_int8_prepare",
           L.llm_int8_prepare(_ptr(X), _ptr(Wq), float(threshold), T, K, N, _ptr(ws),
                              ws.numel(), _stream(X.device)))
    return ws


def gemm(Wq: torch.Tensor, sW: torch.Tensor, T: int, workspace: torch.Tensor,
         out: torch.Tensor | None = None, acc: torch.Tensor | None = None):
    """int8 GEMM + epilogue reading what `prepare` left in `workspace`."""
    L = load_library()
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    N, K = Wq.shape
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=Wq.device)
    _require(out, torch.float16, "out", 2)
    if acc is not None:
        _require(acc, torch.int32, "acc", 2)
    _require(workspace, torch.uint8, "workspace", 1)
    _check("llm_int8_gemm",
           L.llm_int8_gemm(_ptr(Wq), _ptr(sW), T, K, N, _ptr(out), _ptr(acc), _ptr(workspace),
                           workspace.numel(), _stream(Wq.device)))
    return out


def linear_fp16w(X: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, W: torch.Tensor,
                 threshold: float = 6.0, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None):
    """The fp16-weight variant: the outlier columns multiply the fp16 weight
    W [N,K] (the one Wq, sW were quantized from) instead of Wq*sW."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    _require(W, torch.float16, "W", 2)
    T, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or sW.shape[0] != N or tuple(W.shape) != (N, K):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Wq {tuple(Wq.shape)}, "
                         f"sW {tuple(sW.shape)}, W {tuple(W.shape)}")
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=X.device)
    _require(out, torch.float16, "out", 2)
    ws = _ws(workspace, T, K, N, X.device)
    _check("llm_int8_linear_fp16w",
           L.llm_int8_linear_fp16w(_ptr(X), _ptr(Wq), _ptr(sW), _ptr(W), float(threshold), T, K,
                                   N, _ptr(out), _ptr(ws), ws.numel(), _stream(X.device)))
    return out


def prepare_fp16w(X: torch.Tensor, W: torch.Tensor, threshold: float, workspace: torch.Tensor):
    """`prepare` of the fp16-weight variant (gathers the outlier columns of W)."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(W, torch.float16, "W", 2)
    T, K = X.shape
    N = W.shape[0]
    ws = _ws(workspace, T, K, N, X.device)
    _check("llm_int8_prepare_fp16w",
           L.llm_int8_prepare_fp16w(_ptr(X), _ptr(W), float(threshold), T, K, N, _ptr(ws),
                                    ws.numel(), _stream(X.device)))
    return ws


def gemm_fp16w(Wq: torch.Tensor, sW: torch.Tensor, W: torch.Tensor, T: int,
               workspace: torch.Tensor, out: torch.Tensor | None = None,
               acc: torch.Tensor | None = None):
    """`gemm` of the fp16-weight variant, on a workspace from `prepare_fp16w`."""
    L = load_library()
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    _require(W, torch.float16, "W", 2)
    N, K = Wq.shape
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=Wq.device)
    _require(out, torch.float16, "out", 2)
    if acc is not None:
        _require(acc, torch.int32, "acc", 2)
    _require(workspace, torch.uint8, "workspace", 1)
    _check("llm_int8_gemm_fp16w",
           L.llm_int8_gemm_fp16w(_ptr(Wq), _ptr(sW), _ptr(W), T, K, N, _ptr(out), _ptr(acc),
                                 _ptr(workspace), workspace.numel(), _stream(Wq.device)))
    return out


def cache_bytes(K: int, N: int) -> int:
    n = load_library().llm_int8_cache_bytes(K, N)
    if n == 0:
        raise Int8MatmulError("llm_int8_cache_bytes", 2)
    return int(n)


def new_cache(K: int, N: int, device) -> torch.Tensor:
    """An empty outlier-column cache for a weight [N,K] (reset, ready to use)."""
    c = torch.empty(cache_bytes(K, N), dtype=torch.uint8, device=device)
    cache_reset(c, K, N)
    return c


def cache_reset(cache: torch.Tensor, K: int, N: int) -> torch.Tensor:
    """Mark the cache empty; needed after its weight changes."""
    L = load_library()
    _require(cache, torch.uint8, "cache", 1)
    _check("llm_int8_cache_reset",
           L.llm_int8_cache_reset(_ptr(cache), cache.numel(), K, N, _stream(cache.device)))
    return cache


def cache_stats(cache: torch.Tensor) -> dict:
    """valid, nO, hits, misses from the cache header (synchronizes)."""
    h = cache[:16].view(torch.int32).cpu().tolist()
    return dict(valid=h[0], nO=h[1], hits=h[2], misses=h[3])


def linear_cached(X: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, cache: torch.Tensor,
                  threshold: float = 6.0, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None):
    """`linear` with an outlier-column cache bound to Wq (bit-identical Y)."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    _require(cache, torch.uint8, "cache", 1)
    T, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or sW.shape[0] != N:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Wq {tuple(Wq.shape)}, sW {tuple(sW.shape)}")
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=X.device)
    _require(out, torch.float16, "out", 2)
    ws = _ws(workspace, T, K, N, X.device)
    _check("llm_int8_linear_cached",
           L.llm_int8_linear_cached(_ptr(X), _ptr(Wq), _ptr(sW), float(threshold), T, K, N,
                                    _ptr(out), _ptr(ws), ws.numel(), _ptr(cache), cache.numel(),
                                    _stream(X.device)))
    return out


def prepare_cached(X: torch.Tensor, Wq: torch.Tensor, threshold: float, workspace: torch.Tensor,
                   cache: torch.Tensor):
    """`prepare` with an outlier-column cache."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(Wq, torch.int8, "Wq", 2)
    _require(cache, torch.uint8, "cache", 1)
    T, K = X.shape
    N = Wq.shape[0]
    ws = _ws(workspace, T, K, N, X.device)
    _check("llm_int8_prepare_cached",
           L.llm_int8_prepare_cached(_ptr(X), _ptr(Wq), float(threshold), T, K, N, _ptr(ws),
                                     ws.numel(), _ptr(cache), cache.numel(), _stream(X.device)))
    return ws


def gemm_cached(Wq: torch.Tensor, sW: torch.Tensor, T: int, workspace: torch.Tensor,
                cache: torch.Tensor, out: torch.Tensor | None = None,
                acc: torch.Tensor | None = None):
    """`gemm` on a workspace from `prepare_cached` with the same cache."""
    L = load_library()
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    _require(cache, torch.uint8, "cache", 1)
    N, K = Wq.shape
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=Wq.device)
    _require(out, torch.float16, "out", 2)
    if acc is not None:
        _require(acc, torch.int32, "acc", 2)
    _require(workspace, torch.uint8, "workspace", 1)
    _check("llm_int8_gemm_cached",
           L.llm_int8_gemm_cached(_ptr(Wq), _ptr(sW), T, K, N, _ptr(out), _ptr(acc),
                                  _ptr(workspace), workspace.numel(), _ptr(cache), cache.numel(),
                                  _stream(Wq.device)))
    return out


def smoothquant_column_absmax(A: torch.Tensor, out: torch.Tensor | None = None):
    """max_r |A[r,j]| per column of fp16 A [rows,K], as fp32 [K]."""
    L = load_library()
    _require(A, torch.float16, "A", 2)
    rows, K = A.shape
    if out is None:
        out = torch.empty((K,), dtype=torch.float32, device=A.device)
    _require(out, torch.float32, "out", 1)
    _check("smoothquant_column_absmax",
           L.smoothquant_column_absmax(_ptr(A), rows, K, _ptr(out), _stream(A.device)))
    return out


def smoothquant_factors(ax: torch.Tensor, aw: torch.Tensor, alpha: float = 0.5):
    """(s, s_inv) fp32 [K]: s_j = ax_j^alpha / aw_j^(1-alpha) (1 where either
    maximum is 0) and fl32(1/s_j)."""
    L = load_library()
    _require(ax, torch.float32, "ax", 1)
    _require(aw, torch.float32, "aw", 1)
    K = ax.shape[0]
    if aw.shape[0] != K:
        raise ValueError(f"shape mismatch: ax {tuple(ax.shape)}, aw {tuple(aw.shape)}")
    s = torch.empty((K,), dtype=torch.float32, device=ax.device)
    s_inv = torch.empty((K,), dtype=torch.float32, device=ax.device)
    _check("smoothquant_factors",
           L.smoothquant_factors(_ptr(ax), _ptr(aw), float(alpha), K, _ptr(s), _ptr(s_inv),
                                 _stream(ax.device)))
    return s, s_inv


def smoothquant_quantize_weight(W: torch.Tensor, s: torch.Tensor):
    """(Wq int8 [N,K], sW fp32 [N]) of the smoothed weight fl32(W * s)."""
    L = load_library()
    _require(W, torch.float16, "W", 2)
    _require(s, torch.float32, "s", 1)
    N, K = W.shape
    if s.shape[0] != K:
        raise ValueError(f"shape mismatch: W {tuple(W.shape)}, s {tuple(s.shape)}")
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    sW = torch.empty((N,), dtype=torch.float32, device=W.device)
    _check("smoothquant_quantize_weight",
           L.smoothquant_quantize_weight(_ptr(W), _ptr(s), N, K, _ptr(Wq), _ptr(sW),
                                         _stream(W.device)))
    return Wq, sW


def smoothquant_prepare(X: torch.Tensor, s_inv: torch.Tensor, N: int, workspace: torch.Tensor):
    """Smoothed token codes and scales of X into `workspace` (no outlier
    column); `gemm` on it then gives the smoothed W8A8 product."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(s_inv, torch.float32, "s_inv", 1)
    T, K = X.shape
    if s_inv.shape[0] != K:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, s_inv {tuple(s_inv.shape)}")
    ws = _ws(workspace, T, K, N, X.device)
    _check("smoothquant_prepare",
           L.smoothquant_prepare(_ptr(X), _ptr(s_inv), T, K, N, _ptr(ws), ws.numel(),
                                 _stream(X.device)))
    return ws


def smoothquant_linear(X: torch.Tensor, s_inv: torch.Tensor, Wq: torch.Tensor,
                       sW: torch.Tensor, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None):
    """Y fp16 [T,N] of the smoothed W8A8 product (SmoothQuant-style)."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(s_inv, torch.float32, "s_inv", 1)
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    T, K = X.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or sW.shape[0] != N or s_inv.shape[0] != K:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, s_inv {tuple(s_inv.shape)}, "
                         f"Wq {tuple(Wq.shape)}, sW {tuple(sW.shape)}")
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=X.device)
    _require(out, torch.float16, "out", 2)
    ws = _ws(workspace, T, K, N, X.device)
    _check("smoothquant_linear",
           L.smoothquant_linear(_ptr(X), _ptr(s_inv), _ptr(Wq), _ptr(sW), T, K, N, _ptr(out),
                                _ptr(ws), ws.numel(), _stream(X.device)))
    return out


def export_stages(workspace: torch.Tensor, T: int, K: int, N: int) -> dict:
    """Device copies of the intermediate results of the last `prepare`."""
    L = load_library()
    _require(workspace, torch.uint8, "workspace", 1)
    dev = workspace.device
    nw = max((K + 31) // 32, 1)
    r = dict(
        outlier_bits=torch.empty(nw, dtype=torch.int32, device=dev),
        n_outliers=torch.empty(1, dtype=torch.int32, device=dev),
        outlier_idx=torch.empty(max(K, 1), dtype=torch.int32, device=dev),
        Xq=torch.empty((T, K), dtype=torch.int8, device=dev),
        sX=torch.empty(max(T, 1), dtype=torch.float32, device=dev),
        # gathered outlier values in 16-column chunks (see llm_int8.h)
        X_out=torch.empty(max(T * K, 1), dtype=torch.float16, device=dev),
    )
    _check("llm_int8_export_stages",
           L.llm_int8_export_stages(_ptr(workspace), workspace.numel(), T, K, N,
                                    _ptr(r["outlier_bits"]), _ptr(r["n_outliers"]),
                                    _ptr(r["outlier_idx"]), _ptr(r["Xq"]), _ptr(r["sX"]),
                                    _ptr(r["X_out"]), _stream(dev)))
    return r


def stages(X: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, threshold: float,
           workspace: torch.Tensor | None = None) -> dict:
    """Y and every intermediate result of one call (llm_int8_stages)."""
    L = load_library()
    _require(X, torch.float16, "X", 2)
    _require(Wq, torch.int8, "Wq", 2)
    _require(sW, torch.float32, "sW", 1)
    T, K = X.shape
    N = Wq.shape[0]
    dev = X.device
    ws = _ws(workspace, T, K, N, dev)
    r = dict(
        Y=torch.empty((T, N), dtype=torch.float16, device=dev),
        flags=torch.empty(max(K, 1), dtype=torch.uint8, device=dev),
        n_outliers=torch.empty(1, dtype=torch.int32, device=dev),
        outlier_idx=torch.empty(max(K, 1), dtype=torch.int32, device=dev),
        Xq=torch.empty((T, K), dtype=torch.int8, device=dev),
        sX=torch.empty(max(T, 1), dtype=torch.float32, device=dev),
        X_out=torch.empty((T, K), dtype=torch.float16, device=dev),
        acc=torch.empty((T, N), dtype=torch.int32, device=dev),
    )
    _check("llm_int8_stages",
           L.llm_int8_stages(_ptr(X), _ptr(Wq), _ptr(sW), float(threshold), T, K, N, _ptr(r["Y"]),
                             _ptr(ws), ws.numel(), _ptr(r["flags"]), _ptr(r["n_outliers"]),
                             _ptr(r["outlier_idx"]), _ptr(r["Xq"]), _ptr(r["sX"]),
                             _ptr(r["X_out"]), _ptr(r["acc"]), _stream(dev)))
    return r


# ---------------------------------------------------------------------------
# The int8 key/value cache (include/llm_int8_kv.h)
# ---------------------------------------------------------------------------

_KV_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


def _int32(value, name: str) -> int:
    """``value`` as the library's 32-bit fields and arguments take it: ctypes
    would cut a larger number to its low bits."""
    n = operator.index(value)
    if not -(1 << 31) <= n < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {n}")
    return n


class _CKVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _CKVBatch(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int32),
                ("seqs", ctypes.c_int32), ("tokens", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_kv", ctypes.c_int32)]


class _CRope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("dims", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class _Described:
    """An object whose description the library reads at every call: it is made
    once, so no name can be bound anew (the checks would see the new value and
    the library the old one)."""

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} is fixed: make a new object")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        raise AttributeError(f"{type(self).__name__}.{name} is fixed")


class KVCache(_Described):
    """Keys and values in int8, with one scale for each page of tokens and head:
    k, v int8 [pages, heads, page_size, head_dim], k_scale, v_scale fp32 [pages, heads].

    Holds the tensors and their description for the library; the checks are
    made here, once.  What the tensors hold may change, the tensors and their
    memory may not (no assignment, no ``resize_`` or ``set_``)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        _require(k, torch.int8, "k", 4)
        _require(v, torch.int8, "v", 4)
        _require(k_scale, torch.float32, "k_scale", 2)
        _require(v_scale, torch.float32, "v_scale", 2)
        if v.shape != k.shape or k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2]:
            raise ValueError(f"shape mismatch: k {tuple(k.shape)}, v {tuple(v.shape)}, "
                             f"k_scale {tuple(k_scale.shape)}, v_scale {tuple(v_scale.shape)}")
        _same_device(k, v=v, k_scale=k_scale, v_scale=v_scale)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        self.device = k.device
        self._c = _CKVCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), self.pages,
                            _int32(self.heads, "heads"), _int32(self.page_size, "page_size"),
                            _int32(self.head_dim, "head_dim"))
        self._ref = ctypes.addressof(self._c)


class KVBatch(_Described):
    """Sequences and their new rows: q_start int32 [seqs + 1], kv_len int32 [seqs],
    table int32 [seqs, width] of page numbers (rows may be strided).

    The rows q_start[s] .. q_start[s + 1] - 1 of the packed token tensors are
    the last ones of sequence s, which has kv_len[s] tokens with them.
    ``tokens`` is the packed tensors' row count; ``max_q`` and ``max_kv`` are
    at least the longest chunk and the longest sequence (the lengths
    themselves stay on the GPU).  What the tensors hold may change, so one
    object serves every step of a captured graph; the tensors, their memory
    and the numbers are fixed."""

    def __init__(self, q_start: torch.Tensor, kv_len: torch.Tensor, table: torch.Tensor, tokens: int,
                 max_q: int, max_kv: int):
        _require(q_start, torch.int32, "q_start", 1)
        _require(kv_len, torch.int32, "kv_len", 1)
        if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.dtype != torch.int32:
            raise TypeError("table must be a 2-dim torch.int32 tensor")
        if table.device.type != "cuda":
            raise ValueError(f"table must be on a GPU device, got {table.device}")
        S = kv_len.shape[0]
        if q_start.shape[0] != S + 1 or table.shape[0] != S:
            raise ValueError(f"shape mismatch: q_start {tuple(q_start.shape)}, kv_len {tuple(kv_len.shape)}, "
                             f"table {tuple(table.shape)}")
        if table.shape[1] > 1 and table.stride(1) != 1:
            raise ValueError("table's rows must be contiguous")
        _same_device(q_start, kv_len=kv_len, table=table)
        width = table.shape[1]
        stride = table.stride(0) if S > 1 else width
        if S > 1 and stride < width:
            raise ValueError("table's rows overlap")
        for name, n in (("tokens", tokens), ("max_q", max_q), ("max_kv", max_kv)):
            if not 0 <= n < 1 << 31:
                raise ValueError(f"{name} must be in [0, 2^31), got {n}")
        self.q_start, self.kv_len, self.table = q_start, kv_len, table
        self.seqs, self.tokens, self.max_q, self.max_kv = S, tokens, max_q, max_kv
        self.device = q_start.device
        self._c = _CKVBatch(_ptr(q_start), _ptr(kv_len), _ptr(table), stride, _int32(width, "table's width"),
                            _int32(S, "seqs"), tokens, max_q, max_kv)
        self._ref = ctypes.addressof(self._c)


class Rope(_Described):
    """Rotation of the first 2 * cos.shape[1] values of every head by position:
    cos, sin fp32 [rows, dims / 2]; pairs (i, i + dims/2), or (2i, 2i + 1) if
    ``interleaved``."""

    def __init__(self, cos: torch.Tensor, sin: torch.Tensor, interleaved: bool = False):
        _require(cos, torch.float32, "cos", 2)
        _require(sin, torch.float32, "sin", 2)
        if sin.shape != cos.shape:
            raise ValueError(f"shape mismatch: cos {tuple(cos.shape)}, sin {tuple(sin.shape)}")
        _same_device(cos, sin=sin)
        self.cos, self.sin, self.interleaved, self.device = cos, sin, bool(interleaved), cos.device
        self._c = _CRope(_ptr(cos), _ptr(sin), _int32(cos.shape[0], "rows"), _int32(2 * cos.shape[1], "dims"),
                         int(self.interleaved))
        self._ref = ctypes.addressof(self._c)


def _same_device(first: torch.Tensor, **others) -> None:
    for name, t in others.items():
        if t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


def _kv_tokens(t: torch.Tensor, name: str, batch: KVBatch, heads: int | None, dim: int) -> int:
    """Checks a packed token tensor [tokens, heads, dim] with dense rows and
    returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _KV_DTYPES:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != batch.tokens or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have shape ({batch.tokens}, {'heads' if heads is None else heads}, "
                         f"{dim}), got {tuple(shape)}")
    if t.device != batch.device:
        raise ValueError(f"{name} is on {t.device}, expected {batch.device}")
    if stride[2] != 1 or (shape[1] > 1 and stride[1] != dim):
        raise ValueError(f"{name}'s rows must be dense [heads, head_dim]")
    # a single row has no step: its stride may be anything
    return stride[0] if shape[0] > 1 else shape[1] * dim


def _kv_place(batch: KVBatch, cache: KVCache, rope: Rope | None = None) -> None:
    if not isinstance(batch, KVBatch) or not isinstance(cache, KVCache):
        raise TypeError("batch must be a KVBatch and cache a KVCache")
    if rope is not None and not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope or None")
    if cache.device != batch.device or (rope is not None and rope.device != batch.device):
        raise ValueError(f"batch, cache and rope must be on one device, got {batch.device}, {cache.device}"
                         + ("" if rope is None else f", {rope.device}"))


def _kv_call(name: str, device: torch.device, *args) -> None:
    """The library launches on the current device: make it the tensors'."""
    fn = getattr(_lib or load_library(), name)
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != 0:
        raise Int8MatmulError(name, status)


def new_kv_cache(pages: int, heads: int, head_dim: int, page_size: int, device) -> KVCache:
    """An empty cache (codes and scales zero)."""
    k = torch.zeros((pages, heads, page_size, head_dim), dtype=torch.int8, device=device)
    ks = torch.zeros((pages, heads), dtype=torch.float32, device=device)
    return KVCache(k, torch.zeros_like(k), ks, torch.zeros_like(ks))


def kv_append(K: torch.Tensor, V: torch.Tensor, cache: KVCache, batch: KVBatch,
              rope: Rope | None = None) -> KVCache:
    """Store the batch's new keys and values, fp16 or bf16 [tokens, heads, head_dim]
    (rows may be strided), the keys rotated by their positions on the way."""
    _kv_place(batch, cache, rope)
    ks = _kv_tokens(K, "K", batch, cache.heads, cache.head_dim)
    vs = _kv_tokens(V, "V", batch, cache.heads, cache.head_dim)
    if V.dtype != K.dtype:
        raise TypeError(f"V must be {K.dtype} like K, got {V.dtype}")
    _kv_call("int8_kv_append", batch.device, K.data_ptr(), ks, V.data_ptr(), vs, _KV_DTYPES[K.dtype],
             None if rope is None else rope._ref, batch._ref, cache._ref)
    return cache


def kv_read(cache: KVCache, batch: KVBatch, dtype: torch.dtype = torch.float16,
            out: tuple | None = None):
    """The values of the batch's rows back from the cache: (K, V), each
    [tokens, heads, head_dim] of ``dtype``.  Rows of no sequence are not written."""
    _kv_place(batch, cache)
    if dtype not in _KV_DTYPES:
        raise TypeError(f"dtype must be torch.float16 or torch.bfloat16, got {dtype}")
    if out is None:
        shape = (batch.tokens, cache.heads, cache.head_dim)
        K = torch.empty(shape, dtype=dtype, device=cache.device)
        V = torch.empty(shape, dtype=dtype, device=cache.device)
        ks = vs = cache.heads * cache.head_dim
    else:
        K, V = out
        ks = _kv_tokens(K, "out[0]", batch, cache.heads, cache.head_dim)
        vs = _kv_tokens(V, "out[1]", batch, cache.heads, cache.head_dim)
        if K.dtype != dtype or V.dtype != dtype:
            raise TypeError(f"out must be {dtype}, got {K.dtype} and {V.dtype}")
    _kv_call("int8_kv_read", batch.device, cache._ref, batch._ref, _KV_DTYPES[dtype], K.data_ptr(), ks,
             V.data_ptr(), vs)
    return K, V


def kv_attention_workspace_bytes(batch: KVBatch, cache: KVCache, q_heads: int) -> int:
    """Bytes of workspace that ``kv_attention`` needs (0: none)."""
    return int(load_library().int8_kv_attention_workspace_bytes(batch._ref, cache._ref,
                                                                _int32(q_heads, "q_heads")))


def new_kv_attention_workspace(batch: KVBatch, cache: KVCache, q_heads: int) -> torch.Tensor:
    return torch.empty(kv_attention_workspace_bytes(batch, cache, q_heads), dtype=torch.uint8,
                       device=cache.device)


KV_PATHS = {0: "empty", 1: "few", 2: "tiled"}


def kv_attention_plan(batch: KVBatch, cache: KVCache, q_heads: int, causal: bool = True,
                      window: int = 0) -> dict:
    """How ``kv_attention`` runs a batch of this shape: path, and the most
    parts that a row's keys are split into."""
    path, splits = ctypes.c_int32(), ctypes.c_int32()
    _check("int8_kv_attention_plan",
           load_library().int8_kv_attention_plan(batch._ref, cache._ref, _int32(q_heads, "q_heads"),
                                                 int(bool(causal)), _int32(window, "window"),
                                                 ctypes.byref(path), ctypes.byref(splits)))
    return dict(path=KV_PATHS[path.value], splits=splits.value)


def kv_attention(Q: torch.Tensor, cache: KVCache, batch: KVBatch, scale: float | None = None,
                 rope: Rope | None = None, causal: bool = True, window: int = 0,
                 out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the batch's rows Q, fp16 or bf16 [tokens, q_heads, head_dim],
    over the cache, after their keys and values were appended.

    ``scale`` defaults to 1/sqrt(head_dim); ``rope`` rotates Q on the way;
    ``window`` > 0 lets a row see its own and the window - 1 tokens before;
    ``lse`` fp32 [tokens, q_heads] receives the log of each row's sum (-inf
    for a row that sees no key; its output is 0).  Rows of no sequence, and
    those of a chunk past max_q, are not written.  Single tokens over long
    sequences are faster in a call of their own than beside a prompt's chunk."""
    _kv_place(batch, cache, rope)
    D = cache.head_dim
    qs = _kv_tokens(Q, "Q", batch, None, D)
    Hq = Q.shape[1]
    if out is None:
        out = torch.empty((batch.tokens, Hq, D), dtype=Q.dtype, device=Q.device)
        os_ = Hq * D
    else:
        os_ = _kv_tokens(out, "out", batch, Hq, D)
        if out.dtype != Q.dtype:
            raise TypeError(f"out must be {Q.dtype} like Q, got {out.dtype}")
    if lse is not None:
        _require(lse, torch.float32, "lse", 2)
        if tuple(lse.shape) != (batch.tokens, Hq) or lse.device != Q.device:
            raise ValueError(f"lse must be ({batch.tokens}, {Hq}) on {Q.device}, got {tuple(lse.shape)} "
                             f"on {lse.device}")
    if workspace is None:
        workspace = new_kv_attention_workspace(batch, cache, Hq)
    else:
        _require(workspace, torch.uint8, "workspace", 1)
        if workspace.device != Q.device:
            raise ValueError(f"workspace is on {workspace.device}, expected {Q.device}")
    _kv_call("int8_kv_attention", batch.device, Q.data_ptr(), qs, _KV_DTYPES[Q.dtype], _int32(Hq, "q_heads"),
             float(D ** -0.5 if scale is None else scale), None if rope is None else rope._ref,
             int(bool(causal)), _int32(window, "window"), batch._ref, cache._ref, out.data_ptr(), os_,
             _ptr(lse), workspace.data_ptr(), workspace.numel())
    return out


# ---------------------------------------------------------------------------
# The feed-forward operators (include/llm_int8_ffn.h)
# ---------------------------------------------------------------------------

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _matrix(t: torch.Tensor, name: str) -> torch.device:
    """Checks an fp16 [rows, columns] tensor on a GPU and returns its device."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is torch.float16 and t.dim() == 2
            and t.is_contiguous()):
        _require(t, torch.float16, name, 2)
    return t.device


def _fitted(t: torch.Tensor, dtype: torch.dtype, name: str, shape: tuple, device) -> int:
    """Checks a tensor of a known shape on a known device and returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.device == device):
        _require(t, dtype, name, len(shape))
        raise ValueError(f"{name} must be {tuple(shape)} on {device}, got {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _weight(Wq: torch.Tensor, sW: torch.Tensor, device, gated: bool) -> torch.Size:
    if not (isinstance(Wq, torch.Tensor) and Wq.dtype is torch.int8 and Wq.dim() == 2 and Wq.is_contiguous()
            and Wq.device == device):
        _require(Wq, torch.int8, "Wq", 2)
        raise ValueError(f"Wq is on {Wq.device}, expected {device}")
    shape = Wq.shape
    _fitted(sW, torch.float32, "sW", shape[:1], device)
    if gated and shape[0] % 2:
        raise ValueError(f"a gated pair's weight has an even number of rows, got {shape[0]}")
    return shape


def _scratch(workspace: torch.Tensor, device) -> tuple:
    if not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.uint8 and workspace.dim() == 1
            and workspace.is_contiguous() and workspace.device == device):
        _require(workspace, torch.uint8, "workspace", 1)
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    return workspace.data_ptr(), workspace.numel()


def _forward(name: str, X, Wq, sW, threshold, bias, activation, residual, out, pre, workspace, gated):
    dev = _matrix(X, "X")
    T, K = X.shape
    N, KW = _weight(Wq, sW, dev, gated)
    if KW != K:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Wq {tuple(Wq.shape)}")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    half = torch.float16
    F = N // 2 if gated else N
    if out is None:
        out = torch.empty((T, F), dtype=half, device=dev)
        y = out.data_ptr()
    else:
        y = _fitted(out, half, "out", (T, F), dev)
    b = None if bias is None else _fitted(bias, half, "bias", (N,), dev)
    p = None if pre is None else _fitted(pre, half, "pre", (T, N), dev)
    if workspace is None:
        need = linear_workspace_bytes(T, K, N)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    ws, size = (None, 0) if workspace is None else _scratch(workspace, dev)
    if gated:
        _kv_call(name, dev, X.data_ptr(), Wq.data_ptr(), sW.data_ptr(), threshold, T, K, F, b, act, y, p, ws, size)
    else:
        r = None if residual is None else _fitted(residual, half, "residual", (T, N), dev)
        _kv_call(name, dev, X.data_ptr(), Wq.data_ptr(), sW.data_ptr(), threshold, T, K, N, b, act, r, y, p, ws, size)
    return out


def linear_epilogue(X: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, threshold: float = 6.0,
                    bias: torch.Tensor | None = None, activation: str = "none",
                    residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    pre: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Y fp16 [T,N] = act(Z + bias) + residual, Z the product of ``linear``, rounded once.

    ``bias`` fp16 [N]; ``activation`` one of ACTIVATIONS; ``residual`` fp16 [T,N],
    which may be ``out`` itself; ``pre`` fp16 [T,N] receives Z + bias for
    ``linear_backward``.  The workspace is that of ``linear``."""
    return _forward("llm_int8_linear_epilogue", X, Wq, sW, float(threshold), bias, activation, residual, out, pre,
                    workspace, False)


def gated_linear(X: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, threshold: float = 6.0,
                 bias: torch.Tensor | None = None, activation: str = "silu", out: torch.Tensor | None = None,
                 pre: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """H fp16 [T,F] = act(G) * U, [G | U] = Z + bias with the pair's weight Wq [2F,K]
    (the gate's F rows, then the up-projection's).

    ``bias`` fp16 [2F]; ``pre`` fp16 [T,2F] receives [G | U] for ``gated_backward``.
    The workspace is that of ``linear`` for N = 2F."""
    return _forward("llm_int8_gated_linear", X, Wq, sW, float(threshold), bias, activation, None, out, pre, workspace,
                    True)


def _plan(name: str, fields: tuple, paths: dict, T: int, K: int, N: int, gated: bool) -> dict:
    out = (ctypes.c_int32 * len(fields))()
    _check(name, getattr(load_library(), name)(T, K, N, int(bool(gated)), out))
    return {f: paths[v] if f == "path" else v for f, v in zip(fields, out)}


def epilogue_plan(T: int, K: int, N: int, gated: bool = False) -> dict:
    """Which kernels ``linear_epilogue`` and ``gated_linear`` run for a weight of N rows (2F of a
    pair): path, tile_m, tile_n, fold_lo, fold_hi, ranges (of K), per_cu; see
    include/llm_int8_ffn_plan.h."""
    return _plan("llm_int8_epilogue_plan", ("path", "tile_m", "tile_n", "fold_lo", "fold_hi", "ranges", "per_cu"), PATHS,
                 T, K, N, gated)


BACKWARD_PATHS = {0: "empty", 1: "few", 2: "tiled", 3: "rows"}


def backward_plan(T: int, K: int, N: int, gated: bool = False) -> dict:
    """The same of the gradients: path, tile (rows), ranges (of the weight's rows), row_threads,
    row_rounds, strips."""
    return _plan("llm_int8_backward_plan", ("path", "tile", "ranges", "row_threads", "row_rounds", "strips"),
                 BACKWARD_PATHS, T, K, N, gated)


def backward_workspace_bytes(T: int, K: int, N: int) -> int:
    """Bytes of workspace for the gradients through a weight [N,K] (N = 2F for a pair)."""
    return int(load_library().llm_int8_backward_workspace_bytes(T, K, N))


def new_backward_workspace(T: int, K: int, N: int, device) -> torch.Tensor:
    return torch.empty(backward_workspace_bytes(T, K, N), dtype=torch.uint8, device=device)


def _backward(name: str, dY, pre, Wq, sW, activation, out, grad_pre, dbias, workspace, gated):
    dev = _matrix(dY, "dH" if gated else "dY")
    N, K = _weight(Wq, sW, dev, gated)
    T, F = dY.shape
    if F * (2 if gated else 1) != N:
        raise ValueError(f"shape mismatch: {'dH' if gated else 'dY'} {tuple(dY.shape)}, Wq {tuple(Wq.shape)}")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    half = torch.float16
    if pre is None:
        if gated or act:
            raise TypeError("pre must be a torch.Tensor")
        z = None
    else:
        z = _fitted(pre, half, "pre", (T, N), dev)
    g = None if grad_pre is None else _fitted(grad_pre, half, "grad_pre", (T, N), dev)
    b = None if dbias is None else _fitted(dbias, torch.float32, "dbias", (N,), dev)
    if out is None:
        out = torch.empty((T, K), dtype=half, device=dev)
        x = out.data_ptr()
    else:
        x = _fitted(out, half, "out", (T, K), dev)
    if workspace is None:
        need = backward_workspace_bytes(T, K, N)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    ws, size = (None, 0) if workspace is None else _scratch(workspace, dev)
    _kv_call(name, dev, dY.data_ptr(), z, act, Wq.data_ptr(), sW.data_ptr(), T, K, F, x, g, b, ws, size)
    return out


def linear_backward(dY: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, pre: torch.Tensor | None = None,
                    activation: str = "none", out: torch.Tensor | None = None, grad_pre: torch.Tensor | None = None,
                    dbias: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dX fp16 [T,K] of ``linear_epilogue`` (or ``linear``) for dY fp16 [T,N]: the gradient
    through the dequantized, frozen weight, dX = dZ . (Wq * sW), dZ = dY * act'(pre).

    ``pre`` fp16 [T,N] as the forward call stored it (not read without an
    activation); ``grad_pre`` fp16 [T,N] receives dZ, ``dbias`` fp32 [N] its column
    sums.  The residual's gradient is dY itself."""
    return _backward("llm_int8_linear_backward", dY, pre, Wq, sW, activation, out, grad_pre, dbias, workspace, False)


def gated_backward(dH: torch.Tensor, pre: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor,
                   activation: str = "silu", out: torch.Tensor | None = None, grad_pre: torch.Tensor | None = None,
                   dbias: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dX fp16 [T,K] of ``gated_linear`` for dH fp16 [T,F]: dG = dH U act'(G), dU = dH act(G),
    dX = [dG | dU] . (Wq * sW).

    ``pre`` fp16 [T,2F] as the forward call stored it; ``grad_pre`` fp16 [T,2F]
    receives [dG | dU], ``dbias`` fp32 [2F] their column sums."""
    return _backward("llm_int8_gated_backward", dH, pre, Wq, sW, activation, out, grad_pre, dbias, workspace, True)
