"""GPU tests of the attention over the int8 key/value cache against the bounds of
oracle/kv_error.py: every element within the worst that its row's roundings give,
and the norm of all errors within what they give as independent errors."""
import pytest
import torch

import int8_matmul_amd as li8
import test_gpu_kv as base
from oracle import kv_error

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def check(t, Hq, causal, window, q_scale=1.0, path=None, shared=None):
    plan = li8.kv_attention_plan(t.batch, t.cache, Hq, causal, window)
    assert path is None or (plan["path"], plan["splits"] > 1) == (path, shared), plan
    Q = t.rows(Hq, q_scale)
    lse = torch.full((t.tokens, Hq), 7.0, dtype=torch.float32, device=base.DEV)
    out = li8.kv_attention(Q, t.cache, t.batch, rope=t.rope, causal=causal, window=window, lse=lse)
    # fp16 outputs of at most 16 columns a workgroup: probabilities in two parts
    two = t.dtype == F16 and plan["path"] == "few" and min(t.batch.max_q, t.tokens) * (Hq // t.heads) <= 16
    r = kv_error.rows(t.ref, base.f32(Q), t.dim ** -0.5, t.q_start, t.ls, t.table, t.oracle_rope, causal, window,
                      torch.finfo(t.dtype).eps, two)
    wrong = kv_error.check(r, out.double().cpu().numpy(), lse.double().cpu().numpy())
    assert wrong is None, wrong
    return plan


@pytest.mark.parametrize("ns, ls, heads, group, dim, page, rot, causal, window", base.FEW)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_few(ns, ls, heads, group, dim, page, rot, causal, window, dtype):
    t = base.Setup(ns, ls, heads, dim, page, dtype, seed=page + group, rot=rot, inter=group % 2 == 0, lead=1, tail=2)
    check(t, heads * group, causal, window, 2.0, "few", False)


@pytest.mark.parametrize("ns, ls, heads, group, dim, page, rot, causal, window", base.SHARED)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_shared(ns, ls, heads, group, dim, page, rot, causal, window, dtype):
    t = base.Setup(ns, ls, heads, dim, page, dtype, seed=page + group, rot=rot, lead=1, tail=1)
    check(t, heads * group, causal, window, 1.0, "few", True)


@pytest.mark.parametrize("ns, ls, heads, group, dim, page, rot, causal, window, shared", base.TILED_RUNS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tiled(ns, ls, heads, group, dim, page, rot, causal, window, shared, dtype):
    rows = base.tiled_blocks(ns, heads, group, window, shared) * 256 // group
    t = base.Setup(ns, ls, heads, dim, page, dtype, seed=page + group, rot=rot, inter=page == 32, lead=1,
                   max_kv=1 << 14, max_q=rows, tail=max(0, rows - sum(ns)))
    check(t, heads * group, causal, window, 2.0, "tiled", shared)
