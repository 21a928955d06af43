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


WIDE_MERGES = [
    # one block in more than 14 parts: a workgroup merges a column
    ([1], [20000], 1, 64, 64),
    ([1], [20000], 8, 64, 16),
    ([3], [9000], 9, 64, 32),        # 27 columns
    ([3], [9000], 9, 128, 64),
    ([4], [6000], 3, 128, 16),
    ([16], [7000], 1, 64, 128),
]


@pytest.mark.parametrize("ns, ls, group, dim, page", WIDE_MERGES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_merges_of_many_parts(ns, ls, group, dim, page, dtype):
    t = base.Setup(ns, ls, 1, dim, page, dtype, seed=group, rot=64, lead=1, tail=1)
    assert check(t, group, True, 0, 1.0, "few", True)["splits"] > 14


@pytest.mark.parametrize("dim, dtype", [(64, F16), (64, BF16), (128, F16), (128, BF16)])
def test_wide_blocks_past_512(dim, dtype):
    """20 columns in each of 560 blocks with short contexts: 32-column
    workgroups of 4 waves, unshared."""
    t = base.Setup([1] * 70, [(37 * i) % 90 for i in range(70)], 8, dim, 16, dtype, group=20)
    check(t, 160, True, 0, 2.0, "few", False)


@pytest.mark.parametrize("dim, group, dtype", [(64, 1, F16), (128, 1, BF16), (64, 17, F16)])
def test_blocks_past_sharing(dim, group, dtype):
    """4096 blocks or more go unshared whatever their lengths: a long sequence
    of 44 steps among short ones."""
    heads = 64
    t = base.Setup([1] * 64, [1400] + [1 + (7 * i) % 50 for i in range(63)], heads, dim, 64, dtype, group=group)
    check(t, heads * group, True, 0, 1.0, "few", False)
