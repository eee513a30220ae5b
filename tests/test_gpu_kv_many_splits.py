"""The many-row kernel over several runs of positions, and which kernel ran (GPU)."""
import pytest
import torch

from kv_ref import FP8, I8, U4
from test_gpu_kv import Case, ops  # noqa: F401
from test_gpu_kv_many import Copies

pytestmark = pytest.mark.gpu

# D, sequences, waves of a block: those where the rule of k_kvattn.hip takes the many-row kernel and splits
PLANS = [(64, 16, 8), (64, 32, 4), (128, 32, 8), (256, 16, 4)]


def _run(ops, c, waves, tree=False, **kw):  # noqa: F811
    n = max(1, c.blocks // c.heads)
    words = c.tree.shape[1] if tree else 0
    need = ops.kv_attn_workspace_bytes((n * c.q.shape[0], c.q.shape[1]), c.cache, n, c.bt.shape[1], c.max_q,
                                       kw.get("max_kv_len", c.max_kv), c.window, c.sinks, words)
    assert need > 0                                             # split
    got = c.run(ops, **kw)
    assert ops.last_kernel() == f"k_kv_attn_many<{c.fmt}, {c.D}, {waves}>"
    return got


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("D,seqs,waves", PLANS)
@pytest.mark.parametrize("kv", [1437, 4200])
def test_a_bound_that_leaves_the_last_run_the_rest(ops, fmt, D, seqs, waves, kv):  # noqa: F811
    c = Copies(ops, fmt, "f16", 1, 1, D, 32, [600], [kv], seed=70)
    c.blocks = seqs
    lse = torch.empty(600, 1, device="cuda")
    c.check(_run(ops, c, waves, lse=lse, max_kv_len=1437), lse)


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("D,seqs,waves", PLANS[:1] + PLANS[2:])
@pytest.mark.parametrize("window,sinks", [(700, 0), (760, 70)])
def test_windows(ops, fmt, D, seqs, waves, window, sinks):  # noqa: F811
    c = Copies(ops, fmt, "bf16", 1, 1, D, 32, [600], [4200], seed=71, window=window, sinks=sinks)
    c.blocks = seqs
    lse = torch.empty(600, 1, device="cuda")
    c.check(_run(ops, c, waves, lse=lse), lse)


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("D,seqs,waves", PLANS)
def test_trees_and_short_sequences(ops, fmt, D, seqs, waves):  # noqa: F811
    """Runs that a shorter sequence leaves empty, and pages that are not there."""
    c = Copies(ops, fmt, "bf16", 1, 1, D, 32, [600, 3], [1437, 40], seed=72, tree=True, gone=0.2)
    c.blocks = seqs                                             # pairs: half as many of each
    n = seqs // 2
    lse = torch.empty(603, 1, device="cuda")
    need = ops.kv_attn_workspace_bytes((n * 603, 1), c.cache, 2 * n, c.bt.shape[1], 600, 1437, tree_words=c.tree.shape[1])
    assert need > 0
    c.check(c.run(ops, lse=lse), lse)
    assert ops.last_kernel() == f"k_kv_attn_many<{fmt}, {D}, {waves}>"


@pytest.mark.parametrize("cu", [[-5, 3, 7], [0, 3, 1 << 30], [-(1 << 31), 3, (1 << 31) - 1]])
def test_offsets_outside_the_tokens_are_clamped(ops, cu):  # noqa: F811
    c = Case(ops, FP8, "bf16", 2, 2, 64, 16, [3, 4], [20, 30], seed=13)
    lse = torch.empty(7, 4, device="cuda")
    c.check(ops.kv_attn(c.q, c.cache, c.bt, c.lens, torch.tensor(cu, dtype=torch.int32).cuda(), 4, lse=lse), lse)
