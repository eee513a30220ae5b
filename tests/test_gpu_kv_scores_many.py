"""The many-row kernels with other scores, each by its name, against binary64 (GPU).

Batches for which the rule of k_kvattn.hip takes the many-row kernel, in every format, head size and block.  The bound is
that of tests/test_gpu_kv_scores.py, which holds for either kernel.  Quiet queries keep every score below 0.4 of a far cap
(300 and more); loud ones beside them reach past the cap, in waves and blocks of their own and in shared ones.
"""
import copy
import functools

import numpy as np
import pytest
import torch

from kv_ref import FP8, I8, U4
from test_gpu_kv import Case
from test_gpu_kv_many_splits import PLANS
from test_gpu_kv_scores import Scored, ops  # noqa: F401

pytestmark = pytest.mark.gpu
FORMATS = [I8, FP8, U4]
ONLY = [0, 3, 15, 77, 150, 299]          # queries of a sequence that are compared


@functools.lru_cache(maxsize=None)
def case(ops, fmt, D, seqs, group, n, kv, gone, dtype, tree):  # noqa: F811
    """`seqs` sequences of n queries: n group rows each, as the plans count."""
    return Case(ops, fmt, dtype, 1, group, D, 32, [n] * seqs, [kv - 3 * i for i in range(seqs)], seed=D + seqs + fmt, gone=gone, tree=tree)


class Many(Scored):
    """Other queries, masks and scores over the cache of one of the cases."""

    def __init__(self, ops, fmt, D, seqs, *, group=2, n=300, kv=1437, loud=2.0, gone=0.05, dtype="bf16", tree=False, window=0, sinks=0, cap=0.0,  # noqa: F811
                 slopes=None, prefix=None):
        self.c = copy.copy(case(ops, fmt, D, seqs, group, n, kv, gone, dtype, tree))
        self.c.q, self.c.window, self.c.sinks = self.c.q * loud, window, sinks
        self.cap, self.how = cap, dict(softcap=cap)
        self.slopes = self.prefix = None
        if slopes is not None:
            self.slopes = np.resize(np.asarray(slopes, np.float32), group)
            self.how["slopes"] = torch.from_numpy(self.slopes).cuda()
        if prefix is not None:
            self.prefix = [max(0, prefix - 40 * i) for i in range(seqs)]
            self.how["prefix_lens"] = torch.tensor(self.prefix, dtype=torch.int32).cuda()


def run(ops, s, kernel, waves, split=True):  # noqa: F811
    """Through the kernel that is meant, in a workspace of exactly the bytes asked for, twice with the same bits."""
    c = s.c
    words = 0 if c.tree is None else c.tree.shape[1]
    need = ops.kv_attn_workspace_bytes(c.q.shape, c.cache, len(c.q_lens), c.bt.shape[1], c.max_q, c.max_kv, c.window, c.sinks, words)
    assert (need > 0) == split
    outs = []
    for fill in (0xFF, 0x00):
        lse = torch.empty(c.q.shape[:2], device="cuda")
        got = s.run(ops, lse=lse, ws=torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda"))
        assert ops.last_kernel() == f"{kernel}<{c.fmt}, {c.D}, {waves}>"
        outs.append((got, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    s.check(*outs[0], only=ONLY)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,seqs,waves", PLANS)
@pytest.mark.parametrize("how", [dict(slopes=[0.02, 2.0 ** -9]), dict(slopes=[0.0, 1.5]), dict(slopes=[-0.004, 0.1], prefix=1400),
                                 dict(prefix=1400), dict(prefix=2000, gone=0.0), dict(slopes=[0.01, 0.3], window=700, sinks=70),
                                 dict(prefix=1400, window=700, sinks=5)], ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
def test_biased(ops, fmt, D, seqs, waves, how):  # noqa: F811
    run(ops, Many(ops, fmt, D, seqs, **how), "k_kv_attn_many_bias", waves)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,seqs,waves", PLANS)
@pytest.mark.parametrize("how", [dict(cap=25.0), dict(cap=0.5, gone=0.0), dict(cap=256.0, loud=100.0), dict(cap=25.0, prefix=1400),
                                 dict(cap=10.0, window=700, sinks=70), dict(cap=25.0, prefix=1400, window=700)],
                         ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
def test_capped(ops, fmt, D, seqs, waves, how):  # noqa: F811
    run(ops, Many(ops, fmt, D, seqs, **how), "k_kv_attn_many_cap", waves)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,seqs,waves", PLANS)
@pytest.mark.parametrize("queries", ["quiet", "both"])
@pytest.mark.parametrize("how", [dict(cap=300.0), dict(cap=1000.0, gone=0.0), dict(cap=5e4, slopes=[0.01, 2.0 ** -8]),
                                 dict(cap=300.0, slopes=[0.02, 0.0], prefix=1400), dict(cap=300.0, window=700, sinks=70)],
                         ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()))
def test_capped_far(ops, fmt, D, seqs, waves, queries, how):  # noqa: F811
    s = Many(ops, fmt, D, seqs, **how)
    q = s.c.q.view(seqs, 300, *s.c.q.shape[1:])
    power = 2.0 ** (8 if how["cap"] < 2000 else 14)
    if queries == "both":
        q[:seqs // 2] *= power                   # whole sequences
        q[1] /= power
        q[1, 70:90] *= power                     # some rows of a wave
        q[seqs // 2:, 150] *= power
    run(ops, s, "k_kv_attn_many_far_cap", waves)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,seqs,waves", PLANS)
@pytest.mark.parametrize("cap,kernel", [(20.0, "k_kv_attn_many_cap"), (400.0, "k_kv_attn_many_far_cap")])
def test_capped_trees(ops, fmt, D, seqs, waves, cap, kernel):  # noqa: F811
    s = Many(ops, fmt, D, seqs, cap=cap, tree=True)
    if cap > 256:
        s.c.q[600:900] *= 2.0 ** 8
    run(ops, s, kernel, waves)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("how,kernel", [(dict(slopes=[0.02, 0.5]), "k_kv_attn_many_bias"), (dict(cap=20.0), "k_kv_attn_many_cap"),
                                        (dict(cap=20.0, slopes=[0.02]), "k_kv_attn_many_cap_bias"), (dict(cap=500.0, slopes=[0.01]), "k_kv_attn_many_far_cap")],
                         ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()) if isinstance(h, dict) else h)
def test_without_runs_and_in_fp16(ops, fmt, how, kernel):  # noqa: F811
    """As many sequences as fill the device: outputs come from the kernel itself."""
    run(ops, Many(ops, fmt, 128, 96, kv=437, dtype="f16", **how), kernel, 8, split=False)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,seqs,waves", PLANS)
@pytest.mark.parametrize("how,kernel", [(dict(slopes=[0.01]), "k_kv_attn_many_bias"), (dict(cap=20.0), "k_kv_attn_many_cap"),
                                        (dict(cap=500.0), "k_kv_attn_many_far_cap")], ids=lambda h: "-".join(h) if isinstance(h, dict) else h)
def test_rows_of_very_different_sizes(ops, fmt, D, seqs, waves, how, kernel):  # noqa: F811
    s = Many(ops, fmt, D, seqs, **how)
    s.c.q[3] *= 2.0 ** -20
    s.c.q[15] *= 2.0 ** 5
    s.c.q[77, 1] = 0.0
    run(ops, s, kernel, waves)
