"""Windows at the ends of their range, and splits that the plan can take (GPU): the bound of test_gpu_kv.py."""
import pytest
import torch

from kv_ref import FP8, I8, U4
from test_gpu_kv import Case, ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens,kv_lens", [([9, 4], [4, 70]), ([200], [130])])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 40, 160, 129])
def test_windows_wider_than_the_positions_before_them(ops, q_lens, kv_lens, window):  # noqa: F811
    """Queries before the sequence less a wide window stay in range."""
    c = Case(ops, I8, "bf16", 1, 4, 64, 16, q_lens, kv_lens, seed=30, window=window, sinks=3)
    lse = torch.empty(sum(q_lens), 4, device="cuda")
    c.check(c.run(ops, lse=lse), lse)


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,kv,bound", [(1, 5000, 0), (25, 2100, 0), (60, 3000, 0), (150, 4200, 0), (150, 4200, 300), (600, 1500, 0)])
def test_splits(ops, fmt, D, rows, kv, bound):  # noqa: F811
    """Long sequences of few blocks (split and joined), and a bound on lengths that leaves the last split most of them."""
    c = Case(ops, fmt, "f16", 1, 1, D, 32, [rows], [kv], seed=31)
    lse = torch.empty(rows, 1, device="cuda")
    got = c.run(ops, lse=lse, max_kv_len=bound or kv)
    c.check(got, lse)
    assert torch.equal(got, c.run(ops, max_kv_len=bound or kv))


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
def test_value_scales_that_grow_along_the_sequence(ops, fmt):  # noqa: F811
    """The reference of the values' scales moves many times, up to 2^40 between a sequence's tokens."""
    for rows in (4, 150):
        c = Case(ops, fmt, "bf16", 1, 1, 128, 16, [rows], [900], seed=32)
        page = torch.from_numpy(c.table[0].astype("int64"))
        for j in range(0, 900, 16):
            f = 2.0 ** ((j // 64 * 3) % 15 if fmt == U4 else j // 24)
            c.scale[1][page[j // 16]] *= f
        rec = c.cache.v_scales
        new = torch.from_numpy(c.scale[1])
        live = torch.zeros(rec.shape[:3], dtype=torch.bool)
        for j in range(900):
            live[page[j // 16], :, j % 16] = True
        if fmt == U4:
            rec[..., 0] = torch.where(live, new.half(), rec[..., 0].cpu()).cuda()
            c.scale[1] = c.scale[1].astype("float16").astype("float32")
        else:
            rec.copy_(torch.where(live, new, rec.cpu()))
        c.check(c.run(ops))


def test_queries_of_very_different_size_in_one_block(ops):  # noqa: F811
    """Rows 2^20 apart share a block's power of two."""
    for rows in (6, 160):
        c = Case(ops, FP8, "bf16", 1, 2, 128, 16, [rows], [400], seed=33)
        c.q[::3] *= 2.0 ** -12
        c.q[1::3] *= 2.0 ** 4
        c.check(c.run(ops))
