"""Many pages given back in one call: more than the launch has lanes, so that its teams take their items in turns (GPU).

The launch counts on eight pages a sequence: a wave's 64 items for each eight sequences up to 512 of them, blocks of 1,024
beyond.  Every number against the lists of tests/kv_step_ref.py.
"""
import numpy as np
import pytest

import kv_step_ref as ref
from test_gpu_kv_plan import ints, ops, same_state  # noqa: F401

import torch

pytestmark = pytest.mark.gpu


def both(ops, pages, page, batch, width, window=0, sinks=0):  # noqa: F811
    return ops.kv_pool(pages, page, batch, width, window=window, sinks=sinks, device="cuda:0"), ref.Pool(pages, page, batch, width, window, sinks)


def fill(ops, pool, r, lens):  # noqa: F811
    n = sum(lens)
    ops.kv_plan(pool, ints(lens), n)
    assert all(r.plan(lens, n)[2])


def back(ops, pool, r, keep, per_turn):  # noqa: F811
    before = len(r.free)
    ops.kv_release(pool, None if keep is None else ints(keep))
    r.release(keep)
    same_state(pool, r)
    table = pool.block_table.tolist()
    for b, pages in enumerate(r.held):
        assert all(table[b][i] == -1 for i, p in enumerate(pages) if p is None), b
    assert len(r.free) - before > per_turn


@pytest.mark.parametrize("batch,lens", [
    (1, [1000 * 16]), (1, [66 * 16]), (3, [16 * 129, 5, 16 * 300]), (8, [16 * 20 * i + i for i in range(8)]),
    (9, [16 * 40] * 9), (40, [16 * (i % 7) * 12 + i for i in range(40)]), (512, [16 * 33] * 511 + [16 * 200]),
    (513, [16 * 9] * 512 + [16 * 9000]), (600, [16 * (20 + i % 3) for i in range(600)]), (4100, [16 * 10] * 4100)])
def test_ended_sequences(ops, batch, lens):  # noqa: F811
    """All at once, then again after others have come and gone; a sequence of few pages kept."""
    page, per_turn = 16, 64 * -(-batch // 8)
    if batch > 512:
        per_turn = 1024 * -(-per_turn // 1024)
    width = max(lens) // page + 2
    pool, r = both(ops, sum(-(-n // page) for n in lens) + 3, page, batch, width)
    rng = np.random.default_rng(batch)
    for turn in range(3):
        fill(ops, pool, r, [lens[i] for i in rng.permutation(batch)])
        keep = [0] * batch
        if turn:
            keep[batch // 2] = min(r.lens[batch // 2], 5)
        back(ops, pool, r, keep, per_turn)
        ops.kv_release(pool, ints([0] * batch))
        r.release([0] * batch)
        same_state(pool, r)


@pytest.mark.parametrize("batch,tokens,window,sinks", [(1, 16 * 900, 100, 33), (6, 16 * 200, 1, 16), (8, 16 * 150, 40, 0), (30, 16 * 60, 77, 40),
                                                      (530, 16 * 40, 50, 17)])
def test_windows(ops, batch, tokens, window, sinks):  # noqa: F811
    """Slid pages alone; slid ones and the end's together; the sinks' and the end's of sequences whose middle is gone."""
    page, per_turn = 16, 64 * -(-batch // 8)
    if batch > 512:
        per_turn = 1024 * -(-per_turn // 1024)
    lens = [tokens + 5 * (i % 40) for i in range(batch)]
    width = 2 * (max(lens) // page) + 3
    pool, r = both(ops, batch * width, page, batch, width, window, sinks)
    fill(ops, pool, r, lens)
    back(ops, pool, r, None, per_turn)
    fill(ops, pool, r, lens)
    # what slid below the place that is kept, and what lies past it
    back(ops, pool, r, [n - tokens // 2 for n in r.lens], per_turn)
    # the sinks' pages and the last ones: few, whatever lies between
    keep = [3 if sinks else 0] * batch
    ops.kv_release(pool, ints(keep))
    r.release(keep)
    same_state(pool, r)
    assert len(r.free) == batch * width - (batch if sinks else 0)


def test_replayed(ops):  # noqa: F811
    """In a graph: long sequences planned and ended, three times over."""
    pool, r = both(ops, 700, 16, 4, 300)
    q, keep = ints([16 * 200, 5, 16 * 150, 16 * 90]), ints([0, 5, 0, 16])
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ops.kv_plan(pool, q, 16 * 500)
        ops.kv_release(pool, keep)
    same_state(pool, r)
    for new in ([16 * 200, 5, 16 * 150, 16 * 90], [1, 0, 16 * 290, 16 * 299], [0, 16 * 280, 3, 16 * 250]):
        q.copy_(ints(new))
        torch.cuda.synchronize()
        g.replay()
        r.plan(new, 16 * 500)
        r.release([0, 5, 0, 16])
        torch.cuda.synchronize()
        same_state(pool, r)
