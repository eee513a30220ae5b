"""Steps planned over a pool of pages, and pages given back, against lists (GPU): every number equal."""
import numpy as np
import pytest
import torch

import kv_step_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_gemm_w4_amd import ops as _ops
    _ops.lib()
    return _ops


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda:0")


def same_state(pool, r):
    """The pool holds what the lists do."""
    count = len(r.free)
    assert pool.state.tolist() == [count, 0]
    assert pool.free[:count].tolist() == r.free
    assert pool.lens.tolist() == r.lens
    table = pool.block_table.tolist()
    for b, pages in enumerate(r.held):
        assert table[b][:len(pages)] == [-1 if p is None else p for p in pages], b
    held = [p for pages in r.held for p in pages if p is not None]
    assert len(set(held + r.free)) == len(held) + count        # no page twice


def same_plan(plan, want):
    for got, name, x in zip((plan.cu_q, plan.kv_lens, plan.served, plan.positions, plan.slots), ("cu_q", "kv_lens", "served", "positions", "slots"), want):
        assert got.tolist() == x, name


@pytest.mark.parametrize("batch,page,pages,width,tokens,most,window,sinks", [
    (1, 16, 40, 9, 30, 30, 0, 0),
    (3, 16, 25, 12, 64, 40, 0, 0),                # pages run out, tables too
    (7, 64, 200, 20, 1024, 200, 0, 0),
    (5, 16, 300, 60, 300, 90, 40, 4),             # a window and sinks
    (4, 32, 300, 60, 300, 90, 1, 33),             # a window of one token, sinks over a page's end
    (40, 16, 900, 25, 2500, 120, 100, 0),         # several blocks of rows
    (700, 16, 6000, 9, 5000, 9, 30, 17),
    (256, 16, 3000, 9, 300, 5, 40, 3), (257, 16, 3000, 9, 2000, 5, 0, 0), (513, 16, 3000, 9, 1500, 3, 25, 0),      # ends of a turn, of the waves' form
    (4097, 16, 5000, 3, 4096, 2, 0, 0),           # one sequence more than a turn of the blocks takes
])
def test_random_steps(ops, batch, page, pages, width, tokens, most, window, sinks):
    rng = np.random.default_rng(batch * 1000 + page)
    pool = ops.kv_pool(pages, page, batch, width, window=window, sinks=sinks, device="cuda:0")
    r = ref.Pool(pages, page, batch, width, window, sinks)
    same_state(pool, r)
    plan = None
    for step in range(14):
        kind = rng.integers(0, 6)
        if kind < 4:
            q = rng.integers(-1, most + 1, batch) * (rng.random(batch) < rng.choice([0.1, 0.5, 1.0]))
            advance = bool(kind < 3)
            plan = ops.kv_plan(pool, ints(q.tolist()), tokens, advance=advance, out=plan if step % 2 else None)
            *want, have = r.plan(q.tolist(), tokens, advance)
            same_plan(plan, want)
            table = pool.block_table.tolist()
            for b, pgs in enumerate(have):
                assert table[b][:len(pgs)] == [-1 if p is None else p for p in pgs], (step, b)
        elif kind == 4 and window:
            ops.kv_release(pool)
            r.release()
        else:
            # cut by up to a few tokens (a window's pages stay gone further back), end some
            cut = rng.integers(0, 4, batch)
            keep = [0 if rng.random() < 0.2 else max(0, n - int(c)) if not window else n for n, c in zip(r.lens, cut)]
            ops.kv_release(pool, ints(keep))
            r.release(keep)
        same_state(pool, r)


def test_a_step_taken_back_leaves_the_stack(ops):
    rng = np.random.default_rng(3)
    pool = ops.kv_pool(500, 16, 9, 80, device="cuda:0")
    ops.kv_plan(pool, ints([100, 0, 17, 3, 64, 1, 500, 16, 15]), 1000)
    ops.kv_release(pool, ints([50, 9, 0, 3, 64, 0, 30, 16, 99]))         # a stack in some order
    before = [t.clone() for t in (pool.lens, pool.free, pool.state)]
    for _ in range(3):
        ops.kv_plan(pool, ints(rng.integers(0, 90, 9).tolist()), 1000)
        ops.kv_release(pool, before[0])
        count = int(before[2][0])
        assert torch.equal(pool.lens, before[0]) and torch.equal(pool.state, before[2]) and torch.equal(pool.free[:count], before[1][:count])


def test_sequences_that_do_not_fit(ops):
    def plan(q, tokens, lens=(0, 0, 0, 0), free=100, width=4):
        pool = ops.kv_pool(100, 16, 4, width, device="cuda:0")
        pool.lens.copy_(ints(list(lens)))
        pool.state[0] = free
        p = ops.kv_plan(pool, ints(q), tokens)
        return p.served.tolist(), p.cu_q.tolist(), p.kv_lens.tolist(), [int((p.slots[a:b] >= 0).sum()) for a, b in zip(p.cu_q, p.cu_q[1:])]
    # rows: the third passes them, the fourth behind it too
    assert plan([3, 2, 6, 1], 10) == ([1, 1, 0, 0], [0, 3, 5, 10, 10], [3, 2, 0, 0], [3, 2, 0, 0])
    # the table: the second is too long; the others are not touched by it
    assert plan([3, 65, 64, 1], 200) == ([1, 0, 1, 1], [0, 3, 68, 132, 133], [3, 0, 64, 1], [3, 0, 64, 1])
    # pages: two, the second needs two of them; the last needs none
    assert plan([16, 17, 1, 1], 200, lens=(0, 0, 0, 0), free=2) == ([1, 0, 0, 0], [0, 16, 33, 34, 35], [16, 0, 0, 0], [16, 0, 0, 0])
    p = plan([16, 17, 0, 0], 200, free=0)
    assert p[0] == [0, 0, 1, 1] and p[2] == [0, 0, 0, 0]


def test_no_rows_and_absurd_lengths(ops):
    pool = ops.kv_pool(10, 16, 3, 4, device="cuda:0")
    p = ops.kv_plan(pool, ints([0, -5, 0]), 0)
    assert p.cu_q.tolist() == [0, 0, 0, 0] and p.served.tolist() == [1, 1, 1] and p.slots.numel() == 0
    p = ops.kv_plan(pool, ints([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]), 7)
    assert p.cu_q.tolist() == [0, 7, 7, 7] and p.served.tolist() == [0, 0, 0] and p.slots.tolist() == [-1] * 7 and p.positions.tolist() == list(range(7))
    p = ops.kv_plan(pool, ints([2, -2 ** 31, 3]), 9)
    assert p.positions.tolist() == [0, 1, 0, 1, 2, 0, 0, 0, 0] and p.slots.tolist()[5:] == [-1] * 4
    assert pool.state.tolist() == [8, 0]
    # lengths past the table count as its whole width
    pool.lens.copy_(ints([2 ** 31 - 1, -7, 64]))
    p = ops.kv_plan(pool, ints([0, 1, 1]), 2, advance=False)
    assert p.kv_lens.tolist() == [64, 1, 64] and p.served.tolist() == [1, 1, 0]


def test_a_captured_step_is_replayed(ops):
    """A decode loop in a graph: every replay goes on from the last one's pool."""
    pool, r = ops.kv_pool(900, 16, 60, 20, window=50, sinks=4, device="cuda:0"), ref.Pool(900, 16, 60, 20, 50, 4)
    q, keep = ints([40] * 60), None
    ops.kv_plan(pool, q, 2400)
    r.plan([40] * 60, 2400)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    out = ops.kv_plan(pool, q, 2400, advance=False)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        ops.kv_plan(pool, q, 2400, out=out)
        ops.kv_release(pool, keep)
    rng = np.random.default_rng(5)
    for rep in range(5):
        new = rng.integers(0, 41, 60).tolist()
        q.copy_(ints(new))
        torch.cuda.synchronize()
        g.replay()
        *want, _ = r.plan(new, 2400)
        r.release()
        torch.cuda.synchronize()
        same_plan(out, want)
        same_state(pool, r)


def test_another_stream(ops):
    pool, r = ops.kv_pool(300, 16, 6, 30, device="cuda:0"), ref.Pool(300, 16, 6, 30)
    side = torch.cuda.Stream()
    new = [5, 100, 0, 33, 16, 1]
    q = ints(new)
    side.wait_stream(torch.cuda.current_stream())
    p = ops.kv_plan(pool, q, 200, stream=side)
    ops.kv_release(pool, ints([5, 50, 0, 0, 16, 1]), stream=side)
    side.synchronize()
    same_plan(p, r.plan(new, 200)[:-1])
    r.release([5, 50, 0, 0, 16, 1])
    same_state(pool, r)


def test_refusals(ops):
    pool = ops.kv_pool(10, 16, 3, 4, device="cuda:0")
    with pytest.raises(ValueError, match="q_lens"):
        ops.kv_plan(pool, ints([1, 2]), 3)
    with pytest.raises(ValueError, match="q_lens"):
        ops.kv_plan(pool, ints([1, 2, 3]).long(), 6)
    with pytest.raises(ValueError, match="negative"):
        ops.kv_plan(pool, ints([1, 2, 3]), -1)
    with pytest.raises(ops.BitGemmError, match="tokens"):
        ops.kv_plan(pool, ints([1, 2, 3]), 2 ** 24 + 1, out=None)
    with pytest.raises(ValueError, match="one device"):
        ops.kv_plan(pool, ints([1, 2, 3]).cpu(), 6)
    with pytest.raises(ValueError, match="out.positions"):
        ops.kv_plan(pool, ints([1, 2, 3]), 6, out=ops.kv_plan(pool, ints([1, 2, 3]), 7, advance=False))
    with pytest.raises(ValueError, match="keep"):
        ops.kv_release(pool, ints([1, 2]))
    with pytest.raises(ValueError, match="page_size"):
        ops.kv_pool(10, 24, 3, 4, device="cuda:0")
    with pytest.raises(ValueError, match="window"):
        ops.kv_pool(10, 16, 3, 4, window=-1, device="cuda:0")
    with pytest.raises(ValueError, match="state"):
        ops.KVPool(pool.block_table, pool.lens, pool.gone, pool.free, pool.state[:1], 16)
