"""The host's bound on a sequence's queries: without it every query is computed, and those past it are left alone (GPU)."""
import pytest
import torch

from kv_ref import FP8, I8, U4
from test_gpu_kv import Case, ops  # noqa: F401

pytestmark = pytest.mark.gpu

# q_lens, kv_lens, shape, tree: whole and split, both kernels
CALLS = [([5, 1, 3], [70, 1, 300], (2, 4, 128, 16), False), ([1, 1, 1], [900, 1, 5000], (1, 3, 64, 16), False),
         ([40, 300], [100, 900], (2, 2, 64, 16), False), ([150], [2000], (3, 5, 128, 32), False), ([20, 64], [400, 64], (1, 2, 256, 16), True)]


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("q_lens,kv_lens,shape", [c[:3] for c in CALLS if not c[3]])
def test_without_a_bound_every_query_is_computed(ops, fmt, q_lens, kv_lens, shape):  # noqa: F811
    c = Case(ops, fmt, "bf16", *shape, q_lens, kv_lens, seed=50)
    T = sum(q_lens)
    out, lse = torch.full((T, c.q.shape[1], c.D), float("nan"), dtype=c.q.dtype, device="cuda"), torch.empty(T, c.q.shape[1], device="cuda")
    ops.kv_attn(c.q, c.cache, c.bt, c.lens, c.cu, out=out, lse=lse)
    c.check(out, lse)
    need = ops.kv_attn_workspace_bytes(c.q.shape, c.cache, len(q_lens), c.bt.shape[1])
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    assert torch.equal(ops.kv_attn(c.q, c.cache, c.bt, c.lens, c.cu, ws=ws), out)


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("q_lens,kv_lens,shape,tree", CALLS + [([16, 2], [400, 90], (1, 1, 64, 16), False), ([7], [9000], (3, 5, 64, 16), False)])
@pytest.mark.parametrize("most", [1, 3, 37])
def test_queries_past_the_bound_are_left_alone(ops, fmt, q_lens, kv_lens, shape, tree, most):  # noqa: F811
    c = Case(ops, fmt, "bf16", *shape, q_lens, kv_lens, seed=51, tree=tree)
    T = sum(q_lens)
    want, want_lse = torch.empty(T, c.q.shape[1], c.D, dtype=c.q.dtype, device="cuda"), torch.empty(T, c.q.shape[1], device="cuda")
    c.run(ops, out=want, lse=want_lse)
    for copies in (1, 128 // len(q_lens)):       # few blocks (split) and many
        cu = torch.cat([c.cu[:1]] + [c.cu[1:] + n * T for n in range(copies)])
        args = (c.q.repeat(copies, 1, 1), c.cache, c.bt.repeat(copies, 1), c.lens.repeat(copies), cu)
        out = torch.full((copies * T, *want.shape[1:]), 7.0, dtype=c.q.dtype, device="cuda")
        lse = torch.full((copies * T, want.shape[1]), 7.0, device="cuda")
        if tree:
            ops.kv_attn_tree(*args, c.tree.repeat(copies, 1), most, max_kv_len=c.max_kv, out=out, lse=lse)
        else:
            ops.kv_attn(*args, most, max_kv_len=c.max_kv, out=out, lse=lse)
        past = torch.cat([torch.arange(n) >= most for n in q_lens]).repeat(copies).cuda()
        assert (out[past] == 7.0).all() and (lse[past] == 7.0).all()
        for n in range(copies):
            got, got_lse = out[n * T:(n + 1) * T].clone(), lse[n * T:(n + 1) * T].clone()
            p = past[:T]
            got[p], got_lse[p] = want[p], want_lse[p]
            if n in (0, copies - 1):
                c.check(got, got_lse)


def test_rows_that_a_new_output_cannot_get_are_zeros(ops):  # noqa: F811
    c = Case(ops, FP8, "bf16", 1, 2, 64, 16, [1, 1], [40, 90], seed=52)
    q = torch.cat((c.q, c.q, c.q)).contiguous()                  # four rows of padding
    torch.full((6, 2, 64), float("nan"), dtype=q.dtype, device="cuda")
    got = ops.kv_attn(q, c.cache, c.bt, c.lens, c.cu, 1)
    assert not got[2:].any()
    c.check(got[:2])


RAGGED = [  # queries of each sequence, positions, shape: their mean says little
    ([1] * 40, [200 + 7 * i for i in range(40)], (2, 4, 128, 16)),
    ([3, 0, 0, 1, 0, 2, 1, 1], [60, 5, 0, 900, 30, 2, 1, 40], (1, 4, 64, 16)),
    ([0, 0, 300, 0, 1, 1, 1, 0, 0, 1], [9, 0, 700, 3, 50, 1, 33, 2, 4, 800], (2, 2, 64, 32)),
    ([1, 33, 1, 1, 70, 1, 200, 1, 1, 5, 0, 0], [40, 33, 1000, 2, 500, 64, 260, 1, 90, 70, 3, 0], (1, 5, 128, 16)),
    ([130, 1, 1, 1], [4000, 60, 3000, 1], (1, 1, 256, 16)),
    ([1, 150, 150, 1, 1, 1, 1, 1], [30, 150, 1200, 30, 31, 32, 33, 34], (1, 16, 64, 16)),
]


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("q_lens,kv_lens,shape", RAGGED)
@pytest.mark.parametrize("kind", ["causal", "window", "tree"])
def test_sequences_far_from_their_mean(ops, fmt, q_lens, kv_lens, shape, kind):  # noqa: F811
    """A bound of all the queries: each is computed once, in its own sequence's blocks or past the batch's."""
    c = Case(ops, fmt, "bf16", *shape, q_lens, kv_lens, seed=53, tree=kind == "tree", **(dict(window=100, sinks=3) if kind == "window" else {}))
    T, heads = sum(q_lens), c.q.shape[1]
    c.max_q = T
    for copies in (1, 24):                          # few blocks (split) and many
        cu = torch.cat([c.cu[:1]] + [c.cu[1:] + n * T for n in range(copies)])
        q = torch.cat((c.q.repeat(copies, 1, 1), c.q[:5].float().mul(0).to(c.q.dtype)))          # five rows that no sequence owns
        args = (q, c.cache, c.bt.repeat(copies, 1), c.lens.repeat(copies), cu)
        out, lse = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
        kw = dict(max_kv_len=c.max_kv, out=out, lse=lse)
        if kind == "tree":
            tree = torch.cat((c.tree.repeat(copies, 1), c.tree[:5]))
            call = lambda: ops.kv_attn_tree(*args, tree, q.shape[0], **kw)  # noqa: E731
        else:
            call = lambda: ops.kv_attn(*args, window=c.window, sinks=c.sinks, **kw)  # noqa: E731
        call()
        first = out.clone(), lse.clone()
        assert (out[copies * T:] == 7.0).all() and (lse[copies * T:] == 7.0).all()
        for n in (0, copies - 1):
            c.check(out[n * T:(n + 1) * T], lse[n * T:(n + 1) * T])
        call()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_as_many_sequences_as_a_call_takes(ops):  # noqa: F811
    """65,535 sequences of no, one or three queries without a bound; and one fewer, whose grid leaves one block past the batch."""
    for B in (65535, 65534, 40000):
        c = Case(ops, I8, "bf16", 1, 1, 64, 16, [1, 0, 3, 0, 1], [9, 4, 20, 0, 33], seed=54)
        n = B // 5
        T = 5 * n
        cu = torch.cat([c.cu[:1]] + [(c.cu[1:][None] + 5 * torch.arange(n, dtype=torch.int32, device="cuda")[:, None]).reshape(-1),
                                     torch.full((B - 5 * n,), T, dtype=torch.int32, device="cuda")])
        pad = torch.zeros(B - 5 * n, c.bt.shape[1], dtype=torch.int32, device="cuda")
        got = ops.kv_attn(c.q.repeat(n, 1, 1), c.cache, torch.cat((c.bt.repeat(n, 1), pad)), torch.cat((c.lens.repeat(n), pad[:, 0])), cu,
                          max_kv_len=33)
        rows = got.view(n, 5, 1, 64)
        assert torch.equal(rows.view(torch.int16), rows[:1].expand_as(rows).contiguous().view(torch.int16))
        c.check(rows[0])
