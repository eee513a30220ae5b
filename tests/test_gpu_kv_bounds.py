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
