"""What may and what may not be handed to a plan or a release twice (GPU)."""
import pytest
import torch

import kv_step_ref as ref
from test_gpu_kv_plan import ints, ops, same_plan, same_state  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_plan_over_its_own_operands_is_refused(ops):  # noqa: F811
    """The tokens of those served: from another plan's tensors, or a copy."""
    B = 300
    pool, r = ops.kv_pool(400, 16, B, 5, device="cuda:0"), ref.Pool(400, 16, B, 5)
    new = [17 if i % 3 else 1 for i in range(B)]
    plan = ops.kv_plan(pool, ints(new), 4000)
    same_plan(plan, r.plan(new, 4000)[:-1])
    before = [t.clone() for t in pool._tensors]
    for q in (plan.served, plan.kv_lens, plan.cu_q[1:], plan.positions[:B]):
        with pytest.raises(ops.BitGemmError, match="overlap"):
            ops.kv_plan(pool, q, 4000, out=plan)
    for out in (dict(kv_lens=pool.lens), dict(served=plan.kv_lens), dict(served=pool.gone)):
        parts = {n: getattr(plan, n) for n in ("cu_q", "kv_lens", "served", "positions", "slots")}
        with pytest.raises(ops.BitGemmError, match="overlap"):
            ops.kv_plan(pool, ints(new), 4000, out=ops.KVPlan(**{**parts, **out}))
    with pytest.raises(ops.BitGemmError, match="overlap"):
        ops.kv_release(pool, pool.free[:B])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, pool._tensors))
    served = plan.served.tolist()
    assert 0 in served and 1 in served
    for q in (plan.served, plan.served.clone()):
        again = ops.kv_plan(pool, q, 4000, advance=False)
        same_plan(again, r.plan(served, 4000, advance=False)[:-1])
    same_plan(ops.kv_plan(pool, plan.served.clone(), 4000, out=plan), r.plan(served, 4000)[:-1])
    same_state(pool, r)


@pytest.mark.parametrize("batch", [3, 300, 700])
def test_the_pools_own_lengths(ops, batch):  # noqa: F811
    """As many tokens again as each holds; all of them kept."""
    pool, r = ops.kv_pool(batch * 6, 16, batch, 9, device="cuda:0"), ref.Pool(batch * 6, 16, batch, 9)
    new = [i % 23 for i in range(batch)]
    ops.kv_plan(pool, ints(new), 23 * batch)
    r.plan(new, 23 * batch)
    same_plan(ops.kv_plan(pool, pool.lens, 23 * batch), r.plan(list(r.lens), 23 * batch)[:-1])
    ops.kv_release(pool, pool.lens)
    r.release(list(r.lens))
    same_state(pool, r)
    ops.kv_release(pool, pool.gone)                 # no window: zeros
    r.release([0] * batch)
    same_state(pool, r)
