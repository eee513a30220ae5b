"""Caps and slopes at the ends of what is taken (GPU)."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from kv_ref import FP8, I8, U4
from test_gpu_kv_scores import Scored, both, ops  # noqa: F401
from test_gpu_kv_scores_many import Many, run

pytestmark = pytest.mark.gpu
FORMATS = [I8, FP8, U4]


@pytest.mark.parametrize("cap", [1e-50, -1e-50, 5e-324, 9.9e-31, 1.1e30, 3.5e38, 1e300, -1e300])
def test_caps_that_binary32_does_not_hold_are_refused(ops, cap):  # noqa: F811
    s = Scored(ops, I8, "bf16", 1, 2, 64, 16, [2], [40])
    t = Scored(ops, I8, "bf16", 1, 2, 64, 16, [2], [40], tree=True)
    for c in (s.c, t.c):
        with pytest.raises((ValueError, ops.BitGemmError), match="softcap"):
            c.run(ops, softcap=cap)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cap", [1e-30, 1e30])
def test_the_least_and_the_largest_cap(ops, fmt, cap):  # noqa: F811
    both(ops, fmt, "bf16", 2, 4, 128, 16, [5, 1, 0], [70, 300, 4], seed=1, cap=cap)
    run(ops, Many(ops, fmt, 64, 32, cap=cap), "k_kv_attn_many_cap" if cap < 1 else "k_kv_attn_many_far_cap", 4)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("how,slope", [(dict(), 3.4e38), (dict(), 1e30), (dict(cap=1e-30), 1e10), (dict(cap=0.01), 3.4e38), (dict(cap=1e4), 3.4e38)],
                         ids=lambda x: str(x))
def test_slopes_that_leave_a_query_its_own_position(ops, fmt, how, slope):  # noqa: F811
    """Finite slopes whose bias over one position passes binary32, or the slope itself in units of base 2 or of the cap: every
    other position weighs nothing, so a row is its own value, to its rounding."""
    for s in (Scored(ops, fmt, "f16", 1, 3, 64, 16, [1, 1], [40, 300], slopes=[slope, slope, 0.25], **how),
              Many(ops, fmt, 64, 32, group=2, gone=0.0, slopes=[slope, slope], **how)):
        c = s.c
        lse = torch.empty(c.q.shape[:2], device="cuda")
        got = s.run(ops, lse=lse).double().cpu().numpy()
        assert np.isfinite(got).all() and torch.isfinite(lse).all()
        first = 0
        for b, (n, length) in enumerate(zip(c.q_lens, c.kv_lens)):
            at = np.arange(length - n, length)
            page = c.table[b, at // c.page]
            own = (c.code[1][page, 0, at % c.page].astype(np.float64) if fmt != FP8 else ref.e4m3_decode(c.code[1][page, 0, at % c.page]))
            own = (own - c.zero[1][page, 0, at % c.page][:, None]) * c.scale[1][page, 0, at % c.page][:, None]
            u = 2.0 ** (-8 if c.dtype == "bf16" else -11)
            # the weight 1 times its value's scale to FP16, then the output's rounding
            tol = (u + 2.0 ** -11) * (1 + u) * np.abs(own) + 2.0 ** -24
            assert (np.abs(got[first:first + n, :2] - own[:, None]) <= tol[:, None]).all(), (b, n)
            first += n


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cap", [0.0, 20.0, 500.0])
def test_a_slope_of_nan_is_seen_in_its_head_alone(ops, fmt, cap):  # noqa: F811
    for s in (Scored(ops, fmt, "f16", 1, 3, 64, 16, [1, 1, 30], [1, 300, 40], cap=cap, slopes=[0.1, 0.1, 0.25]),
              Many(ops, fmt, 64, 32, group=2, cap=cap, slopes=[0.1, 0.01])):
        want = s.run(ops)
        s.how["slopes"][1] = float("nan")
        got = s.run(ops)
        assert torch.isnan(got[:, 1]).all() and torch.isfinite(got[:, 0]).all() and torch.equal(got[:, 0], want[:, 0])
