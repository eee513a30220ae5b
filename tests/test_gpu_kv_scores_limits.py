"""Caps and slopes at the ends of what is taken (GPU)."""
import pytest

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
