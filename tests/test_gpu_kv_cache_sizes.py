"""The cache's writer and reader at the ends of their sizes (GPU)."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from kv_ref import FP8, I8, U4
from test_gpu_kv import ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
def test_as_many_tokens_as_a_call_takes(ops, fmt):  # noqa: F811
    """2^24 tokens (their rows one and the same in memory), nearly all skipped."""
    T, H, D = 1 << 24, 32, 64
    c = ops.kv_cache(2, 16, H, D, fmt)
    row = torch.randn(1, H, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    k = row.expand(T, H, D)
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    where = {0: 3, 1: 4, (1 << 23) - 1: 17, 1 << 23: 18, T - 2: 30, T - 1: 31}
    for t, s in where.items():
        slots[t] = s
    ops.kv_cache_write(k, k, c, slots)
    code, scale, zero = ref.quantize(row.float().cpu().numpy(), fmt)
    want = torch.from_numpy(ref.values(code, scale, zero, fmt).astype(np.float32))
    got, _ = ops.kv_cache_read(c, torch.arange(32).cuda(), torch.float32)
    for s in range(32):
        assert torch.equal(got[s].cpu(), want[0] if s in where.values() else torch.zeros(H, D)), s
