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


@pytest.mark.parametrize("T,H,strides", [(1, 2, (131, 64, 1)), (5, 1, (72, 67, 1)), (1, 1, (3, 5, 1))])
def test_axes_of_one_element_may_have_any_stride(ops, T, H, strides):  # noqa: F811
    c = ops.kv_cache(2, 16, H, 64, FP8)
    buf = torch.randn(1024, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    x = buf.as_strided((T, H, 64), strides)
    slots = torch.arange(T).cuda()
    ops.kv_cache_write(x, x, c, slots)
    code, scale, zero = ref.quantize(x.float().cpu().numpy(), FP8)
    want = torch.from_numpy(ref.values(code, scale, zero, FP8).astype(np.float32))
    assert torch.equal(ops.kv_cache_read(c, slots, torch.float32)[0].cpu(), want)
    table, lens, cu = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([T], dtype=torch.int32).cuda(), torch.tensor([0, T], dtype=torch.int32).cuda()
    got = ops.kv_attn(x, c, table, lens, cu, T)
    assert torch.equal(got, ops.kv_attn(x.clone(memory_format=torch.contiguous_format), c, table, lens, cu, T))
