"""Rows and outputs that share a buffer: in place in every layout, refused where one would be written over another (GPU)."""
import pytest
import torch

from test_gpu_qk_rope import Rows, ops  # noqa: F401

pytestmark = pytest.mark.gpu
T, D = 37, 128


def views(layout, heads):
    """q, k and v [T][heads][D] in one buffer."""
    new = lambda *s: torch.randn(*s, generator=torch.Generator().manual_seed(1)).to("cuda:0", torch.bfloat16)  # noqa: E731
    if layout == "tokens, kinds, heads":
        return new(T, 3, heads, D).unbind(1)
    if layout == "tokens, heads, kinds":
        return new(T, heads, 3, D).unbind(2)
    if layout == "kinds, heads, tokens":
        return tuple(t.transpose(0, 1) for t in new(3, heads, T, D).unbind(0))
    return tuple(t.transpose(0, 1) for t in new(heads, 3, T, D).unbind(1))


@pytest.mark.parametrize("heads", [1, 5])
@pytest.mark.parametrize("layout", ["tokens, kinds, heads", "tokens, heads, kinds", "kinds, heads, tokens", "heads, kinds, tokens"])
def test_in_place(ops, layout, heads):  # noqa: F811
    c = Rows(ops, T, heads, heads, D, "bf16", 128)
    q, k, v = views(layout, heads)
    kept = v.clone()
    want = ops.qk_norm_rope(q, k, c.positions, c.freqs, **c.how)
    caches = [ops.kv_cache(3, 16, heads, D, ops.I8, "cuda:0") for _ in range(2)]
    slots = torch.arange(T, device="cuda:0")
    ops.kv_cache_write_rope(q, k, v, caches[0], slots, c.positions, c.freqs, **c.how)
    both = q.clone()
    ops.kv_cache_write_rope(q, k, v, caches[1], slots, c.positions, c.freqs, **c.how, q_out=q)
    assert torch.equal(q, want[0]) and torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    q.copy_(both)
    ops.qk_norm_rope(q, k, c.positions, c.freqs, **c.how, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)


@pytest.mark.parametrize("layout", ["tokens, kinds, heads", "tokens, heads, kinds", "kinds, heads, tokens", "heads, kinds, tokens"])
def test_refusals(ops, layout):  # noqa: F811
    c = Rows(ops, T, 5, 5, D, "bf16", 128)
    q, k, v = views(layout, 5)
    before = [t.clone() for t in (q, k, v)]
    new = torch.empty(T + 1, 5, D, dtype=torch.bfloat16, device="cuda:0")
    for out in (dict(q_out=k, k_out=q), dict(q_out=k), dict(k_out=q), dict(q_out=new[1:], k_out=new[:-1]), dict(q_out=new[:-1], k_out=new[:-1])):
        with pytest.raises(ops.BitGemmError, match="overlap"):
            ops.qk_norm_rope(q, k, c.positions, c.freqs, **c.how, **out)
    with pytest.raises(ops.BitGemmError, match="overlap"):          # a token further on
        ops.qk_norm_rope(q[:-1], k[:-1], c.positions[:-1], c.freqs, **c.how, q_out=q[1:])
    cache = ops.kv_cache(3, 16, 5, D, ops.I8, "cuda:0")
    for out in (k, v):
        with pytest.raises(ops.BitGemmError, match="overlap"):
            ops.kv_cache_write_rope(q, k, v, cache, torch.arange(T, device="cuda:0"), c.positions, c.freqs, **c.how, q_out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (q, k, v))) and not cache.k.any()
