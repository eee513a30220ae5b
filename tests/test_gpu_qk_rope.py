"""Head norms and rotary positions, alone and on the way into the quantized cache, against binary64 (GPU).

Queries, and keys that stay rows, are computed in binary32: their norm's factor is off by at most
(13 / 2 + 5) half steps (a sum of 8 products a lane and 5 exchanges at most, under a root; the root, the
quotient, the weight's sum and two products), the rotation by 4 more (cosine and sine rounded, two
operations): 16 2^-24 of |a| + |b|, and the result's rounding to its type, half a step.  Keys on
their way to codes are within 2^-49 of the formula before their rounding to binary32, so about one in 2^24
rounds another way, and of those one in 2^16 gets another code: none here.
"""
import numpy as np
import pytest
import torch

import kv_ref
import kv_step_ref as ref
from kv_ref import FP8, I8, U4

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_gemm_w4_amd import ops as _ops
    _ops.lib()
    return _ops


def wide(t):
    return t.double().cpu().numpy()


class Rows:
    def __init__(self, ops, T, q_heads, kv_heads, dim, dtype, rot, interleaved=False, norm=True, weight="same", offset=0.0, eps=1e-6, far=1000, seed=0,
                 fused=True):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        widths = [q_heads * dim, kv_heads * dim, kv_heads * dim]
        row = torch.randn(T, sum(widths) + 8, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
        row = row.to("cuda:0", dt)
        parts = row[:, :sum(widths)].split(widths, 1)
        self.q, self.k, self.v = (p.unflatten(1, (-1, dim)) if fused or not p.numel() else p.unflatten(1, (-1, dim)).contiguous() for p in parts)
        self.dtype, self.dim, self.T, self.kv_heads = dtype, dim, T, kv_heads
        wt = torch.float32 if weight == "f32" else dt
        self.qw, self.kw = ((1 - offset + 0.3 * torch.randn(dim, generator=g)).to("cuda:0", wt) if norm else None for _ in range(2))
        pos = torch.randint(-far if far < 1000 else 0, far, (T,), generator=g)
        self.positions = pos.to("cuda:0", torch.int32)
        self.inv = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
        self.freqs = ops.rope_freqs(torch.tensor(self.inv, dtype=torch.float64, device="cuda:0")) if rot else None
        self.turns = [f % 2 ** 64 for f in self.freqs.tolist()] if rot else []
        self.how = dict(q_weight=self.qw, k_weight=self.kw, eps=eps, weight_offset=offset, interleaved=interleaved)
        self.ref = dict(interleaved=interleaved, eps=eps, offset=offset)

    def want(self, x, w):
        return ref.turn(wide(x), None if w is None else wide(w), self.positions.tolist(), self.turns, **self.ref)

    def check(self, got, x, w):
        y = self.want(x, w)
        half = len(self.turns)
        size = np.abs(ref.turn(wide(x), None if w is None else wide(w), self.positions.tolist(), [], **self.ref))
        pair = size.copy()
        if self.ref["interleaved"]:
            both = size[..., 0:2 * half:2] + size[..., 1:2 * half:2]
            pair[..., 0:2 * half:2] = pair[..., 1:2 * half:2] = both
        else:
            both = size[..., :half] + size[..., half:2 * half]
            pair[..., :half] = pair[..., half:2 * half] = both
        tiny = 2.0 ** -25 if self.dtype == "f16" else 2.0 ** -150       # half of the least subnormal
        lim = HALF_STEP[self.dtype] * (np.abs(y) + 16 * 2.0 ** -24 * pair) + 16 * 2.0 ** -24 * pair + tiny
        err = np.abs(wide(got) - y)
        assert got.dtype == DT[self.dtype] and (err <= lim).all(), (err / lim).max()


CASES = [
    dict(T=1, q_heads=4, kv_heads=1, dim=128, dtype="bf16", rot=128),
    dict(T=5, q_heads=32, kv_heads=8, dim=128, dtype="bf16", rot=128, interleaved=True),
    dict(T=33, q_heads=6, kv_heads=2, dim=64, dtype="f16", rot=64),
    dict(T=17, q_heads=1, kv_heads=1, dim=64, dtype="f16", rot=16, interleaved=True),
    dict(T=130, q_heads=1, kv_heads=1, dim=256, dtype="bf16", rot=256),
    dict(T=67, q_heads=10, kv_heads=5, dim=256, dtype="f16", rot=64),
    dict(T=40, q_heads=8, kv_heads=8, dim=128, dtype="f32", rot=32, interleaved=True),
    dict(T=9, q_heads=3, kv_heads=3, dim=256, dtype="f32", rot=8),
    dict(T=50, q_heads=4, kv_heads=2, dim=128, dtype="bf16", rot=0),
    dict(T=50, q_heads=4, kv_heads=2, dim=128, dtype="f16", rot=64, norm=False),
    dict(T=50, q_heads=4, kv_heads=2, dim=64, dtype="bf16", rot=64, weight="f32", offset=1.0, eps=1e-5),
    dict(T=20, q_heads=4, kv_heads=2, dim=128, dtype="f32", rot=128, far=2 ** 31 - 1),
    dict(T=70, q_heads=200, kv_heads=3, dim=64, dtype="bf16", rot=64, far=300),      # negative positions too
    dict(T=700, q_heads=16, kv_heads=16, dim=128, dtype="bf16", rot=128),
    dict(T=20, q_heads=4, kv_heads=2, dim=128, dtype="f16", rot=128, fused=False),
    dict(T=1100, q_heads=64, kv_heads=1, dim=256, dtype="f16", rot=256),          # queries in long runs, keys a slot each
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_rows(ops, case):
    c = Rows(ops, **case)
    before = c.q.clone(), c.k.clone()
    q, k = ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs, **c.how)
    c.check(q, c.q, c.qw)
    c.check(k, c.k, c.kw)
    assert torch.equal(c.q, before[0]) and torch.equal(c.k, before[1])
    one, none = ops.qk_norm_rope(c.q, None, c.positions, c.freqs, **c.how)
    assert none is None and torch.equal(one, q)
    none, one = ops.qk_norm_rope(None, c.k, c.positions, c.freqs, **c.how)
    assert none is None and torch.equal(one, k)
    # heads before tokens
    out = torch.zeros(c.q.shape[1], c.T, c.dim, dtype=c.q.dtype, device="cuda:0").transpose(0, 1)
    assert torch.equal(ops.qk_norm_rope(c.q, None, c.positions, c.freqs, **c.how, q_out=out)[0], q)
    # in place, in the fused rows
    ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs, **c.how, q_out=c.q, k_out=c.k)
    assert torch.equal(c.q, q) and torch.equal(c.k, k)


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_rows_into_the_cache(ops, case, fmt):
    c = Rows(ops, **case, seed=fmt)
    page, pages = 16, c.T // 16 + 3
    cache = ops.kv_cache(pages, page, c.kv_heads, c.dim, fmt, "cuda:0")
    g = torch.Generator().manual_seed(7)
    slots = torch.randperm(pages * page, generator=g)[:c.T]
    slots[torch.rand(c.T, generator=g) < 0.1] = -1
    if c.T > 3:
        slots[1], slots[2] = pages * page, -2 ** 40
    at = slots.cuda()
    q = ops.kv_cache_write_rope(c.q, c.k, c.v, cache, at, c.positions, c.freqs, **c.how)
    assert torch.equal(q, ops.qk_norm_rope(c.q, None, c.positions, c.freqs, **c.how)[0])
    ok = ((slots >= 0) & (slots < pages * page)).numpy()
    p, o = slots.numpy()[ok] // page, slots.numpy()[ok] % page
    k32 = c.want(c.k, c.kw).astype(np.float32)
    for x, codes, records in ((k32, cache.k, cache.k_scales), (wide(c.v).astype(np.float32), cache.v, cache.v_scales)):
        code, scale, zero = kv_ref.quantize(x[ok], fmt)
        got = codes.cpu().numpy()
        got = (kv_ref.unpack_u4(got) if fmt == U4 else got)[p, :, o]
        rec = records.cpu().numpy()[p, :, o]
        assert np.array_equal(got, code)
        assert np.array_equal(rec, np.stack((scale, zero), -1).astype(np.float16) if fmt == U4 else scale)
        # nothing else was written
        rest = records.clone()
        rest[torch.from_numpy(p).cuda(), :, torch.from_numpy(o).cuda()] = 0
        assert not rest.any()
    # keys alone
    other = ops.kv_cache(pages, page, c.kv_heads, c.dim, fmt, "cuda:0")
    assert ops.kv_cache_write_rope(None, c.k, c.v, other, at, c.positions, c.freqs, **c.how) is None
    for a, b in ((cache.k, other.k), (cache.v, other.v), (cache.k_scales, other.k_scales), (cache.v_scales, other.v_scales)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_norm_and_rotation_it_is_the_plain_write(ops, fmt, dtype):
    c = Rows(ops, 37, 4, 3, 128, dtype, 0, norm=False)
    a, b = (ops.kv_cache(5, 16, 3, 128, fmt, "cuda:0") for _ in range(2))
    slots = torch.randperm(80)[:37].cuda()
    c.k[3, 1, 5], c.k[4, 0, 0], c.v[5, 2, 127], c.k[6, 1] = float("nan"), float("inf"), -float("inf"), 0.0
    q = ops.kv_cache_write_rope(c.q, c.k, c.v, a, slots, None, None)
    ops.kv_cache_write(c.k, c.v, b, slots)
    assert torch.equal(q, c.q)
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scales, b.k_scales), (a.v_scales, b.v_scales)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("norm", [False, True])
def test_infinities_nan_zeros_and_large_rows(ops, norm):
    """What one row holds reaches no other; rows of zeros stay zeros; keys whose squares pass binary32 are normed."""
    c = Rows(ops, 8, 2, 2, 128, "bf16", 128, norm=norm)
    clean = ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs, **c.how)
    c.q[2, 1, 3], c.k[3, 0, 70], c.q[5], c.k[5] = float("nan"), float("inf"), 0.0, 0.0
    q, k = ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs, **c.how)
    keep = torch.ones(8, 2, dtype=torch.bool)
    keep[2, 1] = keep[5] = False
    assert torch.equal(q[keep], clean[0][keep]) and not torch.isfinite(q[2, 1]).all()
    assert (q[5] == 0).all() and (k[5] == 0).all() and not torch.isfinite(k[3, 0]).all()
    cache = ops.kv_cache(1, 16, 2, 128, I8, "cuda:0")
    c.k[7] = c.k[7] * 2.0 ** 100
    ops.kv_cache_write_rope(c.q, c.k, c.v, cache, torch.arange(8).cuda(), c.positions, c.freqs, **c.how)
    got, _ = ops.kv_cache_read(cache, torch.arange(8).cuda(), torch.float32)
    assert torch.isnan(got[3, 0]).all() and (got[5] == 0).all()
    scale = cache.k_scales[0].T.double().cpu().numpy()[..., None]
    rows = [0, 1, 2, 4, 6, 7]
    want = c.want(c.k, c.kw)[rows]
    # half a step, and a few roundings of the scale, the quotient and the product
    assert (np.abs(wide(got)[rows] - want) <= 0.5 * scale[rows] + 2.0 ** -21 * np.abs(want)).all()


def test_far_positions_turn_exactly(ops):
    """The angle of position p is p times that of 1 modulo a turn, whatever p."""
    freqs = ops.rope_freqs(torch.tensor([1.0, 0.5, 2.0 ** -20, 3.0], dtype=torch.float64, device="cuda:0"))
    pos = [0, 1, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 31 - 1, -1, -2 ** 31]
    x = torch.zeros(len(pos), 1, 64, device="cuda:0")
    x[..., :4] = 1.0
    _, y = ops.qk_norm_rope(None, x, torch.tensor(pos, dtype=torch.int32, device="cuda:0"), freqs)
    from fractions import Fraction
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    for i, p in enumerate(pos):
        for n, f in enumerate((1.0, 0.5, 2.0 ** -20, 3.0)):
            t = float(Fraction(p) * Fraction(f) % (2 * pi))           # within 2^-52 2 pi of the angle
            c, s = np.cos(t), np.sin(t)
            # a frequency is off by half of 2^-64 turns, so a position below 2^31 by 2^-34 turns
            assert abs(float(y[i, 0, n]) - c) <= 2.0 ** -23 and abs(float(y[i, 0, n + 4]) - s) <= 2.0 ** -23


def test_a_captured_call_is_replayed(ops):
    c = Rows(ops, 20, 8, 2, 128, "bf16", 128)
    cache, other = (ops.kv_cache(4, 16, 2, 128, FP8, "cuda:0") for _ in range(2))
    slots, out = torch.randperm(64)[:20].cuda(), torch.empty(20, 8, 128, dtype=torch.bfloat16, device="cuda:0")
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        ops.kv_cache_write_rope(c.q, c.k, c.v, cache, slots, c.positions, c.freqs, **c.how, q_out=out)
    for rep in range(4):
        c.positions += 1000 * rep
        c.k.mul_(1.5)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        want = ops.kv_cache_write_rope(c.q, c.k, c.v, other, slots, c.positions, c.freqs, **c.how)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(cache.k, other.k) and torch.equal(cache.k_scales, other.k_scales), rep


def test_another_stream(ops):
    c = Rows(ops, 20, 8, 2, 128, "bf16", 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs, **c.how, stream=side)
    side.synchronize()
    for a, b in zip(got, ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs, **c.how)):
        assert torch.equal(a, b)


def test_no_tokens(ops):
    c = Rows(ops, 0, 4, 2, 64, "f16", 64)
    q, k = ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs, **c.how)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    cache = ops.kv_cache(1, 16, 2, 64, I8, "cuda:0")
    assert ops.kv_cache_write_rope(c.q, c.k, c.v, cache, torch.zeros(0, dtype=torch.int64, device="cuda:0"), c.positions, c.freqs).shape == (0, 4, 64)


def test_refusals(ops):
    c = Rows(ops, 4, 4, 2, 128, "bf16", 128)
    args = (c.q, c.k, c.positions, c.freqs)
    with pytest.raises(ValueError, match="queries or keys"):
        ops.qk_norm_rope(None, None, c.positions, c.freqs)
    with pytest.raises(ValueError, match="positions"):
        ops.qk_norm_rope(c.q, c.k, c.positions[:3], c.freqs)
    with pytest.raises(ValueError, match="positions"):
        ops.qk_norm_rope(c.q, c.k, None, c.freqs)
    with pytest.raises(ValueError, match="freqs"):
        ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs.double())
    with pytest.raises(ValueError, match="q must be"):
        ops.qk_norm_rope(c.q.half(), c.k, c.positions, c.freqs)
    with pytest.raises(ValueError, match="weights"):
        ops.qk_norm_rope(*args, q_weight=c.qw, k_weight=c.kw.float())
    with pytest.raises(ValueError, match="weights"):
        ops.qk_norm_rope(*args, q_weight=c.qw[:64])
    with pytest.raises(ValueError, match="q_out"):
        ops.qk_norm_rope(*args, q_out=c.k)
    with pytest.raises(ValueError, match="overlap"):
        ops.qk_norm_rope(*args, q_out=c.q[:, :1].expand(4, 4, 128))
    with pytest.raises(ValueError, match="one device"):
        ops.qk_norm_rope(c.q, c.k, c.positions.cpu(), c.freqs)
    with pytest.raises(ValueError, match="device tensors"):
        ops.qk_norm_rope(c.q.cpu(), c.k.cpu(), c.positions.cpu(), c.freqs.cpu())
    with pytest.raises(ops.BitGemmError, match="rot"):
        ops.qk_norm_rope(c.q, c.k, c.positions, torch.zeros(65, dtype=torch.int64, device="cuda:0"))
    with pytest.raises(ops.BitGemmError, match="multiple of 8"):
        ops.qk_norm_rope(c.q, c.k, c.positions, c.freqs[:6])
    with pytest.raises(ops.BitGemmError, match="eps"):
        ops.qk_norm_rope(*args, eps=-1.0)
    with pytest.raises(ops.BitGemmError, match="head_dim"):
        ops.qk_norm_rope(c.q[..., :96].contiguous(), None, c.positions, c.freqs[:48])
    with pytest.raises(ops.BitGemmError, match="16-byte aligned"):
        ops.qk_norm_rope(torch.zeros(4 * 4 * 128 + 4, dtype=torch.bfloat16, device="cuda:0")[4:].view(4, 4, 128), None, c.positions, c.freqs)
    cache = ops.kv_cache(1, 16, 2, 128, I8, "cuda:0")
    with pytest.raises(ValueError, match="must be"):
        ops.kv_cache_write_rope(c.q, c.q, c.v, cache, torch.arange(4).cuda(), c.positions, c.freqs)
    with pytest.raises(ValueError, match="slots"):
        ops.kv_cache_write_rope(c.q, c.k, c.v, cache, torch.arange(4).cuda().int(), c.positions, c.freqs)
