"""Each query row of the attention over the KV cache by itself (GPU): what a row does not see, and what the
other rows of its block hold, must not reach its result.

The bound is taken row by row, over the tokens that the row sees:

* the output's own rounding, u_out |y| (2^-8 BF16, 2^-11 FP16);
* the rounding to FP16 of each weight times its value's scale, w s: 2^-11 relative, or, where it falls below
  FP16's normal range, half of FP16's last step.  The row's largest w s lies at 2^3 at least, so that step is
  2^-24 / 2^3 of it and the error of a token 2^-28 max(w s) |code|, rows of zeros aside;
* binary32 scores and sums as in test_gpu_kv.py.

Where a row sees a value whose scale is infinite, the result is infinite or NaN element by element, as in binary64.
"""
import numpy as np
import pytest
import torch

import kv_ref as ref
from kv_ref import FP8, I8, U4
from test_gpu_kv import Case, _records, ops  # noqa: F401
from test_gpu_kv_many import Copies

pytestmark = pytest.mark.gpu

FORMATS = [I8, FP8, U4]
KERNELS = ["few", "many"]


def check_rows(c, got, lse=None, scale=None):
    scale = c.D ** -0.5 if scale is None else scale
    u_out = 2.0 ** (-8 if c.dtype == "bf16" else -11)
    got, q = got.double().cpu().numpy(), c.q.double().cpu().numpy()
    first = 0
    for b, (n, length) in enumerate(zip(c.q_lens, c.kv_lens)):
        ids = c.table[b, :-(-length // c.page)]
        there = (ids >= 0) & (ids < c.cache.pages)
        see = ref.visible(n, length, there.repeat(c.page)[:length], c.window, c.sinks, c.bits[b] if c.bits else None)
        safe = np.where(there, ids, 0)
        for h in range(c.heads):
            k, v = (ref.values(c.code[x][safe, h], c.scale[x][safe, h], c.zero[x][safe, h], c.fmt).reshape(-1, c.D)[:length] for x in range(2))
            s_v = np.abs(c.scale[1][safe, h].reshape(-1)[:length].astype(np.float64))
            code = np.abs(ref.values(c.code[1][safe, h], np.ones_like(c.scale[1][safe, h]), c.zero[1][safe, h], c.fmt)).reshape(-1, c.D)[:length]
            for i in range(n):
                at = np.flatnonzero(see[i])
                for g in range(c.group):
                    hq = h * c.group + g
                    x = got[first + i, hq]
                    if not at.size:
                        assert not x.any()
                        assert lse is None or lse[first + i, hq].item() == -np.inf
                        continue
                    s = k[at] @ q[first + i, hq] * scale
                    w = np.exp(s - s.max())
                    total = w.sum()
                    y = w @ v[at] / total
                    top = (np.abs(k[at]) @ np.abs(q[first + i, hq])).max() * scale
                    rel = (2 * (c.D + 16) * top + at.size + 16) * 2.0 ** -24
                    lost = 2.0 ** -28 * (w * s_v[at] * code[at].any(1)).max() * code[at].sum(0) / total
                    tol = u_out * np.abs(y) + (1 + u_out) * ((2.0 ** -11 + rel) * (w @ np.abs(v[at]) / total) + lost)
                    tol = tol + (2.0 ** -25 if c.dtype == "f16" else 2.0 ** -133)
                    with np.errstate(invalid="ignore"):
                        bad = ~((np.abs(x - y) <= tol) | (x == y) | (np.isnan(x) & np.isnan(y)))
                    assert not bad.any(), (b, i, hq, np.flatnonzero(bad)[:4], x[bad][:4], y[bad][:4], tol[bad][:4])
                    if lse is not None:
                        want = s.max() + np.log(total)
                        assert abs(lse[first + i, hq].item() - want) <= rel + 2.0 ** -22 * (abs(want) + 1)
        first += n


def _case(ops, kernel, *args, **kw):  # noqa: F811
    return (Case if kernel == "few" else Copies)(ops, *args, **kw)


def _run(ops, c, kernel, **kw):  # noqa: F811
    got = c.run(ops, **kw)
    assert ops.last_kernel().startswith(f"k_kv_attn_{kernel}<")
    return got


def _scales(c, n, change):
    """change(scales, the slots of the sequences' tokens) -> new scales of the keys (0) or values (1)."""
    live = np.zeros(c.scale[n].shape, bool)
    for b, length in enumerate(c.kv_lens):
        for j in range(length):
            live[c.table[b, j // c.page], :, j % c.page] = True
    new = np.where(live, change(c.scale[n].astype(np.float64)), c.scale[n])
    new = new.astype(np.float16).astype(np.float32) if c.fmt == U4 else new.astype(np.float32)
    rec = c.cache.v_scales if n else c.cache.k_scales
    old = rec.cpu().numpy()
    if c.fmt == U4:
        old[..., 0] = np.where(live, new, old[..., 0])
    else:
        old = np.where(live, new, old)
    rec.copy_(torch.from_numpy(old))
    c.scale[n] = np.where(live, new, c.scale[n])


def _token(c, b, j):
    return c.table[b, j // c.page], slice(None), j % c.page


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt,ratio", [(U4, 24), *((f, r) for f in (I8, FP8) for r in (24, 60, 140))])     # an FP16 scale spans 2^40
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_a_loud_value_stays_with_the_rows_that_see_it(ops, kernel, fmt, D, tree, ratio):  # noqa: F811
    """The last token of a chunk, or one drafted token of a tree, has a value 2^ratio times the others'."""
    n = 6 if kernel == "few" else 150
    for length in ((n, 40) if kernel == "few" else (n, 300)):
        c = _case(ops, kernel, fmt, "bf16", 1, 2, D, 16, [n], [length], seed=ratio, tree=tree)
        loud = length - 1 if not tree else length - n + 2
        _scales(c, 1, lambda s: s * 2.0 ** (-8 if fmt == U4 else -40))
        at = _token(c, 0, loud)

        def shout(s):
            s = s.copy()
            s[at] *= 2.0 ** ratio
            return s
        _scales(c, 1, shout)
        lse = torch.empty(n, 2, device="cuda")
        check_rows(c, _run(ops, c, kernel, lse=lse), lse)


def _sink(ops, kernel, fmt, share):  # noqa: F811
    n, length, D = (1, 131072, 64) if kernel == "few" else (130, 40000, 64)
    rng = np.random.default_rng(3)
    c = Copies(ops, fmt, "f16", 1, 1, D, 128, [n], [length], seed=41)
    c.blocks = 512 if kernel == "few" else 256
    u = rng.standard_normal(D)
    c.q.copy_(torch.from_numpy((u + 0.01 * rng.standard_normal((n, 1, D))).astype(np.float16)))
    x = 0.3 * rng.standard_normal(c.code[0].shape)
    x[_token(c, 0, 0)] = u * (np.log(share / (1 - share) * length) + 0.15) * D ** 0.5 / (u @ u)
    code, s, z = ref.quantize(x.astype(np.float32), fmt)
    c.code[0], c.scale[0], c.zero[0] = code, s, z
    c.cache.k.copy_(torch.from_numpy(ref.pack_u4(code) if fmt == U4 else code))
    c.cache.k_scales.copy_(torch.from_numpy(_records(s, z, fmt)))
    return c


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("share", [0.9, 0.99, 0.9999])
def test_a_first_token_that_takes_the_weight(ops, kernel, fmt, share):  # noqa: F811
    """A long sequence whose first token has `share` of each row's weight and a value near zero: the others' small
    weights make the result, in blocks that walk the whole sequence."""
    c = _sink(ops, kernel, fmt, share)
    at = _token(c, 0, 0)

    def hush(s):
        s = s.copy()
        s[at] *= 2.0 ** -10
        return s
    _scales(c, 1, hush)
    check_rows(c, _run(ops, c, kernel))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt", [I8, FP8])
@pytest.mark.parametrize("size", [3.2e38, 1e30, 1e-30, 1e-35])
@pytest.mark.parametrize("kv", [700, 5000])
def test_values_at_the_ends_of_the_range(ops, kernel, fmt, size, kv):  # noqa: F811
    c = _case(ops, kernel, fmt, "bf16", 1, 4, 128, 16, [5 if kernel == "few" else 40], [kv], seed=42)
    v = np.abs(ref.values(c.code[1], c.scale[1], c.zero[1], fmt))
    most = max(v[_token(c, 0, j)].max() for j in range(kv))
    _scales(c, 1, lambda s: s * (size / most))
    got = _run(ops, c, kernel)
    assert got.isfinite().all()
    check_rows(c, got)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_negative_scales(ops, kernel, fmt):  # noqa: F811
    """A scale's sign is its value's, as where slots are read back."""
    c = _case(ops, kernel, fmt, "f16", 1, 4, 128, 16, [5 if kernel == "few" else 40], [700], seed=43)
    rng = np.random.default_rng(4)
    _scales(c, 1, lambda s: -s)
    check_rows(c, _run(ops, c, kernel))
    for n in (0, 1):
        _scales(c, n, lambda s: s * rng.choice([-1.0, 1.0], s.shape))
    check_rows(c, _run(ops, c, kernel))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [30, 60, 90])
def test_scores_past_the_integers_of_binary32(ops, kernel, fmt, size):  # noqa: F811
    """Queries of 2^size: a row is its best token's value, never NaN."""
    n = 6 if kernel == "few" else 150
    c = _case(ops, kernel, fmt, "bf16", 1, 2, 128, 16, [n], [330], seed=46)
    c.q *= 2.0 ** size
    lse = torch.empty(n, 2, device="cuda")
    check_rows(c, _run(ops, c, kernel, lse=lse), lse)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ratio", [20, 40, 90])
def test_queries_of_any_size_in_one_block(ops, kernel, fmt, D, ratio):  # noqa: F811
    """Every third query is 2^ratio times the others, or 2^-ratio; some rows are zeros."""
    n = 6 if kernel == "few" else 150
    for sign in (1, -1):
        c = _case(ops, kernel, fmt, "bf16", 1, 2, D, 16, [n], [330], seed=44)
        c.q[::3] *= 2.0 ** (sign * ratio)
        c.q[1, 0] = 0.0
        lse = torch.empty(n, 2, device="cuda")
        check_rows(c, _run(ops, c, kernel, lse=lse), lse)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_keeps_to_its_row(ops, kernel, bad):  # noqa: F811
    c = _case(ops, kernel, FP8, "bf16", 1, 2, 128, 16, [6 if kernel == "few" else 150], [330], seed=45)
    c.q[2, 1, 7] = bad
    got = _run(ops, c, kernel)
    assert got[2, 1].isnan().all()
    c.q[2, 1] = 0.0
    got[2, 1] = c.run(ops)[2, 1]
    check_rows(c, got)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("share", [0.5, 0.99])
def test_a_first_token_of_zeros_that_takes_the_weight(ops, kernel, fmt, share):  # noqa: F811
    """Its value is written as codes 0 with scale 1, far above the others' scales."""
    c = _sink(ops, kernel, fmt, share)
    _scales(c, 1, lambda s: s * 2.0 ** -6)
    at, pages = _token(c, 0, 0), c.cache
    zeros = torch.zeros(1, 1, c.D, device="cuda")
    keep = pages.k.clone(), pages.k_scales.clone()
    if fmt == FP8:
        zeros[..., ::3] = -0.0                       # E4M3 has two zeros
    ops.kv_cache_write(zeros, zeros, pages, torch.tensor([int(at[0]) * c.page + at[2]]).cuda())
    pages.k.copy_(keep[0])
    pages.k_scales.copy_(keep[1])
    c.code[1][at], c.scale[1][at], c.zero[1][at] = 0, 1.0, 0.0
    check_rows(c, _run(ops, c, kernel))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_of_one_and_rows_of_zeros(ops, kernel, fmt, D):  # noqa: F811
    """Every scale is 1: some rows are zeros, the others are not."""
    c = _case(ops, kernel, fmt, "f16", 1, 4, D, 16, [5 if kernel == "few" else 40], [300], seed=47)
    _scales(c, 1, lambda s: np.ones_like(s))
    rng = np.random.default_rng(5)
    rows = rng.random(c.scale[1].shape) < 0.4
    if fmt == U4:
        rows_z = rng.random(c.scale[1].shape) < 0.5                      # a zero-point of 0 leaves codes that are not
        c.zero[1] = np.where(rows | rows_z, 0.0, c.zero[1]).astype(np.float32)
        live = c.cache.v_scales[..., 0].cpu().numpy() == 1.0
        z = c.cache.v_scales[..., 1].cpu().numpy()
        c.cache.v_scales[..., 1] = torch.from_numpy(np.where(live, c.zero[1], z).astype(np.float16)).cuda()
    c.code[1] = np.where(rows[..., None], 0, c.code[1]).astype(c.code[1].dtype)
    code = c.cache.v.cpu().numpy()
    code[rows] = 0
    c.cache.v.copy_(torch.from_numpy(code))
    check_rows(c, _run(ops, c, kernel))
