"""Attention over the quantized cache with capped scores, distance biases and prefixes, against binary64 (GPU).

The bound of tests/test_gpu_kv.py, with the score's error counted for each position: (D + 16) 2^-24 of the largest sum |q k| scale
(tanh does not stretch it), 2^-21 of a cap up to 256 (tanh as 1 - 2 / (1 + 2^x): the power's and the reciprocal's ulp, two
roundings, 3.5 2^-23) or of the capped score beyond (polynomials within 2^-22.2, their products' roundings), and 2^-22 of the bias (its slope in base 2, the product, the sum; distances
here are exact).  An error e of a score moves its weight by e (1 + e), and the sum by its mean.
"""
import numpy as np
import pytest
import torch

import kv_ref as ref
from kv_ref import FP8, I8, U4
from test_gpu_kv import Case, ops  # noqa: F401

pytestmark = pytest.mark.gpu
FORMATS = [I8, FP8, U4]


def attend(q, k, v, see, at, scale, cap, slope):
    """One sequence and head -> out, lse, mean |v|, and the weighted errors of scores: of |v| and alone."""
    n, D = q.shape
    out, lse = np.zeros_like(q), np.full(n, -np.inf)
    mean, moved, total = np.zeros_like(q), np.zeros_like(q), np.zeros(n)
    for i in range(n):
        j = np.flatnonzero(see[i])
        if not j.size:
            continue
        s = k[j] @ q[i] * scale
        top = (np.abs(k[j]) @ np.abs(q[i])).max() * scale
        e = (D + 16) * 2.0 ** -24 * np.full(j.size, top)
        if cap:
            s = cap * np.tanh(s / cap)
            e = e + 2.0 ** -21 * (cap if cap <= 256 else np.abs(s))
        bias = slope * np.abs(at[i] - j)
        s = s - bias
        e = e + 2.0 ** -22 * np.abs(bias) + 2.0 ** -23 * np.abs(s)
        e = e * (1 + e)
        m = s.max()
        p = np.exp(s - m)
        l = p.sum()
        p = p / l
        out[i], lse[i], mean[i] = p @ v[j], m + np.log(l), p @ np.abs(v[j])
        moved[i], total[i] = (p * e) @ np.abs(v[j]), p @ e
    return out, lse, mean, moved, total


class Scored:
    """A case of the plain attention with other scores."""

    def __init__(self, ops, *args, cap=0.0, slopes=None, prefix=None, **kw):  # noqa: F811
        self.c = Case(ops, *args, **kw)
        heads = self.c.heads * self.c.group
        self.cap, self.prefix = cap, prefix
        self.slopes = None if slopes is None else np.resize(np.asarray(slopes, np.float32), heads)
        self.how = dict(softcap=cap)
        if slopes is not None:
            self.how["slopes"] = torch.from_numpy(self.slopes).cuda()
        if prefix is not None:
            self.how["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32).cuda()

    def run(self, ops, **kw):  # noqa: F811
        return self.c.run(ops, **self.how, **kw)

    def check(self, got, lse=None, only=None):
        c = self.c
        u_out = 2.0 ** (-8 if c.dtype == "bf16" else -11)
        got, q = got.double().cpu().numpy(), c.q.double().cpu().numpy()
        first = 0
        for b, (n, length) in enumerate(zip(c.q_lens, c.kv_lens)):
            ids = c.table[b, :-(-length // c.page)]
            there = (ids >= 0) & (ids < c.cache.pages)
            held = there.repeat(c.page)[:length]
            at = np.arange(length - n, length)
            if c.bits:
                see = ref.visible(n, length, held, tree=c.bits[b])
            else:
                j = np.arange(length)
                see = j <= at[:, None]
                if self.prefix is not None:
                    see |= j < self.prefix[b]
                if c.window:
                    see &= (j > at[:, None] - c.window) | (j < c.sinks)
                see = see & held
            safe = np.where(there, ids, 0)
            rows = range(n) if only is None else [i for i in only if i < n]
            for h in range(c.heads if n else 0):
                k, v = (ref.values(c.code[x][safe, h], c.scale[x][safe, h], c.zero[x][safe, h], c.fmt).reshape(-1, c.D)[:length] for x in range(2))
                top_v = np.abs(v[see.any(0)]).max(initial=0.0)
                for g in range(c.group):
                    hq = h * c.group + g
                    pick = list(rows)
                    y, ls, mean, moved, total = attend(q[first:first + n, hq][pick], k, v, see[pick], at[pick], c.D ** -0.5, self.cap,
                                                       0.0 if self.slopes is None else float(self.slopes[hq]))
                    count = see[pick].sum(1)
                    sums = (count + 16) * 2.0 ** -24
                    tol = (u_out * np.abs(y) + (1 + u_out) * ((2.0 ** -11 + sums + total)[:, None] * mean + moved + (count * 2.0 ** -24 * top_v)[:, None])
                           + (2.0 ** -25 if c.dtype == "f16" else 2.0 ** -133))
                    x = got[first:first + n, hq][pick]
                    bad = ~(np.abs(x - y) <= tol)
                    assert not bad.any(), (b, h, g, np.argwhere(bad)[:4], x[bad][:4], y[bad][:4], tol[bad][:4])
                    assert not x[count == 0].any()
                    if lse is not None:
                        z = lse[first:first + n, hq].double().cpu().numpy()[pick]
                        some = count > 0
                        assert (z[~some] == -np.inf).all()
                        assert (np.abs(z[some] - ls[some]) <= total[some] + sums[some] + 2.0 ** -22 * (np.abs(ls[some]) + 1)).all()
            first += n


def both(ops, *args, only=None, **kw):  # noqa: F811
    s = Scored(ops, *args, **kw)
    lse = torch.empty(s.c.q.shape[0], s.c.q.shape[1], device="cuda")
    s.check(s.run(ops, lse=lse), lse, only)
    return s


SHAPES = [(2, 4, 128, 16), (1, 7, 64, 128), (1, 3, 256, 64)]           # heads, group, D, page
HOW = [dict(cap=50.0), dict(cap=3.0), dict(cap=0.01), dict(cap=1e6), dict(slopes=[0.5, 0.01, 0.0, 2.0 ** -8]), dict(slopes=[-0.03, 4.0]),
       dict(cap=20.0, slopes=[0.1, 0.002])]
IDS = lambda x: "_".join(f"{k}{v}" for k, v in x.items()) if isinstance(x, dict) else None  # noqa: E731


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("how", HOW, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_decode(ops, fmt, how, shape):  # noqa: F811
    for lens in ([1], [0, 1, 500, 64], [16, 17, 2050]):
        both(ops, fmt, "bf16" if shape[2] != 64 else "f16", *shape, [1] * len(lens), lens, seed=len(lens), loud=4.0, **how)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("how", HOW + [dict(prefix="some"), dict(prefix="some", cap=30.0, slopes=[0.3, 0.01])], ids=IDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_chunks(ops, fmt, how, shape):  # noqa: F811
    for q_lens, kv_lens, prefix in (([5, 1, 3], [70, 1, 3], [66, 5, 0]), ([1, 70, 0, 90], [40, 300, 9, 91], [40, 280, 9, 33])):
        h = {**how, "prefix": prefix} if how.get("prefix") else how
        both(ops, fmt, "f16" if shape[2] == 128 else "bf16", *shape, q_lens, kv_lens, seed=sum(q_lens), loud=3.0, **h)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 1), (100, 200), (5000, 4)])
@pytest.mark.parametrize("q_lens,kv_lens,shape", [([1] * 4, [1, 40, 333, 1500], (2, 4, 128, 16)), ([9, 100, 2], [30, 400, 777], (1, 3, 64, 32))])
def test_windows(ops, fmt, window, sinks, q_lens, kv_lens, shape):  # noqa: F811
    both(ops, fmt, "bf16", *shape, q_lens, kv_lens, seed=window, window=window, sinks=sinks, cap=10.0, slopes=[0.05, 0.3])
    both(ops, fmt, "bf16", *shape, q_lens, kv_lens, seed=window, window=window, sinks=sinks, prefix=[n - 1 if i % 2 else n // 2 for i, n in enumerate(kv_lens)])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("prefix", [[-5, 0, 10 ** 9], [2 ** 31 - 1, -2 ** 31, 100], [64, 63, 65], [400, 700, 1]])
def test_prefixes_at_and_past_the_ends(ops, fmt, prefix):  # noqa: F811
    s = both(ops, fmt, "bf16", 2, 3, 128, 16, [64, 3, 100], [400, 3, 130], seed=7, prefix=prefix)
    if prefix == [-5, 0, 10 ** 9]:
        # without a prefix it is the causal form; its first query then sees the last position, too
        only = s.c.run(ops)
        got = s.run(ops)
        assert (got[:67].float() - only[:67].float()).abs().max() <= 2.0 ** -6 * only.float().abs().max()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cap", [30.0, 2.0])
def test_trees(ops, fmt, cap):  # noqa: F811
    for q_lens, kv_lens, shape in (([13], [100], (2, 4, 128, 16)), ([64, 3, 30], [64, 70, 999], (1, 4, 64, 32)), ([70, 1], [1700, 5], (1, 3, 256, 16))):
        both(ops, fmt, "bf16", *shape, q_lens, kv_lens, seed=3, tree=True, loud=3.0, cap=cap)


MANY = [  # heads, group, D, page, q_lens, kv_lens, waves
    (1, 4, 128, 16, [300, 20], [900, 64], 8),
    (1, 1, 64, 32, [500], [1100], 8),
    (1, 2, 256, 64, [200, 7], [600, 300], 4),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("how", [dict(cap=30.0), dict(cap=2.0), dict(slopes=[0.2, 0.01]), dict(cap=15.0, slopes=[0.2, 0.003], prefix=[700, 40]),
                                 dict(prefix=[1000, 10], window=90, sinks=5), dict(cap=300.0), dict(cap=5e4, slopes=[0.01])], ids=IDS)
@pytest.mark.parametrize("heads,group,D,page,q_lens,kv_lens,waves", MANY)
def test_many_rows(ops, fmt, how, heads, group, D, page, q_lens, kv_lens, waves):  # noqa: F811
    how = {**how, "prefix": how["prefix"][:len(q_lens)]} if "prefix" in how else how
    s = both(ops, fmt, "bf16", heads, group, D, page, q_lens, kv_lens, seed=11, loud=3.0, only=[0, 1, 31, 63, 64, 130, 199, 299, 499], **how)
    assert ops.last_kernel().startswith(("k_kv_attn_many_", "k_kv_attn_few_scored<")) and s.c.fmt == fmt


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,seqs,waves", [(64, 16, 8), (64, 32, 4), (128, 32, 8), (256, 16, 4)])
def test_many_rows_by_name_over_runs_of_positions(ops, fmt, D, seqs, waves):  # noqa: F811
    """Batches that take the many-row kernel, with several runs of positions, missing pages and rows of very different sizes."""
    q_lens, kv_lens = [600] * seqs, [1437 - 3 * i for i in range(seqs)]
    s = Scored(ops, fmt, "bf16", 1, 1, D, 32, q_lens, kv_lens, seed=5, loud=2.0, gone=0.05, cap=25.0, slopes=[0.002],
               prefix=[1400 - 40 * i for i in range(seqs)])
    s.c.q[3] *= 2.0 ** -20
    s.c.q[50] *= 2.0 ** 5
    need = ops.kv_attn_workspace_bytes(s.c.q.shape, s.c.cache, seqs, s.c.bt.shape[1], 600, s.c.max_kv)
    lse = torch.empty(600 * seqs, 1, device="cuda")
    got = s.run(ops, lse=lse, ws=torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"))
    assert ops.last_kernel() == f"k_kv_attn_many_cap_bias<{fmt}, {D}, {waves}>" and need > 0
    s.check(got, lse, only=[0, 3, 50, 77, 300, 599])


@pytest.mark.parametrize("shape", [(1, 4, 128, 64), (4, 5, 64, 32)])
def test_long_decode_with_biases(ops, shape):  # noqa: F811
    both(ops, I8, "bf16", *shape, [1, 1], [40000, 777], seed=9, slopes=[2.0 ** -4, 2.0 ** -9, 0.0, 1.0])
    both(ops, FP8, "f16", *shape, [1, 1], [40000, 777], seed=9, cap=30.0)


def test_nothing_asked_is_the_plain_call(ops):  # noqa: F811
    c = Case(ops, FP8, "bf16", 2, 4, 128, 16, [5, 40], [70, 300], seed=1)
    assert torch.equal(c.run(ops), c.run(ops, softcap=0.0, slopes=None, prefix_lens=None))
    assert ops.last_kernel().startswith("k_kv_attn_few<") or ops.last_kernel().startswith("k_kv_attn_many<")


def test_infinite_and_nan_queries_stay_in_their_rows(ops):  # noqa: F811
    for q_lens, kv_lens in (([1, 1, 1], [50, 60, 70]), ([300], [400])):
        s = Scored(ops, I8, "f16", 1, 4, 128, 16, q_lens, kv_lens, seed=2, cap=10.0, slopes=[0.01])
        want = s.run(ops)
        s.c.q[1, 2, 5] = float("nan")
        got = s.run(ops)
        keep = torch.ones(got.shape[:2], dtype=torch.bool)
        keep[1, 2] = False
        assert torch.equal(got[keep], want[keep]) and torch.isnan(got[1, 2]).all()


def test_captured_and_on_another_stream(ops):  # noqa: F811
    s = Scored(ops, FP8, "bf16", 2, 4, 128, 16, [1, 1, 1], [9000, 40, 700], seed=4, cap=20.0, slopes=[0.01, 0.1], prefix=[3, 0, 700])
    out, side, g = torch.empty_like(s.c.q).contiguous(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.run(ops)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        s.run(ops, out=out)
    for rep in range(4):
        s.how["slopes"].mul_(1.5)
        s.c.q.mul_(0.9)
        torch.cuda.synchronize()
        g.replay()
        want = s.run(ops)
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep
        side.wait_stream(torch.cuda.current_stream())
        got = s.run(ops, stream=side)
        side.synchronize()
        assert torch.equal(got, want)


def test_refusals(ops):  # noqa: F811
    c = Case(ops, I8, "bf16", 2, 4, 128, 16, [5, 40], [70, 300], seed=1)
    for cap in (-1.0, float("nan"), float("inf")):
        with pytest.raises(ops.BitGemmError, match="softcap"):
            c.run(ops, softcap=cap)
    with pytest.raises(ValueError, match="slopes"):
        c.run(ops, slopes=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError, match="slopes"):
        c.run(ops, slopes=torch.zeros(8, device="cuda").double())
    with pytest.raises(ValueError, match="prefix_lens"):
        c.run(ops, prefix_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="one device"):
        c.run(ops, prefix_lens=torch.zeros(2, dtype=torch.int32))
    t = Case(ops, I8, "bf16", 2, 4, 128, 16, [5], [70], seed=1, tree=True)
    with pytest.raises(TypeError):
        t.run(ops, slopes=torch.zeros(8, device="cuda"))


@pytest.mark.parametrize("fmt", FORMATS)
def test_queries_before_the_sequence(ops, fmt):  # noqa: F811
    """More queries than positions: those before the first see the prefix alone, or nothing."""
    both(ops, fmt, "bf16", 2, 4, 128, 16, [9, 70, 3], [4, 20, 0], seed=6, prefix=[2, 0, 5], cap=9.0, slopes=[0.3, 0.02])
    both(ops, fmt, "f16", 1, 6, 64, 16, [300], [130], seed=6, prefix=[50], window=20, sinks=3, slopes=[0.1])
