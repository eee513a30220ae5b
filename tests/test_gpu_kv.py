"""The quantized KV cache and the attention over it against the plain binary64 reference (GPU).

Codes, scales and read-back values are exact.  Attention outputs are held to
a bound counted from the roundings, element by element:

* the output's own rounding, u_out |y| (2^-8 BF16, 2^-11 FP16);
* each softmax weight's rounding to FP16, 2^-11 relative, so 2^-11 mean|v|
  under the weights, and 2^-24 of the largest |v| for each weight that falls
  below FP16's normal range (at most the visible positions);
* binary32 scores: D products and sums, the two scales and the base-2 form of
  the exponent, (D + 16) 2^-24 of the largest sum |q k| scale, once in the
  weights and once in their sum, and (positions + 16) 2^-24 for the sums and
  rescalings over positions; 4-bit zero-points and 8-bit offsets are taken off
  before the products.
"""
import numpy as np
import pytest
import torch

import kv_ref as ref
from kv_ref import FP8, I8, U4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FORMATS = [I8, FP8, U4]


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_gemm_w4_amd import ops as _ops
    _ops.lib()
    return _ops


def _np(t):
    return t.detach().float().cpu().numpy()


def _records(scale, zero, fmt):
    return np.stack((scale, zero), -1).astype(np.float16) if fmt == U4 else scale.astype(np.float32)


# ------------------------------------------------------------------ cache ----

def _rows(T, H, D, dtype, seed, wide=False):
    """Keys and values as strided views of one buffer."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 2, H, D, generator=g)
    if T > 6:
        x[1] *= 1e-6
        x[2] = 0.0
        x[3, :, :, 5:] = 0.0
        x[4] = x[4].abs() + 1.0
        x[5] = -x[5].abs() - 1.0
        if wide:
            x[6] *= 1e30
    x = x.to(DT[dtype]).cuda()
    return x[:, 0], x[:, 1]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,H,D,page,T", [("bf16", 8, 128, 16, 33), ("f16", 3, 64, 32, 100), ("f32", 1, 256, 128, 7),
                                             ("bf16", 5, 256, 64, 1), ("f32", 2, 128, 1024, 517)])
def test_write_and_read_back(ops, fmt, dtype, H, D, page, T):
    pages = T // page + 3
    c = ops.kv_cache(pages, page, H, D, fmt)
    k, v = _rows(T, H, D, dtype, seed=T, wide=dtype != "f16")
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(pages * page, generator=g)[:T]
    skip = torch.zeros(T, dtype=torch.bool)
    if T > 20:
        slots[7], slots[11], slots[12] = -1, pages * page, 1 << 40
        skip[[7, 11, 12]] = True
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x5A)
    before = c.k.clone()
    ops.kv_cache_write(k, v, c, slots.cuda())
    out = {n: ops.kv_cache_read(c, slots.cuda(), DT[n]) for n in DT}
    torch.cuda.synchronize()
    keep = np.flatnonzero(~skip.numpy())
    s = slots.numpy()[keep]
    for n, x, codes, rec in ((0, k, c.k, c.k_scales), (1, v, c.v, c.v_scales)):
        code, scale, zero = ref.quantize(_np(x)[keep], fmt)
        got = codes.cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * page, H, -1)[s]
        assert np.array_equal(got, ref.pack_u4(code) if fmt == U4 else code)
        r = rec.cpu().numpy()
        r = r.transpose(0, 2, 1, *range(3, r.ndim)).reshape(pages * page, H, *r.shape[3:])[s]
        assert np.array_equal(r, _records(scale, zero, fmt))
        exact = ref.values(code, scale, zero, fmt).astype(np.float32)      # one binary32 product
        for dt in DT:
            assert torch.equal(out[dt][n].cpu()[keep], torch.from_numpy(exact).to(DT[dt])), dt
            assert not out[dt][n].cpu()[skip].any()
    # nothing but the slots' rows was written
    rest = np.setdiff1d(np.arange(pages * page), s)
    flat = lambda t: t.view(torch.uint8).cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * page, H, -1)[rest]  # noqa: E731
    assert np.array_equal(flat(c.k), flat(before))


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_that_are_not_finite_read_back_as_nan(ops, fmt):
    k, v = (x.clone() for x in _rows(8, 2, 64, "bf16", 3))
    k[0, 0, 9], k[1, 1, 63], v[2, 0, 0], v[3, 1, 31] = float("nan"), float("inf"), -float("inf"), float("nan")
    c = ops.kv_cache(1, 16, 2, 64, fmt)
    slots = torch.arange(8).cuda()
    ops.kv_cache_write(k, v, c, slots)
    kr, vr = ops.kv_cache_read(c, slots)
    for got, x in ((kr, k), (vr, v)):
        bad = ~x.isfinite().all(-1, keepdim=True).expand_as(x)
        assert torch.equal(got.isnan(), bad) and bad.any()
    assert c.k.view(torch.uint8)[0, 0, 0].max() == 0


def test_nothing_to_write_or_read(ops):
    c = ops.kv_cache(1, 16, 1, 64, I8)
    e = torch.empty(0, 1, 64, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    ops.kv_cache_write(e, e, c, s)
    k, v = ops.kv_cache_read(c, s)
    assert k.shape == v.shape == (0, 1, 64)


def test_write_refusals(ops):
    c = ops.kv_cache(2, 16, 2, 64, I8)
    s = torch.arange(3).cuda()
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="must be"):
        ops.kv_cache_write(x[:2], x, c, s)
    with pytest.raises(ValueError, match="int64"):
        ops.kv_cache_write(x, x, c, s.int())
    with pytest.raises(ValueError, match="one type"):
        ops.kv_cache_write(x, x.float(), c, s)
    with pytest.raises(ValueError, match="contiguous"):
        ops.kv_cache_write(torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")[:, :, ::2], x, c, s)
    with pytest.raises(ops.BitGemmError, match="strides"):
        y = torch.zeros(3, 2, 67, dtype=torch.bfloat16, device="cuda")[:, :, :64]
        ops.kv_cache_write(y, y, c, s)
    with pytest.raises(ValueError, match="device"):
        ops.kv_cache_write(x.cpu(), x.cpu(), c, s)


# -------------------------------------------------------------- attention ----

class Case:
    """A batch over a cache whose unseen slots hold what attention must not read into."""

    def __init__(self, ops, fmt, dtype, heads, group, D, page, q_lens, kv_lens, seed=0, window=0, sinks=0, tree=False,
                 gone=0.0, loud=1.0, small_v=False):
        rng = np.random.default_rng(seed)
        self.fmt, self.dtype, self.heads, self.group, self.D, self.page = fmt, dtype, heads, group, D, page
        self.q_lens, self.kv_lens, self.window, self.sinks = q_lens, kv_lens, window, sinks
        B, T = len(q_lens), sum(q_lens)
        per = max(1, -(-max([*kv_lens, 1]) // page))
        pages = B * per + 2
        self.code, self.scale, self.zero, tens = [], [], [], []
        for n in range(2):
            x = rng.standard_normal((pages, heads, page, D)).astype(np.float32)
            if n == 0:
                x = x * np.exp(0.5 * rng.standard_normal((1, heads, 1, D))) + 0.5 * rng.standard_normal((1, heads, 1, D))
            else:
                x = x * np.exp(rng.standard_normal((pages, heads, page, 1)))
                if small_v:
                    x = x * 1e-20
            code, s, z = ref.quantize(x.astype(np.float32), fmt)
            self.code.append(code), self.scale.append(s), self.zero.append(z)
        order = rng.permutation(pages - 1)[:B * per].reshape(B, per) + 1
        self.table = order.astype(np.int32)
        # garbage where no query sees: unwritten slots, unowned pages, page 0
        owned = np.zeros((pages, page), bool)
        for b in range(B):
            for j in range(kv_lens[b]):
                owned[order[b, j // page], j % page] = True
        for b in range(B):
            first = -(-kv_lens[b] // page)
            self.table[b, first:] = rng.choice([-1, pages, 2 ** 31 - 1, 0], per - first)
        if gone:      # pages that are not there, anywhere in the sequences
            drop = rng.random(self.table.shape) < gone
            self.table[drop] = -1
        dead = ~owned[:, None, :].repeat(heads, 1)
        for n in range(2):
            code = self.code[n].copy()
            if fmt == FP8:
                code[dead] = rng.choice([0x7F, 0xFF, 0x7E], (dead.sum(), D))
            rec = _records(self.scale[n], self.zero[n], fmt)
            rec[dead] = rng.choice([np.nan, np.inf, -np.inf, 0.0, 6e4 if fmt == U4 else 3e38], rec[dead].shape)
            tens.append(torch.from_numpy(ref.pack_u4(code) if fmt == U4 else code).cuda())
            tens.append(torch.from_numpy(rec).cuda())
        self.cache = ops.KVCache(tens[0], tens[2], tens[1], tens[3], fmt)
        # queries inside a wider row
        wide = torch.from_numpy(rng.standard_normal((T, (group + 2) * heads * D)).astype(np.float32) * loud).to(DT[dtype]).cuda()
        self.q = wide[:, :group * heads * D].view(T, group * heads, D)
        self.cu = torch.tensor([0, *np.cumsum(q_lens)], dtype=torch.int32).cuda()
        self.lens = torch.tensor(kv_lens, dtype=torch.int32).cuda()
        self.bt = torch.from_numpy(self.table).cuda()
        self.max_q, self.max_kv = max(q_lens), max(kv_lens)
        self.bits = self.tree = None
        if tree:
            self.bits = []
            for n in q_lens:
                rows = []
                for i in range(n):
                    up = rows[rng.integers(max(0, i - 5), i)] if i and rng.random() < 0.9 else 0
                    rows.append(up | 1 << i)
                self.bits.append(rows)
            words = (self.max_q + 63) // 64
            flat = [[np.uint64(r >> 64 * w & (1 << 64) - 1) for w in range(words)] for rows in self.bits for r in rows]
            self.tree = torch.from_numpy(np.array(flat, np.uint64).view(np.int64)).cuda()

    def run(self, ops, **kw):
        kw.setdefault("max_kv_len", self.max_kv)
        if self.tree is not None:
            return ops.kv_attn_tree(self.q, self.cache, self.bt, self.lens, self.cu, self.tree, self.max_q, **kw)
        return ops.kv_attn(self.q, self.cache, self.bt, self.lens, self.cu, self.max_q, window=self.window, sinks=self.sinks, **kw)

    def check(self, got, lse=None, only=None, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        u_out = 2.0 ** (-8 if self.dtype == "bf16" else -11)
        got, q = got.double().cpu().numpy(), self.q.double().cpu().numpy()
        first = 0
        for b, (n, length) in enumerate(zip(self.q_lens, self.kv_lens)):
            if only is not None and b not in only:
                first += n
                continue
            ids = self.table[b, :-(-length // self.page)]
            there = (ids >= 0) & (ids < self.cache.pages)
            held = there.repeat(self.page)[:length]
            see = ref.visible(n, length, held, self.window, self.sinks, self.bits[b] if self.bits else None)
            safe = np.where(there, ids, 0)
            for h in range(self.heads):
                k, v = (ref.values(self.code[x][safe, h], self.scale[x][safe, h], self.zero[x][safe, h], self.fmt)
                        .reshape(-1, self.D)[:length] for x in range(2))
                top_v = np.abs(v[see.any(0)]).max(initial=0.0)
                for g in range(self.group):
                    hq = h * self.group + g
                    y, ls, mean, top = ref.attend(q[first:first + n, hq], k, v, see, scale)
                    count = see.sum(1)
                    rel = (2 * (self.D + 16) * top + count + 16) * 2.0 ** -24
                    tol = (u_out * np.abs(y) + (1 + u_out) * ((2.0 ** -11 + rel)[:, None] * mean + (count * 2.0 ** -24 * top_v)[:, None])
                           + (2.0 ** -25 if self.dtype == "f16" else 2.0 ** -133))
                    x = got[first:first + n, hq]
                    bad = ~(np.abs(x - y) <= tol)
                    assert not bad.any(), (b, h, g, np.argwhere(bad)[:4], x[bad][:4], y[bad][:4], np.broadcast_to(tol, x.shape)[bad][:4])
                    assert not x[count == 0].any()
                    if lse is not None:
                        z = lse[first:first + n, hq].double().cpu().numpy()
                        some = count > 0
                        assert (z[~some] == -np.inf).all()
                        off = np.abs(z[some] - ls[some])
                        lim = rel[some] + 2.0 ** -22 * (np.abs(ls[some]) + 1)
                        assert (off <= lim).all(), (off.max(), lim.min())
            first += n


SHAPES = [  # heads, group, D, page
    (2, 4, 128, 16), (1, 1, 64, 32), (2, 7, 64, 128), (1, 16, 256, 64), (3, 3, 128, 32), (1, 20, 128, 16), (8, 2, 256, 16),
]
DECODES = [[1], [31, 32, 33], [0, 1, 500, 64], [1031], [16, 17, 2050]]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens", DECODES)
def test_decode(ops, fmt, dtype, shape, lens):
    heads, group, D, page = shape
    c = Case(ops, fmt, dtype, heads, group, D, page, [1] * len(lens), lens, seed=len(lens))
    lse = torch.empty(len(lens), heads * group, device="cuda")
    got = c.run(ops, lse=lse)
    c.check(got, lse)
    # one query per sequence needs no offsets, and the bound on lengths only sizes the work
    again = ops.kv_attn(c.q, c.cache, c.bt, c.lens)
    c.check(again)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("q_lens,kv_lens", [([5, 1, 3], [70, 1, 3]), ([37], [37]), ([1, 70, 0, 130], [40, 300, 9, 131]), ([300], [555])])
def test_chunks(ops, fmt, dtype, shape, q_lens, kv_lens):
    heads, group, D, page = shape
    c = Case(ops, fmt, dtype, heads, group, D, page, q_lens, kv_lens, seed=sum(q_lens))
    lse = torch.empty(sum(q_lens), heads * group, device="cuda")
    c.check(c.run(ops, lse=lse), lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (33, 1), (64, 64), (100, 200), (5000, 4), (16, 17)])
@pytest.mark.parametrize("q_lens,kv_lens,shape", [([1] * 4, [1, 40, 333, 1500], (2, 4, 128, 16)), ([9, 150, 2], [30, 400, 777], (1, 3, 64, 32)),
                                                  ([130], [900], (2, 5, 128, 64)), ([20, 4], [90, 600], (1, 2, 256, 16))])
def test_windows_and_sinks(ops, fmt, window, sinks, q_lens, kv_lens, shape):
    c = Case(ops, fmt, "bf16", *shape, q_lens, kv_lens, seed=window, window=window, sinks=sinks)
    lse = torch.empty(sum(q_lens), shape[0] * shape[1], device="cuda")
    c.check(c.run(ops, lse=lse), lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_lens,kv_lens,shape", [([1], [1], (1, 1, 64, 16)), ([13], [100], (2, 4, 128, 16)), ([64, 3, 30], [64, 70, 999], (1, 4, 64, 32)),
                                                  ([65, 130], [300, 130], (1, 2, 128, 64)), ([24, 1], [61, 1200], (2, 2, 256, 128)),
                                                  ([7, 8], [2000, 8], (2, 8, 128, 16)), ([200], [263], (1, 7, 128, 16))])
def test_trees(ops, fmt, dtype, q_lens, kv_lens, shape):
    c = Case(ops, fmt, dtype, *shape, q_lens, kv_lens, seed=sum(q_lens), tree=True)
    lse = torch.empty(sum(q_lens), shape[0] * shape[1], device="cuda")
    c.check(c.run(ops, lse=lse), lse)


def test_a_chain_of_drafts_is_causal_attention(ops):
    c = Case(ops, FP8, "bf16", 2, 4, 128, 16, [40, 9], [200, 41], seed=5)
    rows = [(1 << i + 1) - 1 for n in c.q_lens for i in range(n)]
    tree = torch.from_numpy(np.array([[r & (1 << 64) - 1] for r in rows], np.uint64).view(np.int64)).cuda()
    got = ops.kv_attn_tree(c.q, c.cache, c.bt, c.lens, c.cu, tree, 40, max_kv_len=200)
    c.check(got)                             # c holds no tree: the reference is the causal one


def test_tree_bits_past_the_words_are_not_seen(ops):
    c = Case(ops, I8, "bf16", 1, 2, 64, 16, [100], [150], seed=6, tree=True)
    c.tree = c.tree[:, :1].contiguous()
    c.bits = [[r & (1 << 64) - 1 for r in c.bits[0]]]
    c.check(c.run(ops))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens,kind", [([1, 1, 1], [300, 40, 1000], "causal"), ([60, 200], [100, 500], "causal"), ([30], [700], "tree")])
def test_pages_that_are_not_there(ops, fmt, q_lens, kv_lens, kind):
    c = Case(ops, fmt, "f16", 2, 4, 128, 16, q_lens, kv_lens, seed=7, gone=0.5, tree=kind == "tree")
    lse = torch.empty(sum(q_lens), 8, device="cuda")
    c.check(c.run(ops, lse=lse), lse)
    c.table[:] = -1
    c.bt.fill_(-1)
    assert not c.run(ops).any()


def test_more_queries_than_positions(ops):
    """The first queries stand before the sequence and see nothing."""
    for q_lens, kv_lens in (([5, 4, 2], [2, 0, 1]), ([150], [20])):
        c = Case(ops, I8, "bf16", 2, 4, 64, 16, q_lens, kv_lens, seed=8)
        lse = torch.empty(sum(q_lens), 8, device="cuda")
        c.check(c.run(ops, lse=lse), lse)
    c = Case(ops, FP8, "bf16", 1, 2, 128, 32, [9], [4], seed=8, tree=True)
    c.check(c.run(ops))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [700]), ([150], [700])])
def test_peaked_rows_and_small_values(ops, fmt, q_lens, kv_lens):
    c = Case(ops, fmt, "bf16", 1, 4, 128, 16, q_lens, kv_lens, seed=9, loud=30.0)
    c.check(c.run(ops))
    if fmt != U4:      # a 4-bit scale is at least 2^-24
        c = Case(ops, fmt, "bf16", 1, 4, 128, 16, q_lens, kv_lens, seed=9, small_v=True)
        c.check(c.run(ops))
    c = Case(ops, fmt, "f16", 1, 4, 128, 16, q_lens, kv_lens, seed=9, loud=1e-4)
    c.check(c.run(ops, scale=0.5), scale=0.5)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 70]), ([20, 200], [100, 400])])
@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_stays_with_the_rows_that_see_it(ops, fmt, q_lens, kv_lens):
    c = Case(ops, fmt, "bf16", 1, 4, 64, 16, q_lens, kv_lens, seed=10, window=50, sinks=2)
    q, clean = c.q.clone(), c.run(ops)
    # a query of infinities and one of NaN, and a value row that is NaN inside the first sequence's cache
    c.q[0, 1] = float("inf")
    c.q[0, 2, 5] = float("nan")
    j = kv_lens[1] - 1                       # the last position of the second sequence: its last query alone sees it
    c.cache.v_scales[int(c.table[1, j // 16]), 0, j % 16] = float("nan")
    got = c.run(ops)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 1], bad[0, 2], bad[-1] = True, True, True
    assert torch.equal(got.isnan(), bad)
    c.q = q
    c.check(torch.where(bad, clean, got))


def test_lse_merges_two_halves(ops):
    """Attention over pages split into two calls joins to the whole by lse."""
    c = Case(ops, I8, "f16", 2, 4, 128, 16, [1], [640], seed=11)
    parts = []
    for half in (0, 1):
        t = c.bt.clone()
        t[:, 20 * half:20 * half + 20] = -1
        lse = torch.empty(1, 8, device="cuda")
        parts.append((ops.kv_attn(c.q, c.cache, t, c.lens, lse=lse).double(), lse.double()))
    top = torch.maximum(parts[0][1], parts[1][1])
    w = [(p[1] - top).exp() for p in parts]
    c.check(sum(a[..., None] * p[0] for a, p in zip(w, parts)) / sum(w)[..., None])


def test_a_bound_on_lengths_that_is_too_small_costs_only_speed(ops):
    c = Case(ops, I8, "bf16", 1, 4, 128, 16, [1, 1], [3000, 1200], seed=12)
    c.check(c.run(ops, max_kv_len=1))
    c = Case(ops, I8, "bf16", 1, 4, 128, 16, [140], [2100], seed=12)
    c.check(c.run(ops, max_kv_len=40))


def test_rows_no_sequence_owns_are_left_alone(ops):
    c = Case(ops, FP8, "bf16", 2, 2, 64, 16, [3, 4], [20, 30], seed=13)
    out = torch.full_like(c.q, 7.0).contiguous()
    cu = torch.tensor([1, 4, 6], dtype=torch.int32).cuda()
    ops.kv_attn(c.q, c.cache, c.bt, c.lens, cu, 4, out=out)
    assert (out[0] == 7.0).all() and (out[6] == 7.0).all() and not (out[1:6] == 7.0).any()
    # offsets outside the tokens are clamped
    cu = torch.tensor([-5, 3, 1 << 30], dtype=torch.int32).cuda()
    ops.kv_attn(c.q, c.cache, c.bt, c.lens, cu, 4, out=out)


def test_offsets_past_32_bits(ops):
    """A cache whose code offsets pass 2^32: its last pages and its first."""
    pages, page, D = 36864, 1024, 128
    c = Case(ops, I8, "bf16", 1, 4, D, 16, [1, 40], [500, 900], seed=14)
    big = ops.kv_cache(pages, page, 1, D, I8)
    assert big.k.numel() > 1 << 32
    # sequence 0 in the last page, sequence 1 in page 0; the same codes
    table = torch.tensor([[pages - 1], [0]], dtype=torch.int32).cuda()
    for b, to in ((0, pages - 1), (1, 0)):
        n = c.kv_lens[b]
        ids = torch.from_numpy(c.table[b, :-(-n // 16)].astype(np.int64)).cuda()
        for x in ("k", "v"):
            getattr(big, x)[to, 0, :n] = getattr(c.cache, x)[ids, 0].reshape(-1, D)[:n]
            getattr(big, x + "_scales")[to, 0, :n] = getattr(c.cache, x + "_scales")[ids, 0].reshape(-1)[:n]
    got = ops.kv_attn(c.q, big, table, c.lens, c.cu, 40)
    c.check(got)
    slots = torch.tensor([(pages - 1) * page, pages * page - 1], dtype=torch.int64).cuda()
    x = torch.randn(2, 1, D, device="cuda")
    ops.kv_cache_write(x, x, big, slots)
    code, s, _ = ref.quantize(_np(x), I8)
    assert np.array_equal(big.k[-1, 0, [0, -1]].cpu().numpy(), code[:, 0])
    k, _ = ops.kv_cache_read(big, slots, torch.float32)
    assert np.array_equal(_np(k), ref.values(code, s, 0 * s, I8).astype(np.float32))


def test_wide_strides(ops):
    """Queries whose rows lie far apart, heads apart too."""
    c = Case(ops, FP8, "bf16", 2, 4, 64, 16, [3, 50], [40, 90], seed=15)
    wide = torch.zeros(53, 8, 3, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1] = c.q
    want = c.run(ops)
    c.q = wide[:, :, 1]
    assert torch.equal(c.run(ops), want)


CALLS = [([1, 1, 1], [900, 1, 3000], False), ([40, 200], [400, 1200], False), ([30, 64], [500, 900], True)]


@pytest.mark.parametrize("q_lens,kv_lens,tree", CALLS)
def test_another_stream(ops, q_lens, kv_lens, tree):
    c = Case(ops, I8, "bf16", 2, 4, 128, 16, q_lens, kv_lens, seed=16, tree=tree)
    want = c.run(ops)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(ops, stream=s)
    other = c.run(ops)                       # overlaps the call on s: workspaces are one per stream
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)


@pytest.mark.parametrize("q_lens,kv_lens,tree", CALLS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_graph_replays(ops, fmt, q_lens, kv_lens, tree):
    """Write, attend and read back captured once; replays follow the lengths, pages and rows in memory."""
    c = Case(ops, fmt, "bf16", 2, 4, 128, 16, q_lens, kv_lens, seed=17, tree=tree)
    T = sum(q_lens)
    k = torch.randn(T, 2, 128, device="cuda").bfloat16()
    v = torch.randn(T, 2, 128, device="cuda").bfloat16()
    slots = torch.tensor([int(c.table[b, j // 16]) * 16 + j % 16 for b, n in enumerate(q_lens)
                          for j in range(kv_lens[b] - n, kv_lens[b])]).cuda()
    out = torch.empty_like(c.q).contiguous()

    def step():
        ops.kv_cache_write(k, v, c.cache, slots)
        c.run(ops, out=out)
        return ops.kv_cache_read(c.cache, slots)

    def eager(lens):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        r = step()
        torch.cuda.synchronize()
        return [x.clone() for x in (out, *r)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        read = step()
    other = Case(ops, fmt, "f16", 1, 8, 64, 32, [1], [5000], seed=18)
    for rep, lens in enumerate((kv_lens, [max(1, n - 3) for n in kv_lens], [max(1, n // 2) for n in kv_lens])):
        k.normal_()
        want = eager(lens)
        out.fill_(0)
        other.run(ops)                       # eager work between the replays, through the cached workspace
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, *read), want):
            assert torch.equal(a, b), rep


def test_repeated_calls_agree_bit_for_bit(ops):
    for q_lens, kv_lens, tree in CALLS:
        c = Case(ops, FP8, "bf16", 2, 4, 128, 16, q_lens, kv_lens, seed=19, tree=tree)
        want = c.run(ops)
        for _ in range(3):
            assert torch.equal(c.run(ops), want)


def test_attention_refusals(ops):
    c = Case(ops, I8, "bf16", 2, 2, 64, 16, [3], [20], seed=20)
    with pytest.raises(ValueError, match="q must be"):
        ops.kv_attn(c.q[:, :, :32], c.cache, c.bt, c.lens, c.cu, 3)
    with pytest.raises(ValueError, match="float16/bfloat16"):
        ops.kv_attn(c.q.float(), c.cache, c.bt, c.lens, c.cu, 3)
    with pytest.raises(ValueError, match="block_table"):
        ops.kv_attn(c.q, c.cache, c.bt.long(), c.lens, c.cu, 3)
    with pytest.raises(ValueError, match="kv_lens"):
        ops.kv_attn(c.q, c.cache, c.bt, c.lens.repeat(2), c.cu, 3)
    with pytest.raises(ValueError, match="cu_q"):
        ops.kv_attn(c.q, c.cache, c.bt, c.lens, c.cu[:1], 3)
    with pytest.raises(ValueError, match="out must be"):
        ops.kv_attn(c.q, c.cache, c.bt, c.lens, c.cu, 3, out=torch.empty(3, 4, 64, device="cuda"))
    with pytest.raises(ValueError, match="lse"):
        ops.kv_attn(c.q, c.cache, c.bt, c.lens, c.cu, 3, lse=torch.empty(3, device="cuda"))
    with pytest.raises(ops.BitGemmError, match="multiple of kv_heads"):
        ops.kv_attn(c.q[:, :3], c.cache, c.bt, c.lens, c.cu, 3)
    with pytest.raises(ops.BitGemmError, match="window"):
        ops.kv_attn(c.q, c.cache, c.bt, c.lens, c.cu, 3, window=-1)
    with pytest.raises(ops.BitGemmError, match="one query"):
        ops.kv_attn(c.q, c.cache, c.bt, c.lens)
    with pytest.raises(ops.BitGemmError, match="scale"):
        ops.kv_attn(c.q, c.cache, c.bt, c.lens, c.cu, 3, scale=0.0)
    with pytest.raises(ValueError, match="tree must be"):
        ops.kv_attn_tree(c.q, c.cache, c.bt, c.lens, c.cu, torch.zeros(2, 1, dtype=torch.int64).cuda(), 3)
    with pytest.raises(ValueError, match="device"):
        ops.kv_attn(c.q, c.cache, c.bt.cpu(), c.lens, c.cu, 3)
    big = Case(ops, I8, "bf16", 1, 1, 64, 16, [1], [9000], seed=20)
    if ops.kv_attn_workspace_bytes((1, 1), big.cache, 1, big.bt.shape[1]):
        with pytest.raises(ops.BitGemmError, match="workspace"):
            big.run(ops, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
