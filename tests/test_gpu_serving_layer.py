"""Planned steps, normed and rotated heads, the quantized cache and attention with other scores, together as a layer runs them (GPU).

Where two layers do the same arithmetic on the same codes (pages of their own or of a pool, chunks or tokens) what the cache
holds is equal bit for bit; attention's outputs differ by their roundings at most where another kernel runs (tests/test_gpu_attention_layer.py).
"""
import numpy as np
import pytest
import torch

import kv_step_ref as step
from test_gpu_attention_layer import DIM, HIDDEN, _near, _rows, _same_projections, mod  # noqa: F401
from test_gpu_kv_scores import attend

pytestmark = pytest.mark.gpu
FULL = dict(rope_base=10000.0, norm=True, softcap=20.0)


def _layer(mod, fmt, batch=2, **kw):  # noqa: F811
    return mod.AttentionLayer(HIDDEN, 4, 2, DIM, batch, 512, mod.FORMATS[fmt], page_size=16, **kw)


def _slots(layer, b, n=None):
    at = torch.arange(layer.lens[b] if n is None else n, device="cuda:0")
    return layer.table[b, at // 16].long() * 16 + at % 16


def _held(layer, b):
    from bit_gemm_w4_amd import ops
    return ops.kv_cache_read(layer.cache, _slots(layer, b), torch.float32)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("how", [{}, FULL, dict(rope_base=500.0, slopes=True), dict(norm=True, window=50, sinks=4)], ids=lambda h: "-".join(h) or "plain")
def test_pages_of_a_pool(mod, fmt, how):  # noqa: F811
    """Interleaved sequences, ended and begun again, in few pages: the same as with pages of their own."""
    own, pool = _layer(mod, fmt, **how), _layer(mod, fmt, pool_pages=40, **how)
    x = _rows(700, 5)
    at = 0
    for counts in ([100, 3], [1, 1], [0, 90], [1, 1], [5, 30], "end", [60, 1], [1, 1]):
        if counts == "end":
            for layer in (own, pool):
                layer.end([0])
            assert pool.lens == own.lens == [0, 125]
            continue
        n = sum(counts)
        a, b = own.extend(x[at:at + n], counts), pool.extend(x[at:at + n], counts)
        assert torch.equal(a, b), counts
        at += n
    for b in range(2):
        if "window" not in how:
            assert all(torch.equal(s, t) for s, t in zip(_held(own, b), _held(pool, b)))
    assert pool.pool.lens.tolist() == pool.lens
    assert int(pool.pool.state[0]) == 40 - sum(pool._pages(n) for n in pool.lens)


def test_a_window_gives_pages_back(mod):  # noqa: F811
    """Sequences far longer than the pool: what slid out of the window serves again."""
    how = dict(rope_base=10000.0, window=40, sinks=5)
    own, pool = _layer(mod, "fp8", **how), _layer(mod, "fp8", pool_pages=14, **how)
    x = _rows(2 * 400, 6)
    for i in range(20):
        part = x[40 * i:40 * i + 40]
        assert torch.equal(own.extend(part, [20, 20]), pool.extend(part, [20, 20])), i
    assert pool.lens == [400, 400]


def test_a_pool_that_is_used_up(mod):  # noqa: F811
    layer = _layer(mod, "int8", pool_pages=10)
    layer.extend(_rows(100, 1), [100, 0])
    before = [t.clone() for t in layer.pool._tensors]
    with pytest.raises(ValueError, match="no pages"):       # 113 tokens in 8 pages, 48 in 3
        layer.extend(_rows(61, 2), [13, 48])
    assert layer.lens == [100, 0] and all(torch.equal(a, b) for a, b in zip(before, layer.pool._tensors))
    layer.extend(_rows(60, 2), [12, 48])                    # 112 in 7
    layer.end([0, 1])
    assert int(layer.pool.state[0]) == 10 and sorted(layer.pool.free.tolist()) == list(range(10))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
def test_a_text_in_chunks_or_token_by_token(mod, fmt):  # noqa: F811
    x = _rows(120, 1)
    layers, outs = [], []
    for counts in ([120], [70, 30] + [1] * 20):
        layer = _layer(mod, fmt, batch=1, pool_pages=9, **FULL)
        _same_projections(layer, x)
        y, at = [], 0
        for n in counts:
            part, _, _ = layer._attend(x[at:at + n], [n])
            layer.lens = [layer.lens[0] + n]
            y.append(part)
            at += n
        outs.append(torch.cat(y))
        layers.append(layer)
    assert all(torch.equal(a, b) for a, b in zip(_held(layers[0], 0), _held(layers[1], 0)))
    _near(outs[0], outs[1], _own_order(layers[0]))


def _own_order(layer):
    """The layer as _near reads it: its first sequence's slots in its table's order."""
    layer._slots = lambda b, first, n: _slots(layer, b, first + n)[first:].tolist()
    return layer


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("pool", [None, 30])
def test_a_checked_tree_is_its_branches(mod, fmt, pool):  # noqa: F811
    """Drafts stand at the positions of their depths; the accepted branch is what the text would have been."""
    x, drafts = _rows(90, 2), _rows(6, 3)
    parents = [-1, 0, 0, 2, -1, 3]
    layer = _layer(mod, fmt, batch=1, pool_pages=pool, **FULL)
    layer.extend(x, [90])
    whole = layer._project(drafts)
    layer._project = lambda part: whole
    y = layer._attend(drafts, [6], layer._ints(mod.tree_bits(parents), torch.int64), [mod.tree_depths(parents)])[0]
    for token in range(6):
        branch = [token]
        while parents[branch[0]] >= 0:
            branch.insert(0, parents[branch[0]])
        other = _layer(mod, fmt, batch=1, **FULL)
        other.extend(x, [90])
        other._project = lambda part, r=torch.tensor(branch).cuda(): tuple(t[r] for t in whole)
        z, _, _ = other._attend(drafts[:len(branch)], [len(branch)])
        other.lens = [90 + len(branch)]
        _near(y[token], z[-1], other)
    layer.check(drafts, [parents])
    assert layer.lens == [90]
    layer.accept([[0, 2, 3, 5]])
    assert layer.lens == [94] and (pool is None or layer.pool.lens.tolist() == [94])
    after = _layer(mod, fmt, batch=1, **FULL)
    after.extend(x, [90])
    after._project = lambda part: tuple(t[[0, 2, 3, 5]] for t in whole)
    after._attend(drafts[:4], [4])
    after.lens = [94]
    assert all(torch.equal(a, b) for a, b in zip(_held(layer, 0), _held(after, 0)))


@pytest.mark.parametrize("fmt,how", [("int8", FULL), ("fp8", dict(rope_base=10000.0, slopes=True)), ("int4", dict(rope_base=100.0, norm=True, softcap=5.0, slopes=True))])
def test_a_step_against_its_formulas(mod, fmt, how):  # noqa: F811
    """From the projected rows on: rotated queries to BF16 (half a step of each, 2^-8, moves a score by 2^-8 of its sum |q k|), keys
    as read back, scores, prefix and softmax in binary64."""
    layer = _layer(mod, fmt, pool_pages=64, **how)
    x = _rows(150, 8)
    q, _, _ = layer._project(x)
    y, _, _ = layer._attend(x, [110, 40], prefix=[60, 0])
    layer.lens = [110, 40]
    first = 0
    turns = [f % 2 ** 64 for f in layer.freqs.tolist()]
    for b, n in enumerate(layer.lens):
        k, v = (t.double().cpu().numpy() for t in _held(layer, b))
        rows = q[first:first + n].double().cpu().numpy()
        w = None if layer.q_weight is None else layer.q_weight.double().cpu().numpy()
        turned = step.turn(rows, w, range(n), turns)
        at = np.arange(n)
        see = (at <= at[:, None]) | (at < [60, 0][b])
        for h in range(4):
            kh, vh = k[:, h // 2], v[:, h // 2]
            out, _, mean, moved, total = attend(turned[:, h], kh, vh, see, at, DIM ** -0.5, layer.softcap,
                                                float(layer.slopes[h]) if layer.slopes is not None else 0.0)
            off = 2.0 ** -8 * (np.abs(turned[:, h]) @ np.abs(kh).T).max(1) * DIM ** -0.5
            got = y[first:first + n, h].double().cpu().numpy()
            weights = (np.exp(2 * off) - 1)[:, None] * (mean + np.abs(out))
            tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + (n + 16) * 2.0 ** -24 + total)[:, None] * mean * 2 + moved + weights + n * 2.0 ** -24 * np.abs(vh).max()
            assert (np.abs(got - out) <= tol).all()
        first += n


def test_a_decode_step_in_a_graph(mod):  # noqa: F811
    """Plan, cache write and attention of a step, captured once: every replay is the next token of all sequences."""
    from bit_gemm_w4_amd import ops
    B, heads, kv, page = 5, 8, 2, 16
    freqs = ops.rope_freqs([10000.0 ** (-2.0 * i / DIM) for i in range(DIM // 2)]).cuda()
    g = torch.Generator().manual_seed(0)
    rows = torch.randn(60, B, (heads + 2 * kv) * DIM, generator=g).to("cuda:0", torch.bfloat16)
    row = rows[0].clone()
    parts = [t.unflatten(1, (-1, DIM)) for t in row.split([heads * DIM, kv * DIM, kv * DIM], 1)]
    ones = torch.ones(B, dtype=torch.int32, device="cuda:0")
    slopes = torch.exp2(-torch.arange(1, heads + 1, device="cuda:0").float())

    def make():
        return ops.kv_cache(100, page, kv, DIM, ops.FP8_E4M3, "cuda:0"), ops.kv_pool(100, page, B, 20, window=30, sinks=2, device="cuda:0")

    def once(cache, pool):
        p = ops.kv_plan(pool, ones, B)
        q = ops.kv_cache_write_rope(*parts, cache, p.slots, p.positions, freqs)
        y = ops.kv_attn(q, cache, pool.block_table, p.kv_lens, p.cu_q, 1, max_kv_len=320, window=30, sinks=2, softcap=10.0, slopes=slopes)
        ops.kv_release(pool)
        return y

    eager, captured = make(), make()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    once(*make())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        out = once(*captured)
    for i in range(60):
        row.copy_(rows[i])
        want = once(*eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
    assert all(torch.equal(a, b) for a, b in zip(eager[1]._tensors[1:], captured[1]._tensors[1:])) and captured[1].lens.tolist() == [60] * B


def test_the_command_runs(mod, capsys):  # noqa: F811
    mod.main(["--format", "fp8", "--rope", "10000", "--norm", "--softcap", "30", "--pool", "24"])
    mod.main(["--format", "int8", "--rope", "10000", "--slopes", "--window", "100", "--sinks", "4", "--pool", "30"])
    out = capsys.readouterr().out
    assert "lengths [707, 338]" in out and "lengths [704, 337]" in out


def test_refusals(mod):  # noqa: F811
    layer = _layer(mod, "int8", batch=1, slopes=True)
    with pytest.raises(ValueError, match="no slopes"):
        layer.check(_rows(2, 4), [[-1, 0]])
