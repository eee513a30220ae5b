"""Many query rows: batches that fill the device, as copies of the sequences of the smaller tests (GPU).

A batch of few sequences takes blocks of few rows however many its queries
are.  Here each call holds as many copies of its sequences as make the blocks
of many rows the faster choice; every copy has to agree with the first bit for
bit, and the first is held to the same bounds.
"""
import pytest
import torch

import test_gpu_kv as base
import test_gpu_kv_edges as edges
from kv_ref import FP8, I8, U4
from test_gpu_kv import ops  # noqa: F401

pytestmark = pytest.mark.gpu

FORMATS = [I8, FP8, U4]


class Copies(base.Case):
    blocks = 256          # sequences x kv heads of a call

    def run(self, ops, *, out=None, lse=None, stream=None, **kw):  # noqa: F811
        n, T = max(1, self.blocks // (len(self.q_lens) * self.heads)), self.q.shape[0]
        cu = self.cu[1:][None] + T * torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
        cu = torch.cat((self.cu[:1], cu.reshape(-1)))
        q, bt, lens = self.q.repeat(n, 1, 1), self.bt.repeat(n, 1), self.lens.repeat(n)
        all_lse = None if lse is None else torch.empty(n * T, q.shape[1], device="cuda")
        kw.setdefault("max_kv_len", self.max_kv)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        if self.tree is not None:
            got = ops.kv_attn_tree(q, self.cache, bt, lens, cu, self.tree.repeat(n, 1), self.max_q, lse=all_lse, stream=stream, **kw)
        else:
            got = ops.kv_attn(q, self.cache, bt, lens, cu, self.max_q, window=self.window, sinks=self.sinks, lse=all_lse,
                              stream=stream, **kw)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        for x, to in ((got, out), (all_lse, lse)):
            if x is not None:
                bits = x.view(n, T, *x.shape[1:]).view(torch.int32 if x.dtype == torch.float32 else torch.int16)
                if not torch.cuda.is_current_stream_capturing():
                    assert torch.equal(bits, bits[:1].expand_as(bits))
            if to is not None:
                to.copy_(x[:T])
        return got[:T] if out is None else out


@pytest.fixture(autouse=True)
def copies(monkeypatch):
    monkeypatch.setattr(base, "Case", Copies)
    monkeypatch.setattr(edges, "Case", Copies)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", base.SHAPES)
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 70, 0, 130], [40, 300, 9, 131]), ([300], [555]), ([100, 67], [100, 1000])])
def test_chunks(ops, fmt, dtype, shape, q_lens, kv_lens):  # noqa: F811
    base.test_chunks(ops, fmt, dtype, shape, q_lens, kv_lens)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (33, 1), (64, 64), (100, 200), (5000, 4), (16, 17)])
@pytest.mark.parametrize("q_lens,kv_lens,shape", [([9, 150, 2], [30, 400, 777], (1, 3, 64, 32)), ([130], [900], (2, 5, 128, 64)),
                                                  ([90, 70], [90, 600], (1, 2, 256, 16))])
def test_windows_and_sinks(ops, fmt, window, sinks, q_lens, kv_lens, shape):  # noqa: F811
    base.test_windows_and_sinks(ops, fmt, window, sinks, q_lens, kv_lens, shape)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_lens,kv_lens,shape", [([64, 3, 30], [64, 70, 999], (1, 4, 64, 32)), ([65, 130], [300, 130], (1, 2, 128, 64)),
                                                  ([70, 1], [71, 1200], (2, 2, 256, 128)), ([17, 8], [2000, 8], (2, 8, 128, 16)),
                                                  ([200], [263], (1, 7, 128, 16))])
def test_trees(ops, fmt, dtype, q_lens, kv_lens, shape):  # noqa: F811
    base.test_trees(ops, fmt, dtype, q_lens, kv_lens, shape)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens,kind", [([60, 200], [100, 500], "causal"), ([30], [700], "tree")])
def test_pages_that_are_not_there(ops, fmt, q_lens, kv_lens, kind):  # noqa: F811
    base.test_pages_that_are_not_there(ops, fmt, q_lens, kv_lens, kind)


def test_tree_bits_past_the_words_are_not_seen(ops):  # noqa: F811
    base.test_tree_bits_past_the_words_are_not_seen(ops)


def test_more_queries_than_positions(ops):  # noqa: F811
    base.test_more_queries_than_positions(ops)


@pytest.mark.parametrize("fmt", FORMATS)
def test_peaked_rows_and_small_values(ops, fmt):  # noqa: F811
    base.test_peaked_rows_and_small_values(ops, fmt, [150], [700])


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_stays_with_the_rows_that_see_it(ops, fmt):  # noqa: F811
    base.test_nan_stays_with_the_rows_that_see_it(ops, fmt, [20, 200], [100, 400])


@pytest.mark.parametrize("q_lens,kv_lens,tree", base.CALLS[1:])
def test_another_stream(ops, q_lens, kv_lens, tree):  # noqa: F811
    base.test_another_stream(ops, q_lens, kv_lens, tree)


@pytest.mark.parametrize("q_lens,kv_lens,tree", base.CALLS[1:])
@pytest.mark.parametrize("fmt", FORMATS)
def test_graph_replays(ops, fmt, q_lens, kv_lens, tree):  # noqa: F811
    base.test_graph_replays(ops, fmt, q_lens, kv_lens, tree)


def test_repeated_calls_agree_bit_for_bit(ops):  # noqa: F811
    base.test_repeated_calls_agree_bit_for_bit(ops)


@pytest.mark.parametrize("q_lens,kv_lens", [([100, 4], [70, 70]), ([200], [130])])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 40, 160, 129])
def test_windows_wider_than_the_positions_before_them(ops, q_lens, kv_lens, window):  # noqa: F811
    edges.test_windows_wider_than_the_positions_before_them(ops, q_lens, kv_lens, window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,kv,bound,blocks", [(150, 4200, 0, 64), (150, 4200, 0, 256), (150, 4200, 300, 256), (600, 1500, 0, 64),
                                                  (600, 1500, 0, 256), (128, 6000, 0, 17)])
def test_splits(ops, fmt, D, rows, kv, bound, blocks, monkeypatch):  # noqa: F811
    monkeypatch.setattr(Copies, "blocks", blocks)
    edges.test_splits(ops, fmt, D, rows, kv, bound)


@pytest.mark.parametrize("fmt", FORMATS)
def test_value_scales_that_grow_along_the_sequence(ops, fmt):  # noqa: F811
    edges.test_value_scales_that_grow_along_the_sequence(ops, fmt)


def test_queries_of_very_different_size_in_one_block(ops):  # noqa: F811
    edges.test_queries_of_very_different_size_in_one_block(ops)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens,group,window,sinks,tree", [([100, 67], [100, 1000], 1, 0, 0, False), ([18], [333], 7, 0, 0, False),
                                                                    ([25, 20], [700, 20], 5, 70, 9, False), ([64, 33], [300, 33], 2, 0, 0, True),
                                                                    ([128, 0], [40, 50], 1, 0, 0, False)])
def test_blocks_of_128_rows(ops, fmt, q_lens, kv_lens, group, window, sinks, tree, monkeypatch):  # noqa: F811
    """Head size 64, up to 128 rows: two blocks of four waves a compute unit."""
    monkeypatch.setattr(Copies, "blocks", 512)
    c = Copies(ops, fmt, "bf16", 1, group, 64, 16, q_lens, kv_lens, seed=40, window=window, sinks=sinks, tree=tree, gone=0.1)
    lse = torch.empty(sum(q_lens), group, device="cuda")
    got = c.run(ops, lse=lse)
    assert ops.last_kernel() == f"k_kv_attn_many<{fmt}, 64, 4>"
    c.check(got, lse)
    assert torch.equal(got, c.run(ops))
