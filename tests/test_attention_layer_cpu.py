"""The attention layer's own state: which drafts can be accepted, and where they go (no GPU needed)."""
import pytest
import torch

from bit_gemm_w4_amd import attention_layer


@pytest.fixture
def layer(monkeypatch):
    """A layer of two sequences whose operators note what they are given."""
    x = object.__new__(attention_layer.AttentionLayer)
    x.q_heads = x.kv_heads = 1
    x.head_dim, x.window, x.sinks, x.page_size, x.max_tokens = 4, 0, 0, 16, 32
    x.qkv = x.o = x.cache = None
    x.table = torch.arange(4, dtype=torch.int32).view(2, 2)
    x.lens, x.drafts, x.written = [0, 0], None, []
    x._project = lambda rows: (rows[:, None],) * 3
    ops = attention_layer.ops
    monkeypatch.setattr(ops, "gemm_w4a16", lambda rows, w: rows)
    monkeypatch.setattr(ops, "kv_cache_write", lambda k, v, cache, slots: x.written.append((k[:, 0, 0].tolist(), slots.tolist())))
    monkeypatch.setattr(ops, "kv_attn", lambda q, *a, **kw: q)
    monkeypatch.setattr(ops, "kv_attn_tree", lambda q, *a, **kw: q)
    return x


def _rows(*ids):
    return torch.tensor(ids, dtype=torch.float32)[:, None].expand(-1, 4)


def test_an_accepted_branch_moves_up(layer):
    layer.extend(_rows(*range(8)), [5, 3])
    layer.check(_rows(10, 11, 12, 13, 20, 21), [[-1, 0, 0, 2], [-1, -1]])
    assert layer.written[-1] == ([10, 11, 12, 13, 20, 21], [5, 6, 7, 8, 32 + 3, 32 + 4])
    layer.accept([[0, 2, 3], [1]])
    assert layer.written[-1] == ([10, 12, 13, 21], [5, 6, 7, 32 + 3])
    assert layer.lens == [8, 4] and layer.drafts is None


def test_empty_branches_and_trees(layer):
    layer.extend(_rows(0, 1), [1, 1])
    layer.check(_rows(10), [[-1], []])
    layer.accept([[], []])
    assert layer.lens == [1, 1]
    layer.check(_rows().view(0, 4), [[], []])
    layer.accept([[], []])
    assert layer.lens == [1, 1]


def test_nothing_checked(layer):
    with pytest.raises(ValueError, match="no checked drafts"):
        layer.accept([[0], [0]])
    layer.extend(_rows(0, 1), [1, 1])
    layer.check(_rows(10, 20), [[-1], [-1]])
    layer.accept([[0], [0]])
    with pytest.raises(ValueError, match="no checked drafts"):
        layer.accept([[0], [0]])


def test_new_tokens_take_the_drafts_place(layer):
    layer.extend(_rows(0, 1), [1, 1])
    layer.check(_rows(10, 20), [[-1], [-1]])
    layer.extend(_rows(2, 3), [1, 1])
    before = list(layer.written)
    with pytest.raises(ValueError, match="no checked drafts"):
        layer.accept([[0], [0]])
    assert layer.lens == [2, 2] and layer.written == before


@pytest.mark.parametrize("branches", [[[0, 1], [2]], [[0, 1], [-1]], [[0, 3], [0]], [[1], [0]], [[0, 1, 2], [0]], [[0, 0], [0]], [[0], [0, 1]]])
def test_what_is_no_branch_is_refused(layer, branches):
    layer.extend(_rows(0, 1), [1, 1])
    layer.check(_rows(10, 11, 12, 13, 20, 21), [[-1, 0, 0, 2], [-1, -1]])
    before = list(layer.written)
    with pytest.raises(ValueError, match="no branch"):
        layer.accept(branches)
    assert layer.lens == [1, 1] and layer.written == before
    layer.accept([[0, 1], [0]])                             # the drafts are still there


def test_one_branch_per_sequence(layer):
    layer.extend(_rows(0, 1), [1, 1])
    layer.check(_rows(10, 20), [[-1], [-1]])
    with pytest.raises(ValueError, match="1 branches for 2"):
        layer.accept([[0]])
