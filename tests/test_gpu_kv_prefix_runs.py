"""A window with a prefix far wider than it: the runs of positions of a row are about equal, and right (GPU).

Without a bound on a sequence's queries their number is taken from the mean, so a long sequence's rows see more tiles of
positions than its runs were sized for.  Where the queries are zeros a run's partial log-sum-exp is the log of its positions,
which says how many it took: none more than its share.
"""
import pytest
import torch

from test_gpu_kv_scores import Scored, ops  # noqa: F401

pytestmark = pytest.mark.gpu
FORM = [  # D, group, queries of the long sequence, sequences, window, sinks, kernel of a prefix alone, tile
    (64, 1, 1000, 16, 64, 4, "few", 32), (64, 1, 3000, 8, 64, 5, "few", 32), (128, 1, 3000, 16, 64, 4, "few", 32), (256, 1, 1000, 8, 64, 3, "few", 32),
    (64, 4, 8000, 8, 64, 0, "many", 64), (128, 4, 8000, 2, 400, 9, "many", 64), (256, 4, 3000, 2, 64, 0, "many", 64),
]


def case(ops, D, group, long, seqs, window, sinks, **how):  # noqa: F811
    lens = [long] + [1 + 3 * i for i in range(seqs - 1)]
    return Scored(ops, 3, "bf16", 1, group, D, 32, [long] + [1] * (seqs - 1), lens, seed=D + seqs, window=window, sinks=sinks, prefix=[long - 7] + lens[1:], **how)


def run(ops, s):  # noqa: F811
    """Without a bound on the queries: outputs, log-sum-exps, and the partial ones of each run."""
    c = s.c
    T, heads, D = c.q.shape
    need = ops.kv_attn_workspace_bytes(c.q.shape, c.cache, len(c.q_lens), c.bt.shape[1], T, 0, c.window, c.sinks)
    splits = need // (T * heads * (D + 1) * 4)
    assert splits > 1
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    lse = torch.empty(T, heads, device="cuda")
    got = ops.kv_attn(c.q, c.cache, c.bt, c.lens, c.cu, window=c.window, sinks=c.sinks, ws=ws, lse=lse, **s.how)
    return got, lse, ws.view(torch.float32)[splits * T * heads * D:].view(splits, T, heads)


@pytest.mark.parametrize("D,group,long,seqs,window,sinks,form,tile", FORM)
def test_runs_are_equal(ops, D, group, long, seqs, window, sinks, form, tile):  # noqa: F811
    s = case(ops, D, group, long, seqs, window, sinks)
    s.c.q.zero_()
    _, _, parts = run(ops, s)
    assert ops.last_kernel().startswith("k_kv_attn_few_scored<" if form == "few" else "k_kv_attn_many_bias<")
    splits = parts.shape[0]
    took = torch.exp2(parts[:, :long, 0])           # positions of each run
    at = torch.arange(long, device="cuda")
    low = (at - window + 1).clamp(min=0)
    high = torch.maximum(at + 1, torch.full_like(at, long - 7))
    seen = high - low + low.clamp(max=sinks)
    assert (took.sum(0) - seen).abs().max() < 0.5
    # a run is what the plan counted on (a row's window, the mean of the queries or a block's, two tiles, the sinks and theirs, over the
    # splits) if a block's tiles are no more than that, else an equal share of them: of what its row sees, up to 256 positions that
    # others of the block see besides, a part of a tile at either end, rounded up to a tile
    mean = max(-(-parts.shape[1] // seqs), 256)
    counted = (window + mean + 64 + sinks + 64) / splits + tile
    assert (took.max(0).values <= ((seen + 256) / splits + 2 * tile).clamp(min=counted)).all(), (took.max().item(), seen.max().item(), splits)
    assert took.max() <= (long + 256) / splits + 2 * tile


@pytest.mark.parametrize("D,group,long,seqs,window,sinks,form,tile", FORM)
@pytest.mark.parametrize("how", [dict(), dict(cap=20.0), dict(slopes=[0.01, 0.1]), dict(cap=300.0, slopes=[0.01])], ids=lambda h: "-".join(h) or "prefix")
def test_against_binary64(ops, D, group, long, seqs, window, sinks, form, tile, how):  # noqa: F811
    s = case(ops, D, group, long, seqs, window, sinks, **how)
    got, lse, _ = run(ops, s)
    s.check(got, lse, only=[0, 1, 63, 64, 300, 700, 999, long - 8, long - 1])
