"""Captured attention calls whose sequences are split: each graph has its own workspace (GPU)."""
import pytest
import torch

from kv_ref import FP8, I8, U4
from test_gpu_kv import Case, ops  # noqa: F401

pytestmark = pytest.mark.gpu


def _span(t):
    return t.data_ptr(), t.data_ptr() + t.numel()


def _apart(a, b):
    return a[1] <= b[0] or b[1] <= a[0]


@pytest.mark.parametrize("tree", [False, True])
def test_graphs_and_eager_calls_share_no_workspace(ops, tree, monkeypatch):  # noqa: F811
    cases = [Case(ops, fmt, "bf16", 2, 4, 128, 16, q, kv, seed=60 + fmt, tree=tree)
             for fmt, q, kv in ((I8, [2, 3], [4000, 9000]), (FP8, [4], [7000]), (U4, [3, 1, 2], [5000, 30, 800]))]
    seen = []
    own = ops._kv_workspace

    def watch(*args):
        ws = own(*args)
        seen.append(_span(ws))
        return ws
    monkeypatch.setattr(ops, "_kv_workspace", watch)
    want = [c.run(ops) for c in cases]
    assert len(seen) == len(cases)                  # every call is split
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs, spans = [], [], []
    for c in cases[:2]:
        g, out = torch.cuda.CUDAGraph(), torch.empty_like(c.q).contiguous()
        seen.clear()
        with torch.cuda.graph(g, stream=side):
            c.run(ops, out=out)
        spans.append(seen[-1])
        graphs.append(g), outs.append(out)
    seen.clear()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cases[2].run(ops)
    torch.cuda.synchronize()
    spans.append(seen[-1])
    assert all(_apart(a, b) for i, a in enumerate(spans) for b in spans[:i])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(5):
        for out in outs:
            out.fill_(7.0)
        torch.cuda.synchronize()
        got = None
        for _ in range(4):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
            with torch.cuda.stream(side):
                got = cases[2].run(ops)
        torch.cuda.synchronize()
        for a, b in zip((*outs, got), want):
            assert torch.equal(a, b), rep
