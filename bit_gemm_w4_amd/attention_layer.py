"""The attention half of a decoder layer on quantized weights and a quantized
KV cache: the framework's W4A16 linears, the paged cache and the attention
over it, together as a serving program uses them.

    python -m bit_gemm_w4_amd.attention_layer [--format int8|fp8|int4] [--window W --sinks S]

runs an answer of a small batch: prompts enter in chunks, tokens follow one at
a time, then a tree of drafted tokens is checked in one pass and its accepted
branch kept.  Rotary positions, norms and the MLP are the model's and left out.
"""
from __future__ import annotations

import argparse

import torch

from . import ops, synth

FORMATS = {"int8": ops.I8, "fp8": ops.FP8_E4M3, "int4": ops.U4}


def tree_bits(parents: list[int]) -> list[list[int]]:
    """int64 words of each drafted token's ancestors, itself included; parents[i] < i, or -1 for
    a token that follows the prefix."""
    words = (len(parents) + 63) // 64
    rows: list[int] = []
    for i, up in enumerate(parents):
        if up >= i or up < -1:
            raise ValueError(f"tree_bits: parent {up} of token {i} does not come before it")
        rows.append((rows[up] if up >= 0 else 0) | 1 << i)
    word = lambda b: b - (1 << 64) if b >> 63 else b  # noqa: E731
    return [[word(b >> 64 * w & (1 << 64) - 1) for w in range(words)] for b in rows]


class AttentionLayer:
    """Weights, cache pages and lengths of `batch` sequences of up to max_tokens."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, batch: int, max_tokens: int, format: int = ops.FP8_E4M3,
                 page_size: int = 64, window: int = 0, sinks: int = 0, dtype: torch.dtype = torch.bfloat16, device: str = "cuda:0"):
        self.q_heads, self.kv_heads, self.head_dim, self.dtype = q_heads, kv_heads, head_dim, dtype
        self.window, self.sinks, self.page_size, self.max_tokens = window, sinks, page_size, max_tokens
        self.widths = [q_heads * head_dim, kv_heads * head_dim, kv_heads * head_dim]
        pack = lambda n, k, seed: ops.w4_pack(torch.from_numpy(synth.weights(n, k, seed)).to(device), 128, False)  # noqa: E731
        self.qkv, self.o = pack(sum(self.widths), hidden, 0), pack(hidden, q_heads * head_dim, 1)
        per = -(-max_tokens // page_size)
        self.cache = ops.kv_cache(batch * per, page_size, kv_heads, head_dim, format, torch.device(device))
        self.table = torch.arange(batch * per, dtype=torch.int32, device=device).view(batch, per)
        self.lens = [0] * batch
        self.drafts = None

    def _ints(self, x, dt=torch.int32):
        return torch.tensor(x, dtype=dt, device=self.table.device)

    def _slots(self, b: int, first: int, n: int):
        per = self.table.shape[1] * self.page_size          # a sequence's pages lie in order here
        return [b * per + j for j in range(first, first + n)]

    def _project(self, x):
        qkv = ops.gemm_w4a16(x, self.qkv)
        q, k, v = qkv.split(self.widths, 1)                 # views: the operators take the rows as they lie
        heads = lambda t, n: t.unflatten(1, (n, self.head_dim))  # noqa: E731
        return heads(q, self.q_heads), heads(k, self.kv_heads), heads(v, self.kv_heads)

    def _attend(self, x, counts: list[int], tree=None):
        """x: the rows of counts[b] new tokens of each sequence, one sequence after the other."""
        if any(n + c > self.max_tokens for n, c in zip(self.lens, counts)):
            raise ValueError("AttentionLayer: the cache is full")
        q, k, v = self._project(x)
        slots = [s for b, n in enumerate(counts) for s in self._slots(b, self.lens[b], n)]
        ops.kv_cache_write(k, v, self.cache, self._ints(slots, torch.int64))
        kv = [n + c for n, c in zip(self.lens, counts)]
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        args = (q, self.cache, self.table, self._ints(kv), self._ints(cu))
        if tree is None:
            y = ops.kv_attn(*args, max(counts), max_kv_len=max(kv), window=self.window, sinks=self.sinks)
        else:
            y = ops.kv_attn_tree(*args, tree, max(counts), max_kv_len=max(kv))
        return y, k, v

    def extend(self, x: torch.Tensor, counts: list[int]) -> torch.Tensor:
        """counts[b] further tokens of each sequence (a prompt's chunk; one each: a decode step)."""
        y, _, _ = self._attend(x, counts)
        self.lens = [n + c for n, c in zip(self.lens, counts)]
        self.drafts = None                                  # their rows are overwritten
        return ops.gemm_w4a16(y.flatten(1), self.o)

    def check(self, x: torch.Tensor, parents: list[list[int]]) -> torch.Tensor:
        """Drafted tokens of each sequence as a tree: their rows lie behind the sequence until `accept`."""
        if self.window:
            raise ValueError("AttentionLayer: draft trees see the whole prefix: no window")
        words = max(1, (max(len(p) for p in parents) + 63) // 64)
        rows = [r + [0] * (words - len(r)) for p in parents for r in tree_bits(p)]
        y, k, v = self._attend(x, [len(p) for p in parents], self._ints(rows, torch.int64).view(-1, words))
        self.drafts = (k, v, [list(p) for p in parents])
        return ops.gemm_w4a16(y.flatten(1), self.o)

    def accept(self, branches: list[list[int]]) -> None:
        """Keep one branch of the last `check` per sequence, from the prefix on (empty: none of its tokens): they move
        up behind the prefix."""
        if self.drafts is None:
            raise ValueError("AttentionLayer: no checked drafts to accept from")
        k, v, trees = self.drafts
        if len(branches) != len(trees):
            raise ValueError(f"AttentionLayer: {len(branches)} branches for {len(trees)} sequences")
        rows, slots, first = [], [], 0
        for b, (branch, parents) in enumerate(zip(branches, trees)):
            for up, i in zip([-1, *branch], branch):
                if not 0 <= i < len(parents) or parents[i] != up:
                    raise ValueError(f"AttentionLayer: {list(branch)} is no branch of sequence {b}'s tree {parents}")
            rows += [first + i for i in branch]
            slots += self._slots(b, self.lens[b], len(branch))
            first += len(parents)
        at = self._ints(rows, torch.int64)
        ops.kv_cache_write(k[at], v[at], self.cache, self._ints(slots, torch.int64))
        self.lens = [n + len(branch) for n, branch in zip(self.lens, branches)]
        self.drafts = None


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--format", choices=sorted(FORMATS), default="fp8")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    a = ap.parse_args(argv)
    hidden, counts = 1024, [700, 333]
    layer = AttentionLayer(hidden, 8, 2, 128, 2, 1024, FORMATS[a.format], window=a.window, sinks=a.sinks)
    rows = lambda n, seed: torch.from_numpy(synth.activations(n, hidden, "f32", seed)).to("cuda:0", layer.dtype)  # noqa: E731
    y = layer.extend(rows(sum(counts), 2), counts)
    print(f"prompts of {counts} tokens: {tuple(y.shape)}, cache {layer.cache.nbytes / 2 ** 20:.1f} MiB in {a.format}")
    for step in range(4):
        y = layer.extend(rows(2, 3 + step), [1, 1])
    print(f"4 decode steps: {tuple(y.shape)}, lengths {layer.lens}")
    if not a.window:
        parents = [[-1, 0, 0, 1, 2], [-1, -1, 0]]
        y = layer.check(rows(8, 9), parents)
        layer.accept([[0, 2, 4], [1]])
        print(f"trees of {[len(p) for p in parents]} drafted tokens: {tuple(y.shape)}, lengths {layer.lens}")
    k, _ = ops.kv_cache_read(layer.cache, layer._ints(layer._slots(0, 0, layer.lens[0]), torch.int64))
    print(f"keys read back: {tuple(k.shape)}, largest {k.abs().max().item():.3f}")
    return layer


if __name__ == "__main__":
    main()
