"""The attention half of a decoder layer on quantized weights and a quantized
KV cache: the framework's W4A16 linears, the paged cache and the attention
over it, together as a serving program uses them.

    python -m bit_gemm_w4_amd.attention_layer [--format int8|fp8|int4] [--window W --sinks S]
                                              [--rope BASE] [--norm] [--softcap C] [--slopes] [--pool PAGES]

runs an answer of a small batch: prompts enter in chunks, tokens follow one at
a time, then a tree of drafted tokens is checked in one pass and its accepted
branch kept.  On request heads are normed and rotated on their way into the
cache, scores capped or biased by distance, and pages come from a shared pool, on the
device.  The MLP and the residual stream's norms are the model's and left out.
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


def tree_depths(parents: list[int]) -> list[int]:
    """How many of its ancestors each drafted token has: its position behind the prefix."""
    depths: list[int] = []
    for up in parents:
        depths.append(depths[up] + 1 if up >= 0 else 0)
    return depths


class AttentionLayer:
    """Weights, cache pages and lengths of `batch` sequences of up to max_tokens.

    rope_base: queries and keys are rotated by their positions; norm: and each head
    normed before; softcap: scores are capped; slopes: and fall with distance, by
    2^(-8 i / q_heads) in head i; pool_pages: the sequences share so many pages, which kv_plan hands out (without
    it each has its own, in order)."""

    freqs = q_weight = k_weight = slopes = pool = None
    softcap = 0.0

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, batch: int, max_tokens: int, format: int = ops.FP8_E4M3,
                 page_size: int = 64, window: int = 0, sinks: int = 0, dtype: torch.dtype = torch.bfloat16, device: str = "cuda:0", *,
                 rope_base: float | None = None, norm: bool = False, softcap: float = 0.0, slopes: bool = False, pool_pages: int | None = None):
        self.q_heads, self.kv_heads, self.head_dim, self.dtype = q_heads, kv_heads, head_dim, dtype
        self.window, self.sinks, self.page_size, self.max_tokens = window, sinks, page_size, max_tokens
        self.widths = [q_heads * head_dim, kv_heads * head_dim, kv_heads * head_dim]
        pack = lambda n, k, seed: ops.w4_pack(torch.from_numpy(synth.weights(n, k, seed)).to(device), 128, False)  # noqa: E731
        self.qkv, self.o = pack(sum(self.widths), hidden, 0), pack(hidden, q_heads * head_dim, 1)
        per = -(-max_tokens // page_size)
        self.cache = ops.kv_cache(pool_pages or batch * per, page_size, kv_heads, head_dim, format, torch.device(device))
        if pool_pages:
            self.pool = ops.kv_pool(pool_pages, page_size, batch, per, window=window, sinks=sinks, device=torch.device(device))
            self.table = self.pool.block_table
        else:
            self.table = torch.arange(batch * per, dtype=torch.int32, device=device).view(batch, per)
        if rope_base is not None:
            self.freqs = ops.rope_freqs([rope_base ** (-2.0 * i / head_dim) for i in range(head_dim // 2)]).to(device)
        if norm:
            self.q_weight, self.k_weight = (torch.ones(head_dim, dtype=dtype, device=device) for _ in range(2))
        self.softcap = softcap
        if slopes:
            self.slopes = torch.exp2(-8.0 * torch.arange(1, q_heads + 1, device=device) / q_heads)
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

    def _write(self, q, k, v, slots, positions):
        """Keys and values into the cache -> the queries to attend with (q None: none)."""
        if self.freqs is None and self.q_weight is None:
            ops.kv_cache_write(k, v, self.cache, slots)
            return q
        return ops.kv_cache_write_rope(q, k, v, self.cache, slots, positions, self.freqs, q_weight=self.q_weight, k_weight=self.k_weight)

    def _pages(self, n: int) -> int:
        """Pages that a sequence of n tokens holds."""
        held = -(-n // self.page_size)
        if not self.window:
            return held
        sink, slid = -(-self.sinks // self.page_size), max(0, n - self.window + 1) // self.page_size
        return held - max(0, min(slid, held) - sink)

    def _has_room(self, counts: list[int]) -> None:
        if any(n + c > self.max_tokens for n, c in zip(self.lens, counts)):
            raise ValueError("AttentionLayer: the cache is full")
        if self.pool is not None:
            page = self.page_size
            need = sum(-(-(n + c) // page) + -n // page for n, c in zip(self.lens, counts))
            if need > self.cache.pages - sum(self._pages(n) for n in self.lens):
                raise ValueError("AttentionLayer: no pages left")

    def _plan(self, counts: list[int], keep: bool = True):
        """cu_q, kv_lens, positions and slots of counts[b] new tokens of each sequence (keep: which it has from then on)."""
        if self.pool is not None:
            plan = ops.kv_plan(self.pool, self._ints(counts), sum(counts), advance=keep)
            return plan.cu_q, plan.kv_lens, plan.positions, plan.slots
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        slots = [s for b, n in enumerate(counts) for s in self._slots(b, self.lens[b], n)]
        positions = self._ints([n + i for n, c in zip(self.lens, counts) for i in range(c)]) if self.freqs is not None else None
        return self._ints(cu), self._ints([n + c for n, c in zip(self.lens, counts)]), positions, self._ints(slots, torch.int64)

    def _attend(self, x, counts: list[int], tree=None, depths: list[list[int]] | None = None, prefix: list[int] | None = None):
        """x: the rows of counts[b] new tokens of each sequence, one sequence after the other."""
        self._has_room(counts)
        q, k, v = self._project(x)
        cu, kv, positions, slots = self._plan(counts, tree is None)
        if depths is not None and self.freqs is not None:
            positions = self._ints([n + d for n, of in zip(self.lens, depths) for d in of])
        q = self._write(q, k, v, slots, positions)
        args = (q, self.cache, self.table, kv, cu)
        most = max(n + c for n, c in zip(self.lens, counts))
        if tree is None:
            how = {}
            if self.softcap or self.slopes is not None or prefix is not None:
                how = dict(softcap=self.softcap, slopes=self.slopes, prefix_lens=None if prefix is None else self._ints(prefix))
            y = ops.kv_attn(*args, max(counts), max_kv_len=most, window=self.window, sinks=self.sinks, **how)
        else:
            y = ops.kv_attn_tree(*args, tree, max(counts), max_kv_len=most, **(dict(softcap=self.softcap) if self.softcap else {}))
        return y, k, v

    def extend(self, x: torch.Tensor, counts: list[int], prefix: list[int] | None = None) -> torch.Tensor:
        """counts[b] further tokens of each sequence (a prompt's chunk; one each: a decode step).  prefix: positions
        below prefix[b] are seen by all of its tokens."""
        y, _, _ = self._attend(x, counts, prefix=prefix)
        self.lens = [n + c for n, c in zip(self.lens, counts)]
        if self.pool is not None and self.window:
            ops.kv_release(self.pool)                       # pages that slid out of the window
        self.drafts = None                                  # their rows are overwritten
        return ops.gemm_w4a16(y.flatten(1), self.o)

    def check(self, x: torch.Tensor, parents: list[list[int]]) -> torch.Tensor:
        """Drafted tokens of each sequence as a tree: their rows lie behind the sequence until `accept`."""
        if self.window:
            raise ValueError("AttentionLayer: draft trees see the whole prefix: no window")
        if self.slopes is not None:
            raise ValueError("AttentionLayer: drafted tokens do not lie in order: no slopes")
        words = max(1, (max(len(p) for p in parents) + 63) // 64)
        rows = [r + [0] * (words - len(r)) for p in parents for r in tree_bits(p)]
        y, k, v = self._attend(x, [len(p) for p in parents], self._ints(rows, torch.int64).view(-1, words), [tree_depths(p) for p in parents])
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
        rows, first = [], 0
        for b, (branch, parents) in enumerate(zip(branches, trees)):
            for up, i in zip([-1, *branch], branch):
                if not 0 <= i < len(parents) or parents[i] != up:
                    raise ValueError(f"AttentionLayer: {list(branch)} is no branch of sequence {b}'s tree {parents}")
            rows += [first + i for i in branch]
            first += len(parents)
        at = self._ints(rows, torch.int64)
        _, _, positions, slots = self._plan([len(branch) for branch in branches])
        self._write(None, k[at], v[at], slots, positions)
        self.lens = [n + len(branch) for n, branch in zip(self.lens, branches)]
        self.drafts = None

    def end(self, sequences: list[int]) -> None:
        """The sequences have ended: with a pool their pages are free for others."""
        self.lens = [0 if b in sequences else n for b, n in enumerate(self.lens)]
        if self.pool is not None:
            ops.kv_release(self.pool, self._ints(self.lens))
        self.drafts = None


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--format", choices=sorted(FORMATS), default="fp8")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--rope", type=float, metavar="BASE", help="rotate queries and keys by their positions")
    ap.add_argument("--norm", action="store_true", help="norm each head of queries and keys")
    ap.add_argument("--softcap", type=float, default=0.0)
    ap.add_argument("--slopes", action="store_true", help="scores fall with distance (no draft tree)")
    ap.add_argument("--pool", type=int, metavar="PAGES", help="pages that the sequences share")
    a = ap.parse_args(argv)
    hidden, counts = 1024, [700, 333]
    layer = AttentionLayer(hidden, 8, 2, 128, 2, 1024, FORMATS[a.format], window=a.window, sinks=a.sinks,
                           rope_base=a.rope, norm=a.norm, softcap=a.softcap, slopes=a.slopes, pool_pages=a.pool)
    rows = lambda n, seed: torch.from_numpy(synth.activations(n, hidden, "f32", seed)).to("cuda:0", layer.dtype)  # noqa: E731
    y = layer.extend(rows(sum(counts), 2), counts)
    print(f"prompts of {counts} tokens: {tuple(y.shape)}, cache {layer.cache.nbytes / 2 ** 20:.1f} MiB in {a.format}")
    for step in range(4):
        y = layer.extend(rows(2, 3 + step), [1, 1])
    print(f"4 decode steps: {tuple(y.shape)}, lengths {layer.lens}")
    if not a.window and not a.slopes:
        parents = [[-1, 0, 0, 1, 2], [-1, -1, 0]]
        y = layer.check(rows(8, 9), parents)
        layer.accept([[0, 2, 4], [1]])
        print(f"trees of {[len(p) for p in parents]} drafted tokens: {tuple(y.shape)}, lengths {layer.lens}")
    at = torch.arange(layer.lens[0], device=layer.table.device)
    k, _ = ops.kv_cache_read(layer.cache, layer.table[0, at // layer.page_size].long() * layer.page_size + at % layer.page_size)
    print(f"keys read back: {tuple(k.shape)}, largest {k.abs().max().item():.3f}")
    return layer


if __name__ == "__main__":
    main()
