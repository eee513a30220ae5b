"""Operands that share memory: the host's test of it against every byte (no GPU needed), and the calls it refuses."""
import ctypes
import os
import random
import subprocess

import pytest

from test_kv_cpu import BF16, E_UNSUP, F32, P, cache
from test_kv_steps_cpu import L, rope  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "bg_overlap.h"
static bg::RowSet set(const long long* x) { return bg::RowSet((const void*)x[0], x[1], x[2], x[3], x[4], x[5]); }
extern "C" int rows_apart(const long long* a, const long long* b) { return bg::apart(set(a), set(b)); }
extern "C" int rows_distinct(const long long* a) { return set(a).distinct(); }
extern "C" int rows_same(const long long* a, const long long* b) { return set(a).same(set(b)); }
extern "C" int spans_apart(long long a, long long n, long long b, long long m) { return bg::apart(bg::Span((const void*)a, n), bg::Span((const void*)b, m)); }
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "bit_gemm_w4_amd", "csrc"), str(d / "shim.cpp"), "-o",
                    str(d / "shim.so")], check=True)
    return ctypes.CDLL(str(d / "shim.so"))


def words(rows):
    return (ctypes.c_longlong * 6)(*rows)


def bytes_of(rows):
    at, tokens, ts, heads, hs, run = rows
    return [at + t * ts + h * hs + i for t in range(tokens) for h in range(heads) for i in range(run)]


def test_rows_against_every_byte(shim):
    rng = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(20000):
        strides = [rng.choice([0, 1, 2, 3, 4, 6, 8, 12, 24, -4, -12]) for _ in range(4)]
        if rng.random() < 0.6:
            strides[2:] = strides[:2]
        tokens = rng.choice([1, 2, 3, 5])
        a = (1000 + rng.randrange(30), tokens, strides[0], rng.choice([1, 2, 3]), strides[1], rng.choice([1, 2, 4]))
        b = (1000 + rng.randrange(30), tokens, strides[2], rng.choice([1, 2, 3]), strides[3], a[5])
        x, y = bytes_of(a), bytes_of(b)
        said = bool(shim.rows_apart(words(a), words(b)))
        assert said == bool(shim.rows_apart(words(b), words(a)))
        if said:
            assert not set(x) & set(y), (a, b)
        seen[said] += 1
        if shim.rows_distinct(words(a)):
            assert len(set(x)) == len(x), a
        if shim.rows_same(words(a), words(b)):
            assert set(x) == set(y)
    assert min(seen.values()) > 1000


D = 256          # bytes of a row


@pytest.mark.parametrize("a,b", [
    ((0, 7, 12 * D, 8, D, D), (8 * D, 7, 12 * D, 2, D, D)),                  # queries and keys of fused rows
    ((8 * D, 7, 12 * D, 2, D, D), (10 * D, 7, 12 * D, 2, D, D)),             # keys and values of fused rows
    ((0, 7, 12 * D, 8, D, D), (8 * D, 7, 12 * D, 1, 0, D)),                  # one key head
    ((0, 1, 0, 8, D, D), (8 * D, 1, 0, 2, D, D)),                            # one token
    ((0, 7, 9 * D, 3, 3 * D, D), (D, 7, 9 * D, 3, 3 * D, D)),                # [tokens][heads][q, k, v]
    ((D, 7, 9 * D, 3, 3 * D, D), (2 * D, 7, 9 * D, 3, 3 * D, D)),
    ((0, 7, D, 4, 7 * D, D), (28 * D, 7, D, 2, 7 * D, D)),                   # heads before tokens
    ((0, 7, D, 4, 14 * D, D), (7 * D, 7, D, 4, 14 * D, D)),                  # [heads][q, k][tokens]
    ((0, 7, 8 * D, 8, D, D), (56 * D, 7, 2 * D, 2, D, D)),                   # buffers of their own, next to each other
])
def test_layouts_that_are_apart(shim, a, b):
    assert shim.rows_apart(words(a), words(b)) and shim.rows_apart(words(b), words(a))
    assert shim.rows_distinct(words(a)) and shim.rows_distinct(words(b)) and not set(bytes_of(a)) & set(bytes_of(b))


def test_spans(shim):
    for a, n, b, m, apart in ((100, 10, 110, 5, 1), (100, 11, 110, 5, 0), (110, 5, 100, 10, 1), (105, 0, 100, 10, 1), (100, 10, 100, 10, 0), (100, 10, 103, 2, 0)):
        assert shim.spans_apart(a, n, b, m) == apart


def fused(q_heads=4, kv_heads=4, **over):
    """Rows of queries, keys and values, fused, BF16, in place."""
    width, row = (q_heads + 2 * kv_heads) * 128, 128 * 2
    a = dict(q=P, k=P + q_heads * row, v=P + (q_heads + kv_heads) * row, q_out=P, k_out=P + q_heads * row, q_heads=q_heads, kv_heads=kv_heads)
    a.update({f"{n}_token_stride": width for n in ("q", "k", "v", "q_out", "k_out")})
    return rope(**{**a, **over})


ROW, FAR = 256, 1 << 30
OVERLAPS = [
    dict(q_out=P + 4 * ROW, k_out=P),                                            # the two exchanged
    dict(q_out=P + 4 * ROW, k_out=FAR), dict(k_out=P, q_out=FAR),                # one into the other's rows
    dict(q_out=FAR, k_out=FAR), dict(q_out=FAR, k_out=FAR + 3 * ROW),            # both into one buffer
    dict(q_out=P + ROW, k_out=FAR), dict(q_out=P + 12 * ROW, k_out=FAR),         # a head or a token further on
    dict(q_out=P, q_out_token_stride=4 * 128, k_out=FAR),                        # the same place, other strides
    dict(q_out=FAR, q_out_token_stride=0, k_out=FAR << 1), dict(q_out=FAR, q_out_head_stride=64, k_out=FAR << 1),       # rows in one another
]


@pytest.mark.parametrize("over", OVERLAPS)
def test_overlapping_outputs_are_refused(L, over):  # noqa: F811
    assert L.qk_norm_rope(ctypes.addressof(fused(**over)), None) == E_UNSUP
    assert L.bg_last_error().decode().startswith("qk_norm_rope: ")


def test_overlapping_outputs_into_the_cache_are_refused(L):  # noqa: F811
    c = cache(kv_heads=4, k=FAR, v=FAR, k_scales=FAR, v_scales=FAR)
    for q_out in (P + 4 * ROW, P + 8 * ROW, P + ROW):                           # keys, values, queries a head further on
        assert L.kv_cache_write_rope(ctypes.addressof(c), ctypes.addressof(fused(q_out=q_out)), None) == E_UNSUP
    a = fused(x_dtype=F32, weight_dtype=F32, q_out=P + 4 * ROW)
    assert L.kv_cache_write_rope(ctypes.addressof(c), ctypes.addressof(a), None) == E_UNSUP
    assert BF16 != F32


def plan_args(**over):
    """A plan of 3 sequences and 5 rows whose operands lie apart."""
    a = dict(q_lens=P, cu_q=P + 0x1000, kv_lens=P + 0x2000, served=P + 0x3000, positions=P + 0x4000, slots=P + 0x5000)
    a.update(over)
    return [a["q_lens"], 5, 1, a["cu_q"], a["kv_lens"], a["served"], a["positions"], a["slots"]]


def apart_pool():
    from test_kv_steps_cpu import pool
    return pool(block_table=FAR, lens=FAR + 0x1000, gone=FAR + 0x2000, free_pages=FAR + 0x3000, state=FAR + 0x4000)


@pytest.mark.parametrize("over", [
    dict(q_lens=P + 0x3000), dict(q_lens=P + 0x2000), dict(q_lens=P + 0x1000), dict(q_lens=P + 0x5000 + 36),      # a plan's own output as its input
    dict(kv_lens=P + 0x3000), dict(cu_q=P + 0x2000 - 12), dict(positions=P + 0x5000 - 16),                       # outputs in one another
    dict(kv_lens=FAR + 0x1000), dict(served=FAR + 0x2000), dict(slots=FAR + 0x3000), dict(cu_q=FAR + 0x4000), dict(positions=FAR + 44),       # in the pool
    dict(q_lens=FAR + 0x1000 + 4), dict(q_lens=FAR), dict(q_lens=FAR + 0x3000 - 8), dict(q_lens=FAR + 0x4000 + 4)])
def test_plans_over_their_own_operands_are_refused(L, over):  # noqa: F811
    p = apart_pool()
    assert L.kv_plan(ctypes.addressof(p), *plan_args(**over), None) == E_UNSUP
    assert L.bg_last_error().decode().startswith("kv_plan: ")


@pytest.mark.parametrize("keep", [FAR + 0x1000 + 4, FAR + 0x1000 - 8, FAR + 0x2000 + 8, FAR + 44, FAR + 0x3000, FAR + 0x4000])
def test_lengths_to_keep_inside_the_pool_are_refused(L, keep):  # noqa: F811
    p = apart_pool()
    assert L.kv_release(ctypes.addressof(p), keep, None) == E_UNSUP
    assert L.bg_last_error().decode().startswith("kv_release: ")
