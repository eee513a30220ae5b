"""Host-side checks of the page pool's and the rotary entry points, and pins of their plain references (no GPU needed)."""
import ctypes
import math
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

import kv_step_ref as ref
from test_kv_cpu import BF16, E_ALIGN, E_DTYPE, E_NULL, E_SHAPE, F16, F32, I8, OK, P, Cache, cache

VP, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


@pytest.fixture(scope="module")
def L():
    from bit_gemm_w4_amd import build, ops
    if not os.path.exists(ops.LIB_PATH):
        build.build()
    return ops.lib()


class Pool(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("block_table", "lens", "gone", "free_pages", "state")] + \
               [(n, I64) for n in ("batch", "max_pages", "pages", "window", "sinks")] + [("page_size", I32)]


class Rope(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("q", "k", "v", "q_out", "k_out")] + \
               [(f"{n}_{a}_stride", I64) for n in ("q", "k", "v", "q_out", "k_out") for a in ("token", "head")] + \
               [(n, VP) for n in ("q_weight", "k_weight", "positions", "freqs", "slots")] + \
               [("tokens", I64), ("eps", ctypes.c_double), ("weight_offset", ctypes.c_double)] + \
               [(n, I32) for n in ("q_heads", "kv_heads", "head_dim", "rot", "interleaved", "x_dtype", "weight_dtype")]


def pool(**over):
    a = dict(block_table=P, lens=P, gone=P, free_pages=P, state=P, batch=3, max_pages=4, pages=10, window=0, sinks=0, page_size=16)
    return Pool(**{**a, **over})


def rope(**over):
    a = dict(q=P, k=P, v=P, q_out=P, k_out=P, q_weight=P, k_weight=P, positions=P, freqs=P, slots=P, tokens=5, eps=1e-6, weight_offset=0.0,
             q_heads=8, kv_heads=2, head_dim=128, rot=128, interleaved=0, x_dtype=BF16, weight_dtype=BF16)
    a.update({f"{n}_token_stride": 1024 for n in ("q", "k", "v", "q_out", "k_out")})
    a.update({f"{n}_head_stride": 128 for n in ("q", "k", "v", "q_out", "k_out")})
    return Rope(**{**a, **over})


def test_struct_layouts_match_the_binding():
    from bit_gemm_w4_amd import ops
    for packed, Struct, tail in ((ops._KV_POOL, Pool, ()), (ops._QK_ROPE, Rope, (0.5, 0.25))):
        assert packed.size == ctypes.sizeof(Struct)
        values = list(range(1, len(Struct._fields_) + 1))
        for i, (name, _) in enumerate(Struct._fields_):
            if name in ("eps", "weight_offset"):
                values[i] = tail[name == "weight_offset"]
        s = Struct.from_buffer_copy(packed.pack(*values))
        assert [getattr(s, n) for n, _ in Struct._fields_] == values


BAD_POOLS = [(dict(block_table=None), E_NULL), (dict(lens=None), E_NULL), (dict(free_pages=None), E_NULL), (dict(state=None), E_NULL),
             (dict(gone=None, window=5), E_NULL), (dict(batch=0), E_SHAPE), (dict(batch=65536), E_SHAPE), (dict(page_size=8), E_SHAPE),
             (dict(page_size=48), E_SHAPE), (dict(pages=0), E_SHAPE), (dict(pages=2 ** 30 + 1), E_SHAPE), (dict(max_pages=0), E_SHAPE),
             (dict(max_pages=1 << 27), E_SHAPE), (dict(window=-1), E_SHAPE), (dict(sinks=-1), E_SHAPE), (dict(lens=P + 2), E_ALIGN),
             (dict(state=P + 1), E_ALIGN)]


@pytest.mark.parametrize("over,status", BAD_POOLS)
def test_bad_pools(L, over, status):
    p = pool(**over)
    assert L.kv_plan(ctypes.addressof(p), P, 5, 1, P, P, P, P, P, None) == status
    assert L.bg_last_error().decode().startswith("kv_plan: ")
    assert L.kv_release(ctypes.addressof(p), P, None) == status


def test_plan_and_release_refusals(L):
    p = pool()
    at = ctypes.addressof(p)
    good = [P, 5, 1, P, P, P, P, P]
    for i, bad, status in ((0, None, E_NULL), (3, None, E_NULL), (4, None, E_NULL), (5, None, E_NULL), (6, None, E_NULL), (7, None, E_NULL),
                           (1, -1, E_SHAPE), (1, 2 ** 24 + 1, E_SHAPE), (0, P + 2, E_ALIGN), (6, P + 2, E_ALIGN), (7, P + 4, E_ALIGN)):
        args = list(good)
        args[i] = bad
        assert L.kv_plan(at, *args, None) == status, (i, bad)
    assert L.kv_plan(None, *good, None) == E_NULL
    assert L.kv_release(None, P, None) == E_NULL
    assert L.kv_release(at, P + 2, None) == E_ALIGN


@pytest.mark.parametrize("over,status", [
    (dict(x_dtype=I8), E_DTYPE), (dict(weight_dtype=F16), E_DTYPE), (dict(head_dim=96), E_SHAPE), (dict(rot=-8), E_SHAPE), (dict(rot=136), E_SHAPE),
    (dict(rot=12), E_SHAPE), (dict(q_heads=-1), E_SHAPE), (dict(q_heads=16385), E_SHAPE), (dict(q_heads=0, kv_heads=0), E_SHAPE),
    (dict(tokens=-1), E_SHAPE), (dict(tokens=2 ** 24 + 1), E_SHAPE), (dict(tokens=2 ** 20, q_heads=257), E_SHAPE), (dict(eps=-1.0), E_SHAPE),
    (dict(eps=float("nan")), E_SHAPE), (dict(weight_offset=float("inf")), E_SHAPE), (dict(q=None), E_NULL), (dict(q_out=None), E_NULL),
    (dict(k=None), E_NULL), (dict(k_out=None), E_NULL), (dict(positions=None), E_NULL), (dict(freqs=None), E_NULL), (dict(q=P + 8), E_ALIGN),
    (dict(k_out=P + 8), E_ALIGN), (dict(q_weight=P + 4), E_ALIGN), (dict(positions=P + 2), E_ALIGN), (dict(freqs=P + 4), E_ALIGN),
    (dict(q_token_stride=1028), E_ALIGN), (dict(k_head_stride=130), E_ALIGN), (dict(k_out_head_stride=4), E_ALIGN),
    (dict(x_dtype=F32, weight_dtype=F32, q_out_token_stride=2), E_ALIGN)])
def test_rope_refusals(L, over, status):
    a = rope(**over)
    assert L.qk_norm_rope(ctypes.addressof(a), None) == status
    assert L.bg_last_error().decode().startswith("qk_norm_rope: ")


def test_rope_write_refusals(L):
    c = cache()
    call = lambda **over: L.kv_cache_write_rope(ctypes.addressof(c), ctypes.addressof(rope(**over)), None)  # noqa: E731
    for over, status in ((dict(slots=None), E_NULL), (dict(v=None), E_NULL), (dict(v=P + 8), E_ALIGN), (dict(slots=P + 4), E_ALIGN),
                         (dict(v_token_stride=4), E_ALIGN), (dict(rot=12), E_SHAPE)):
        assert call(**over) == status, over
    assert L.kv_cache_write_rope(ctypes.addressof(c), None, None) == E_NULL
    assert L.kv_cache_write_rope(None, ctypes.addressof(rope()), None) == E_NULL
    bad = cache(head_dim=96)
    assert L.kv_cache_write_rope(ctypes.addressof(bad), ctypes.addressof(rope()), None) == E_SHAPE


def test_nothing_to_turn(L):
    none = dict(q=None, k=None, v=None, q_out=None, k_out=None, positions=None, freqs=None, slots=None)
    a = rope(tokens=0, **none)
    assert L.qk_norm_rope(ctypes.addressof(a), None) == OK
    c = cache()
    assert L.kv_cache_write_rope(ctypes.addressof(c), ctypes.addressof(a), None) == OK
    assert isinstance(c, Cache)


def test_frequencies_are_the_nearest_turns():
    from bit_gemm_w4_amd import ops
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    inv = [1.0, 0.1, 10000.0 ** -0.75, 2.0 ** -40, 100.0, 0.0]
    got = ops.rope_freqs(inv)
    assert got.dtype == torch.int64
    for x, f in zip(inv, got.tolist()):
        exact = Fraction(x) * 2 ** 63 / pi
        off = (f - exact) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 10 ** 6)
    assert torch.equal(ops.rope_freqs(torch.tensor(inv, dtype=torch.float64)), got)
    with pytest.raises(ValueError):
        ops.rope_freqs([float("nan")])


def test_python_refuses_host_pools():
    from bit_gemm_w4_amd import ops
    with pytest.raises(ValueError, match="device tensors"):
        ops.kv_pool(4, 16, 2, 2, device="cpu")
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="lens"):
        ops.KVPool(z(2, 3), z(3), z(2), z(5), z(2), 16)
    with pytest.raises(ValueError, match="free"):
        ops.KVPool(z(2, 3), z(2), z(2), z(5).long(), z(2), 16)
    with pytest.raises(ValueError, match="page_size"):
        ops.KVPool(z(2, 3), z(2), z(2), z(5), z(2), 17)


def test_a_copied_pool_describes_its_own_tensors(monkeypatch):
    import copy
    import pickle
    from bit_gemm_w4_amd import ops
    monkeypatch.setattr(ops, "_ptr", lambda t: ctypes.c_void_p(t.data_ptr()))       # host tensors, never launched on
    a = ops.kv_pool(9, 32, 2, 3, window=7, sinks=1, device="cpu")
    for b in (copy.deepcopy(a), pickle.loads(pickle.dumps(a)), copy.copy(a)):
        d = Pool.from_address(b.address)
        assert (d.block_table, d.lens, d.gone, d.free_pages, d.state) == tuple(t.data_ptr() for t in b._tensors)
        assert (d.batch, d.max_pages, d.pages, d.window, d.sinks, d.page_size) == (2, 3, 9, 7, 1, 32) and b.address != a.address


# ---- pins of the plain references ----

def test_reference_pool():
    r = ref.Pool(6, 16, 2, 4)
    cu, kv, served, positions, slots, have = r.plan([20, 3], 25)
    assert (cu, kv, served) == ([0, 20, 23], [20, 3], [1, 1]) and have == [[0, 1], [2]]
    assert positions == [*range(20), 0, 1, 2, 0, 0] and slots == [*range(20), 32, 33, 34, -1, -1]
    assert r.free == [5, 4, 3]
    assert r.plan([40, 0, ], 50, advance=False)[5] == [[0, 1, 3, 4], [2]] and r.free == [5, 4, 3]
    r.release([16, 0])
    assert r.held == [[0], []] and r.free == [5, 4, 3, 2, 1]
    w = ref.Pool(20, 16, 1, 20, window=20, sinks=17)
    w.plan([100], 100)
    w.release()           # the next query at 100 sees 81 and later, and 0 to 16
    assert w.held == [[0, 1, None, None, None, 5, 6]]


def test_reference_turn():
    x = np.zeros((2, 1, 8))
    x[:, 0, 0], x[:, 0, 6] = 1.0, 5.0
    y = ref.turn(x, None, [1, 2], [2 ** 62, 2 ** 61])
    assert np.allclose(y[0, 0], [0, 0, 1, 0, 0, 0, 5, 0]) and np.allclose(y[1, 0], [-1, 0, 0, 0, 0, 0, 5, 0])
    y = ref.turn(x, None, [1, 2], [2 ** 62, 2 ** 61], interleaved=True)
    assert np.allclose(y[0, 0], [0, 1, 0, 0, 0, 0, 5, 0])
    y = ref.turn(np.full((1, 1, 4), 3.0), np.full(4, 0.5), [0], [], eps=7.0, offset=1.0)
    assert np.allclose(y, 3 / math.sqrt(16) * 1.5)
    assert F32 == 0


# ---- attention with other scores ----

class Scores(ctypes.Structure):
    _fields_ = [("slopes", VP), ("prefix_lens", VP), ("softcap", ctypes.c_float)]


def test_scores_are_checked(L):
    from test_kv_cpu import E_UNSUP, E_WS, attn
    from bit_gemm_w4_amd import ops
    assert ops._KV_SCORES.size == ctypes.sizeof(Scores)
    c = cache()
    call = lambda a, s: L.kv_attn_scored(ctypes.addressof(a), ctypes.addressof(s), P, 1 << 40, None)  # noqa: E731
    a, tree = attn(c), attn(c, tree_words=1, tree=P)
    for s, status in ((Scores(None, None, -1.0), E_SHAPE), (Scores(None, None, float("nan")), E_SHAPE), (Scores(None, None, 2e30), E_SHAPE),
                      (Scores(P + 2, None, 1.0), E_ALIGN), (Scores(None, P + 1, 1.0), E_ALIGN)):
        assert call(a, s) == status
        assert L.bg_last_error().decode().startswith("kv_attn_scored: ")
    assert call(tree, Scores(P, None, 0.0)) == E_UNSUP and call(tree, Scores(None, P, 1.0)) == E_UNSUP
    assert L.kv_attn_scored(ctypes.addressof(a), None, P, 1 << 40, None) == E_NULL
    assert L.kv_attn_scored(None, ctypes.addressof(Scores()), P, 1 << 40, None) == E_NULL
    assert call(attn(c, max_q=0), Scores(None, None, 1.0)) == E_SHAPE
    assert call(attn(c, tokens=0), Scores(P, P, 1.0)) == OK
    big = cache(pages=100000, kv_heads=8)
    long = attn(big, tokens=1, batch=1, max_q=1, cu_q=None, q_heads=32, max_pages=8192)
    assert L.kv_attn_scored(ctypes.addressof(long), ctypes.addressof(Scores(P, None, 0.0)), None, 0, None) == E_WS


def test_tree_depths():
    from bit_gemm_w4_amd.attention_layer import tree_depths
    assert tree_depths([-1, 0, 0, 2, -1, 4]) == [0, 1, 1, 2, 0, 1] and tree_depths([]) == []
