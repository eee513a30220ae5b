"""Host-side checks of the KV cache's entry points, and the pins of its plain reference (no GPU needed)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import kv_ref as ref

OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE, E_UNSUP, E_HIP, E_WS = range(8)
F32, F16, BF16, I8, FP8, I32, U4 = range(7)
P = 0x10000          # fake, 16-byte aligned device address


@pytest.fixture(scope="module")
def L():
    from bit_gemm_w4_amd import build, ops
    if not os.path.exists(ops.LIB_PATH):
        build.build()
    return ops.lib()


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class Attn(ctypes.Structure):
    _fields_ = [("cache", ctypes.c_void_p), ("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int64),
                ("kv_lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("tree", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("tokens", ctypes.c_int64), ("batch", ctypes.c_int64), ("max_q", ctypes.c_int64),
                ("max_kv", ctypes.c_int64), ("window", ctypes.c_int64), ("sinks", ctypes.c_int64), ("q_heads", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("tree_words", ctypes.c_int32), ("scale", ctypes.c_float)]


def cache(**over):
    c = dict(k=P, v=P, k_scales=P, v_scales=P, pages=10, page_size=16, kv_heads=2, head_dim=128, format=I8)
    c.update(over)
    return Cache(**c)


def attn(c, **over):
    a = dict(cache=ctypes.addressof(c) if c is not None else None, q=P, q_token_stride=1024, q_head_stride=128, block_table=P,
             max_pages=5, kv_lens=P, cu_q=P, tree=None, out=P, lse=None, tokens=7, batch=2, max_q=4, max_kv=0, window=0, sinks=0,
             q_heads=8, dtype=BF16, tree_words=0, scale=0.1)
    a.update(over)
    return Attn(**a)


BAD_CACHES = [(dict(k=None), E_NULL), (dict(v_scales=None), E_NULL), (dict(format=F16), E_DTYPE), (dict(head_dim=96), E_SHAPE),
              (dict(kv_heads=0), E_SHAPE), (dict(page_size=8), E_SHAPE), (dict(page_size=48), E_SHAPE),
              (dict(page_size=2048), E_SHAPE), (dict(pages=0), E_SHAPE), (dict(pages=1 << 31), E_SHAPE), (dict(v=P + 8), E_ALIGN),
              (dict(k_scales=P + 4), E_ALIGN)]


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_every_entry_point_refuses_a_bad_cache(L, over, status):
    c = cache(**over)
    at = ctypes.addressof(c)
    assert L.kv_cache_write(at, P, 256, 128, P, 256, 128, BF16, P, 3, None) == status
    assert L.kv_cache_read(at, P, 3, P, P, BF16, None) == status
    a = attn(c)
    assert L.kv_attn(ctypes.addressof(a), P, 1 << 40, None) == status
    assert L.kv_attn_workspace_bytes(ctypes.addressof(a)) == 0


def test_write_and_read_refusals(L):
    c = cache()
    at, w, r = ctypes.addressof(c), L.kv_cache_write, L.kv_cache_read
    assert w(None, P, 256, 128, P, 256, 128, BF16, P, 3, None) == E_NULL
    assert w(at, None, 256, 128, P, 256, 128, BF16, P, 3, None) == E_NULL
    assert w(at, P, 256, 128, P, 256, 128, BF16, None, 3, None) == E_NULL
    assert w(at, P, 256, 128, P, 256, 128, I8, P, 3, None) == E_DTYPE
    assert w(at, P, 256, 128, P, 256, 128, BF16, P, -1, None) == E_SHAPE
    assert w(at, P, 252, 128, P, 256, 128, BF16, P, 3, None) == E_ALIGN
    assert w(at, P, 256, 128, P, 256, 124, BF16, P, 3, None) == E_ALIGN
    assert w(at, P, 256, 128, P + 8, 256, 128, BF16, P, 3, None) == E_ALIGN
    assert w(at, P, 256, 128, P, 256, 128, BF16, P + 4, 3, None) == E_ALIGN
    assert w(at, P, 256, 128, P, 256, 126, F32, P, 3, None) == E_ALIGN
    assert w(at, None, 256, 128, None, 256, 128, BF16, None, 0, None) == OK       # nothing to write
    assert r(at, P, 3, None, P, BF16, None) == E_NULL
    assert r(at, P, 3, P, P, I32, None) == E_DTYPE
    assert r(at, P, 1 << 25, P, P, BF16, None) == E_SHAPE
    assert r(at, P, 3, P, P + 2, BF16, None) == E_ALIGN
    assert r(at, None, 0, None, None, BF16, None) == OK


@pytest.mark.parametrize("over,status", [
    (dict(q=None), E_NULL), (dict(out=None), E_NULL), (dict(kv_lens=None), E_NULL), (dict(block_table=None), E_NULL),
    (dict(dtype=F32), E_DTYPE), (dict(tokens=-1), E_SHAPE), (dict(tokens=1 << 25), E_SHAPE), (dict(batch=65536), E_SHAPE),
    (dict(q_heads=7), E_SHAPE), (dict(q_heads=1), E_SHAPE), (dict(max_pages=0), E_SHAPE), (dict(max_pages=1 << 27), E_SHAPE),
    (dict(max_q=0), E_SHAPE), (dict(max_kv=-1), E_SHAPE), (dict(window=-1), E_SHAPE), (dict(sinks=-4), E_SHAPE),
    (dict(q_token_stride=1028), E_ALIGN), (dict(q_head_stride=130), E_ALIGN), (dict(q=P + 8), E_ALIGN), (dict(out=P + 2), E_ALIGN),
    (dict(lse=P + 2), E_ALIGN), (dict(kv_lens=P + 1), E_ALIGN), (dict(scale=0.0), E_SHAPE), (dict(scale=-1.0), E_SHAPE),
    (dict(scale=float("nan")), E_SHAPE), (dict(scale=float("inf")), E_SHAPE), (dict(cu_q=None), E_SHAPE),
    (dict(cu_q=None, tokens=2), E_SHAPE)])
def test_attention_refusals(L, over, status):
    c = cache()
    a = attn(c, **over)
    assert L.kv_attn(ctypes.addressof(a), P, 1 << 40, None) == status
    assert L.bg_last_error().decode().startswith("kv_attn: ")


def test_tree_refusals(L):
    c = cache()
    for over, status in ((dict(tree_words=0, tree=P), E_SHAPE), (dict(tree_words=1, tree=None), E_NULL),
                         (dict(tree_words=1, tree=P + 4), E_ALIGN), (dict(tree_words=1, tree=P, window=5), E_UNSUP)):
        a = attn(c, **over)
        assert L.kv_attn_tree(ctypes.addressof(a), P, 1 << 40, None) == status, over


def test_nothing_to_attend(L):
    c = cache()
    for over in (dict(tokens=0), dict(batch=0)):
        a = attn(c, q=None, out=None, **over)
        assert L.kv_attn(ctypes.addressof(a), None, 0, None) == OK
        assert L.kv_attn_workspace_bytes(ctypes.addressof(a)) == 0


def test_workspace_refusals(L):
    c = cache(pages=100000, kv_heads=8)
    a = attn(c, tokens=1, batch=1, max_q=1, cu_q=None, q_heads=32, max_pages=8192)
    need = L.kv_attn_workspace_bytes(ctypes.addressof(a))
    if need:      # one sequence of 131072 positions is split
        assert L.kv_attn(ctypes.addressof(a), None, 0, None) == E_WS
        assert L.kv_attn(ctypes.addressof(a), P, need - 1, None) == E_WS
        assert L.kv_attn(ctypes.addressof(a), P + 8, need, None) == E_ALIGN


def test_python_refuses_host_tensors_and_wrong_shapes():
    from bit_gemm_w4_amd import ops
    z = lambda *s, dt=torch.int8: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="device tensors"):
        ops.KVCache(z(2, 1, 16, 64), z(2, 1, 16, 64), z(2, 1, 16, dt=torch.float32), z(2, 1, 16, dt=torch.float32), ops.I8)
    with pytest.raises(ValueError, match="scales"):
        ops.KVCache(z(2, 1, 16, 64), z(2, 1, 16, 64), z(2, 1, 8, dt=torch.float32), z(2, 1, 16, dt=torch.float32), ops.I8)
    with pytest.raises(ValueError, match="head size"):
        ops.KVCache(z(2, 1, 16, 32), z(2, 1, 16, 32), z(2, 1, 16, dt=torch.float32), z(2, 1, 16, dt=torch.float32), ops.I8)
    with pytest.raises(ValueError, match="page_size"):
        ops.KVCache(z(2, 1, 24, 64), z(2, 1, 24, 64), z(2, 1, 24, dt=torch.float32), z(2, 1, 24, dt=torch.float32), ops.I8)
    with pytest.raises(ValueError, match="k and v"):
        ops.KVCache(z(2, 1, 16, 64), z(2, 1, 16, 64), z(2, 1, 16, dt=torch.float32), z(2, 1, 16, dt=torch.float32), ops.FP8_E4M3)
    with pytest.raises(ValueError, match="format"):
        ops.kv_cache(2, 16, 1, 64, ops.F16, device="cpu")


def test_struct_layouts_match_the_header():
    from bit_gemm_w4_amd import ops
    assert ops._KV_CACHE.size == ctypes.sizeof(Cache)
    assert ops._KV_ATTN.size == ctypes.sizeof(Attn)
    a = Attn.from_buffer_copy(ops._KV_ATTN.pack(*range(1, 21), 0.5))
    assert [getattr(a, n) for n, _ in Attn._fields_] == [*range(1, 21), 0.5]


# ---- pins of the plain reference ----

def test_e4m3_reference_matches_torch():
    x = np.concatenate((np.linspace(-460, 460, 20001), np.geomspace(2.0 ** -12, 448, 5000))).astype(np.float32)
    t = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(ref.e4m3_encode(x), t.view(torch.uint8).numpy())
    b = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(want), np.isnan(ref.e4m3_decode(b)))
    assert np.array_equal(want[~np.isnan(want)], ref.e4m3_decode(b)[~np.isnan(want)])


@pytest.mark.parametrize("fmt", [I8, FP8, U4])
def test_reference_round_trip_bounds(fmt):
    x = np.random.default_rng(0).standard_normal((200, 64)).astype(np.float32)
    code, s, z = ref.quantize(x, fmt)
    err = np.abs(ref.values(code, s, z, fmt) - x)
    if fmt == I8:
        bound = s[:, None] * (0.5 + 1e-4) + 0 * x
    elif fmt == U4:
        bound = s[:, None] * (1.0 + 1e-2) + 0 * x       # the ends: half a step of the value, half of the zero-point
    else:
        bound = np.maximum(np.abs(x) * 2.0 ** -4, s[:, None] * 2.0 ** -10) * (1 + 1e-4)
    assert (err <= bound).all()
    assert np.array_equal(ref.unpack_u4(ref.pack_u4(code)), code) if fmt == U4 else True


def test_reference_masks():
    see = ref.visible(3, 10, np.ones(10, bool), window=4, sinks=2)
    assert [list(np.flatnonzero(r)) for r in see] == [[0, 1, 4, 5, 6, 7], [0, 1, 5, 6, 7, 8], [0, 1, 6, 7, 8, 9]]
    see = ref.visible(3, 5, np.array([1, 1, 0, 1, 1], bool), tree=[1, 0b11, 0b101])
    assert [list(np.flatnonzero(r)) for r in see] == [[0, 1], [0, 1, 3], [0, 1, 4]]
    assert not ref.visible(4, 2, np.ones(2, bool))[:2].any()


def test_tree_bits():
    from bit_gemm_w4_amd.attention_layer import tree_bits
    assert tree_bits([-1, 0, 0, 2, -1]) == [[1], [3], [5], [13], [16]]
    chain = tree_bits([i - 1 for i in range(70)])
    assert chain[63] == [-1, 0] and chain[69] == [-1, 63] and chain[62] == [(1 << 63) - 1, 0]
    with pytest.raises(ValueError, match="parent"):
        tree_bits([-1, 1])


def test_tokens_times_heads_are_bounded(L):
    c = cache(kv_heads=1)
    a = attn(c, tokens=1 << 20, q_heads=512, cu_q=P)
    assert L.kv_attn(ctypes.addressof(a), P, 1 << 40, None) == E_SHAPE


def test_positions_leave_room_for_a_window_in_32_bits(L):
    for shift in (4, 6, 10):
        c = cache(page_size=1 << shift)
        most = (2 ** 31 - 1 - 2 ** 25) >> shift
        for pages, status in ((most, E_WS), (most + 1, E_SHAPE)):       # E_WS: past the sizes' checks
            a = attn(c, tokens=1, batch=1, max_q=1, cu_q=None, max_pages=pages)
            assert L.kv_attn(ctypes.addressof(a), None, 0, None) == status


def test_workspace_follows_the_split(L):
    """Many rows of a short sequence, or more blocks than the device holds at once, need none; it grows with neither pages nor window alone."""
    c = cache(pages=100000, kv_heads=8)

    def need(**kw):
        a = attn(c, **{**dict(q_heads=32, max_pages=8192), **kw})
        return L.kv_attn_workspace_bytes(ctypes.addressof(a))
    assert need(tokens=64, batch=64, max_q=1, max_kv=200) == 0
    assert need(tokens=4096, batch=1, max_q=4096, max_kv=65536) == 0
    one = need(tokens=1, batch=1, max_q=1, max_kv=131072)
    assert one > 0 and one % (32 * 129 * 4) == 0
    assert need(tokens=1, batch=1, max_q=1, max_kv=131072, window=4096) < one


@pytest.mark.parametrize("how", ["deepcopy", "copy", "pickle", "replace"])
def test_a_copied_cache_describes_its_own_tensors(monkeypatch, how):
    """The descriptor that the library reads holds the addresses of the copy's tensors."""
    import copy
    import dataclasses
    import pickle
    from bit_gemm_w4_amd import ops
    monkeypatch.setattr(ops, "_ptr", lambda t: ctypes.c_void_p(t.data_ptr()))       # host tensors, never launched on
    for fmt in (I8, FP8, U4):
        a = ops.kv_cache(2, 16, 1, 64, fmt, device="cpu")
        b = {"deepcopy": copy.deepcopy, "copy": copy.copy, "pickle": lambda c: pickle.loads(pickle.dumps(c)),
             "replace": lambda c: dataclasses.replace(c, v=c.v.clone())}[how](a)
        for c in (a, b):
            d = Cache.from_address(c.address)
            assert (d.k, d.v, d.k_scales, d.v_scales) == tuple(t.data_ptr() for t in (c.k, c.v, c.k_scales, c.v_scales))
            assert (d.pages, d.page_size, d.kv_heads, d.head_dim, d.format) == (2, 16, 1, 64, fmt)
        assert a.address != b.address and (b.v.data_ptr() != a.v.data_ptr()) == (how != "copy")
        del a
        assert Cache.from_address(b.address).v == b.v.data_ptr()


def test_a_long_sequence_alone_needs_a_workspace(L):
    c = cache(pages=100000, kv_heads=8)
    a = attn(c, tokens=1, batch=1, max_q=1, cu_q=None, q_heads=32, max_pages=8192)
    need = L.kv_attn_workspace_bytes(ctypes.addressof(a))
    assert need > 0
    assert L.kv_attn(ctypes.addressof(a), None, 0, None) == E_WS
    assert L.kv_attn(ctypes.addressof(a), P, need - 1, None) == E_WS
    assert L.kv_attn(ctypes.addressof(a), P + 8, need, None) == E_ALIGN
