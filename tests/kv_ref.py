"""The KV cache and the attention over it, plainly and in binary64 (numpy).

Shares no code with the library.  Rows quantize by the readings the other
oracles pin: symmetric INT8 s = amax / 127, E4M3 s = amax / 448, 4-bit
s = fp16((max - min) / 15) with the range widened to hold 0; binary32 quotients,
round half to even; an all-zero row (or a scale that underflows) has s = 1.
"""
import numpy as np

I8, FP8, U4 = 3, 4, 6
F = np.float32


def e4m3_decode(b):
    b = np.asarray(b, np.uint8).astype(np.int64)
    e, m = b >> 3 & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def e4m3_encode(x):
    """Nearest finite E4M3 byte, ties to the even code, saturating."""
    table = e4m3_decode(np.arange(127))
    a = np.abs(np.asarray(x, np.float64))
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 448.0, 126, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantize(x, fmt):
    """x [..., D] float32 -> codes (unpacked, one per element), scale, zero (0 but for U4)."""
    x = np.asarray(x, F)
    bad = ~np.isfinite(x).all(-1, keepdims=True)
    y = np.where(bad, F(0), x)
    if fmt == U4:
        lo = np.minimum(y.min(-1, keepdims=True), F(0))
        hi = np.maximum(y.max(-1, keepdims=True), F(0))
        s = np.clip((hi - lo) / F(15), F(2.0 ** -24), F(65504)).astype(np.float16).astype(F)
        s = np.where(hi == lo, F(1), s)
        z = np.clip(np.rint(-lo / s), 0, 15).astype(F)
        code = np.clip(np.rint(y / s) + z, 0, 15).astype(np.uint8)
        code, z = np.where(bad, 0, code).astype(np.uint8), np.where(bad, F(0), z)
    else:
        s = (np.abs(y).max(-1, keepdims=True) / F(127 if fmt == I8 else 448)).astype(F)
        s = np.where(s == 0, F(1), s)
        with np.errstate(over="ignore"):
            t = (y / s).astype(F)
        code = np.clip(np.rint(t), -127, 127).astype(np.int8) if fmt == I8 else e4m3_encode(t)
        z = np.zeros_like(s)
    return code, np.where(bad, F(np.nan), s)[..., 0], z[..., 0]


def values(code, scale, zero, fmt):
    """binary64 values of codes."""
    c = e4m3_decode(code) if fmt == FP8 else code.astype(np.float64) - zero[..., None].astype(np.float64)
    return c * scale[..., None].astype(np.float64)


def pack_u4(code):
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8)


def unpack_u4(b):
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)


def visible(q_len, kv_len, held, window=0, sinks=0, tree=None):
    """[q_len][kv_len] truth values; held [kv_len]: the position's page exists; tree: rows of Python ints."""
    j = np.arange(kv_len)
    first = kv_len - q_len
    see = np.zeros((q_len, kv_len), bool)
    for i in range(q_len):
        at = first + i
        if tree is None:
            see[i] = (j <= at) & ((j > at - window) | (j < sinks)) if window else j <= at
        else:
            see[i] = j < first
            for e in range(max(0, -first), q_len):
                see[i, first + e] = bool(tree[i] >> e & 1)
    return see & held[None]


def attend(q, k, v, see, scale):
    """One sequence and head: q [n][D], k and v [L][D], see [n][L] -> out, lse, and the bound's two parts:
    mean |v| under the weights and the largest sum of |q k| scale over visible positions."""
    n, length = see.shape
    out, lse = np.zeros_like(q), np.full(n, -np.inf)
    mean, top = np.zeros_like(q), np.zeros(n)
    for i in range(n):
        at = np.flatnonzero(see[i])
        if not at.size:
            continue
        s = k[at] @ q[i] * scale
        m = s.max()
        p = np.exp(s - m)
        l = p.sum()
        out[i], lse[i] = p @ v[at] / l, m + np.log(l)
        mean[i] = p @ np.abs(v[at]) / l
        top[i] = (np.abs(k[at]) @ np.abs(q[i])).max() * scale
    return out, lse, mean, top
