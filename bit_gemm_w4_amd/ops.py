"""Thin Python binding of ``libbitgemm.so`` (the C ABI in ``include/bitgemm.h``).

Argument marshalling only: every step runs in the HIP kernels behind the C
ABI.  Torch tensors supply device memory and the current HIP stream; the
functions here check dtypes/devices, allocate outputs with torch, pass raw
pointers and raise :class:`BitGemmError` on a non-zero status.  There is no
CPU fallback: if the library is missing, :func:`lib` raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("BG_LIB_PATH") or os.path.join(_PKG, "libbitgemm.so")

# enums of include/bitgemm.h
F32, F16, BF16, I8, FP8_E4M3, I32, U4 = 0, 1, 2, 3, 4, 5, 6
GRAN_TENSOR, GRAN_ROW, GRAN_ROW_G128, GRAN_BLOCK128 = 0, 1, 2, 3
ALGO_AUTO, ALGO_GEMV, ALGO_SKINNY, ALGO_TILED, ALGO_SPLITK, ALGO_MID = 0, 1, 2, 3, 4, 5
PACK_FORMAT_VERSION = 1

EXPORTS = (
    "w4_pack", "gemm_w4a16", "gemm_w4a16_ex", "gemm_w4a16_ws", "gemm_w4a16_noalloc", "gemm_w4a16_workspace_bytes", "act_quant_int8", "act_quant_fp8",
    "act_quant_int8_smooth", "act_quant_fp8_smooth", "act_quant_mxfp8", "gemm_mxfp8", "act_quant_mxfp4", "gemm_mxfp4", "act_quant_int8_outlier", "act_quant_outlier_workspace_bytes",
    "gemm_w8a8_outlier", "gemm_w8a8",
    "gemm_w8a8_ex", "gemm_w8a8_ws", "gemm_w8a8_workspace_bytes", "gemm_w4a8", "gemm_w4a8_ws", "gemm_w4a8_workspace_bytes",
    "gemm_w4a16_algo", "gemm_w8a8_algo",
    "kv_cache_write", "kv_cache_read", "kv_attn", "kv_attn_tree", "kv_attn_workspace_bytes",
    "bg_status_string", "bg_last_error",
    "bg_pack_format_version", "bg_last_kernel",
)

_TORCH_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


class BitGemmError(RuntimeError):
    def __init__(self, status: int, fn: str):
        L = lib()
        self.status = status
        msg = L.bg_last_error().decode() or L.bg_status_string(status).decode()
        super().__init__(f"{fn}: status {status} ({L.bg_status_string(status).decode()}): {msg}")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libbitgemm.so (built in-tree by ``bit_gemm_w4_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m bit_gemm_w4_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        sig = {
            "w4_pack": [P, I, I64, I64, I, I, P, P, P, P],
            "gemm_w4a16": [P, I, I64, I64, P, P, P, I64, I, P, P],
            "gemm_w4a16_ex": [P, I, I64, I64, P, P, P, I64, I, P, I, P],
            "gemm_w4a16_ws": [P, I, I64, I64, P, P, P, I64, I, P, P, I64, I, P],
            "gemm_w4a16_noalloc": [P, I, I64, I64, P, P, P, I64, I, P, P],
            "gemm_w4a16_workspace_bytes": [I64, I64, I64, I],
            "act_quant_int8": [P, I, I64, I64, I, P, P, P],
            "act_quant_fp8": [P, I, I64, I64, I, P, P, P],
            "act_quant_int8_smooth": [P, I, I64, I64, I, P, P, P, P],
            "act_quant_fp8_smooth": [P, I, I64, I64, I, P, P, P, P],
            "act_quant_mxfp8": [P, I, I64, I64, P, P, P],
            "gemm_mxfp8": [P, P, P, P, I64, I64, I64, P, I, P],
            "act_quant_mxfp4": [P, I, I64, I64, P, P, P],
            "gemm_mxfp4": [P, P, P, P, I64, I64, I64, P, I, P],
            "act_quant_int8_outlier": [P, I, I64, I64, ctypes.c_float, P, P, P, P, P, I64, P],
            "gemm_w8a8_outlier": [P, P, P, P, I, P, I, P, P, I64, I64, I64, P, I, P],
            "act_quant_outlier_workspace_bytes": [I64, I64],
            "gemm_w8a8": [P, P, I, P, P, I, I, I64, I64, I64, P, I, P],
            "gemm_w8a8_ex": [P, P, I, P, P, I, I, I64, I64, I64, P, I, I, P],
            "gemm_w8a8_ws": [P, P, I, P, P, I, I, I64, I64, I64, P, I, P, I64, I, P],
            "gemm_w8a8_workspace_bytes": [I64, I64, I64, I, I, I],
            "gemm_w4a8": [P, P, I, I64, I64, P, P, P, I64, I, P, I, P],
            "gemm_w4a8_ws": [P, P, I, I64, I64, P, P, P, I64, I, P, I, P, I64, P],
            "gemm_w4a8_workspace_bytes": [I64, I64, I64],
            "gemm_w4a16_algo": [I64, I64, I64, I],
            "gemm_w8a8_algo": [I64, I64, I64, I],
            "kv_cache_write": [P, P, I64, I64, P, I64, I64, I, P, I64, P],
            "kv_cache_read": [P, P, I64, P, P, I, P],
            "kv_attn": [P, P, I64, P],
            "kv_attn_tree": [P, P, I64, P],
            "kv_attn_workspace_bytes": [P],
            "bg_status_string": [I],
            "bg_last_error": [],
            "bg_pack_format_version": [],
            "bg_last_kernel": [],
        }
        for name, argtypes in sig.items():
            fn = getattr(L, name)
            fn.argtypes = argtypes
            fn.restype = (ctypes.c_char_p if name in ("bg_status_string", "bg_last_error", "bg_last_kernel")
                          else ctypes.c_int64 if name.endswith("_workspace_bytes") else ctypes.c_int)
        _lib = L
    return _lib


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("bitgemm operands must be device tensors")
    if not t.is_contiguous():
        raise ValueError("bitgemm operands must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, fn: str):
    if status != 0:
        raise BitGemmError(status, fn)


def last_kernel() -> str:
    """Kernel instance enqueued by the last successful call on this thread."""
    return lib().bg_last_kernel().decode()


# --------------------------------------------------------------------- W4 ----

@dataclass
class PackedW4:
    """INT4 weights in the tiled w4_pack layout (BG_PACK_FORMAT_VERSION 1):
    one 1 KB tile per (16 output channels, 128-wide group)."""
    qweight: torch.Tensor        # int32 [N/16][K/128][64][4]
    scales: torch.Tensor         # float16 [N/16][K/128][16]
    zeros: torch.Tensor | None   # uint8 [N/16][K/256][16] (two 4-bit zero-points) or None
    N: int
    K: int
    group: int = 128

    @property
    def nbytes(self) -> int:
        z = 0 if self.zeros is None else self.zeros.numel()
        return self.qweight.numel() * 4 + self.scales.numel() * 2 + z


def w4_pack(w: torch.Tensor, group: int = 128, asymmetric: bool = False, stream=None) -> PackedW4:
    N, K = w.shape
    dt = _TORCH_DT.get(w.dtype)
    if dt is None:
        raise ValueError(f"w4_pack: unsupported dtype {w.dtype}")
    if N % 16 or K % 256 or group != 128:
        raise ValueError(f"w4_pack: need N % 16 == 0, K % 256 == 0, group == 128 (N={N}, K={K}, group={group})")
    qweight = torch.empty((N // 16, K // 128, 64, 4), dtype=torch.int32, device=w.device)
    scales = torch.empty((N // 16, K // 128, 16), dtype=torch.float16, device=w.device)
    zeros = torch.empty((N // 16, K // 256, 16), dtype=torch.uint8, device=w.device) if asymmetric else None
    _check(lib().w4_pack(_ptr(w), dt, N, K, group, int(asymmetric), _ptr(qweight), _ptr(scales), _ptr(zeros),
                         _stream(stream)), "w4_pack")
    return PackedW4(qweight, scales, zeros, N, K, group)


_workspaces: dict = {}
_retired: list = []


def workspace(nbytes: int, device) -> torch.Tensor:
    """A device workspace of at least nbytes, cached per device.  It needs no
    initialisation; calls sharing it must not overlap in time (use one per
    stream when streams run concurrently)."""
    key = torch.device(device).index or 0
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        if ws is not None:
            _retired.append(ws)       # HIP graphs captured earlier may still use it
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def gemm_w4a16_workspace_bytes(M: int, N: int, K: int, algo: int = ALGO_AUTO) -> int:
    return int(lib().gemm_w4a16_workspace_bytes(M, N, K, algo))


def gemm_w4a16(x: torch.Tensor, packed: PackedW4, out: torch.Tensor | None = None, algo: int = ALGO_AUTO,
               ws: torch.Tensor | None | bool = None, stream=None) -> torch.Tensor:
    """Y = X W^T.  ws: a workspace tensor, None to use the cached per-device
    workspace (enables the split-K small-M kernel), or False for none."""
    M, K = x.shape
    if K != packed.K:
        raise ValueError(f"gemm_w4a16: x has K={K}, weights K={packed.K}")
    dt = _TORCH_DT.get(x.dtype)
    if dt not in (F16, BF16):
        raise ValueError(f"gemm_w4a16: activations must be float16/bfloat16, got {x.dtype}")
    if out is None:
        out = torch.empty((M, packed.N), dtype=x.dtype, device=x.device)
    L = lib()
    if ws is False:
        _check(L.gemm_w4a16_ex(_ptr(x), dt, M, K, _ptr(packed.qweight), _ptr(packed.scales), _ptr(packed.zeros),
                               packed.N, packed.group, _ptr(out), algo, _stream(stream)), "gemm_w4a16")
        return out
    if ws is None:
        need = gemm_w4a16_workspace_bytes(M, packed.N, K, algo)
        ws = workspace(need, x.device) if need > 0 else None
    _check(L.gemm_w4a16_ws(_ptr(x), dt, M, K, _ptr(packed.qweight), _ptr(packed.scales), _ptr(packed.zeros),
                           packed.N, packed.group, _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(), algo,
                           _stream(stream)), "gemm_w4a16")
    return out


NOALLOC_SCRATCH_BYTES = 16 << 20   # BG_NOALLOC_SCRATCH_BYTES


def gemm_w4a16_noalloc(x: torch.Tensor, packed: PackedW4, out: torch.Tensor, stream=None) -> torch.Tensor:
    """Y = X W^T through gemm_w4a16_noalloc: the split-K partials go to the
    library's static per-device scratch, so the call allocates nothing (the
    caller supplies `out`).  Calls on one GPU must not overlap in time."""
    M, K = x.shape
    if K != packed.K:
        raise ValueError(f"gemm_w4a16_noalloc: x has K={K}, weights K={packed.K}")
    dt = _TORCH_DT.get(x.dtype)
    if dt not in (F16, BF16):
        raise ValueError(f"gemm_w4a16_noalloc: activations must be float16/bfloat16, got {x.dtype}")
    if out.shape != (M, packed.N) or out.dtype != x.dtype:
        raise ValueError(f"gemm_w4a16_noalloc: out must be [{M}, {packed.N}] of {x.dtype}")
    _check(lib().gemm_w4a16_noalloc(_ptr(x), dt, M, K, _ptr(packed.qweight), _ptr(packed.scales),
                                    _ptr(packed.zeros), packed.N, packed.group, _ptr(out), _stream(stream)),
           "gemm_w4a16_noalloc")
    return out


def gemm_w4a16_algo(M: int, N: int, K: int, x_dtype: torch.dtype = torch.bfloat16) -> int:
    return lib().gemm_w4a16_algo(M, N, K, _TORCH_DT[x_dtype])


# ------------------------------------------------------------------- W8A8 ----

def scale_shape(gran: int, rows: int, cols: int):
    return {GRAN_TENSOR: (2,), GRAN_ROW: (rows,), GRAN_ROW_G128: (rows, cols // 128),
            GRAN_BLOCK128: (rows // 128, cols // 128)}[gran]


def _act_quant(fn: str, x: torch.Tensor, gran: int, out_dtype: torch.dtype, stream=None, col_mul=None):
    R, C = x.shape
    dt = _TORCH_DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"{fn}: unsupported dtype {x.dtype}")
    q = torch.empty((R, C), dtype=out_dtype, device=x.device)
    s = torch.empty(scale_shape(gran, R, C), dtype=torch.float32, device=x.device)
    if col_mul is None:
        _check(getattr(lib(), fn)(_ptr(x), dt, R, C, gran, _ptr(q), _ptr(s), _stream(stream)), fn)
    else:
        if col_mul.dtype != torch.float32 or col_mul.numel() != C:
            raise ValueError(f"{fn}: col_mul must be {C} float32 values")
        _check(getattr(lib(), fn)(_ptr(x), dt, R, C, gran, _ptr(col_mul), _ptr(q), _ptr(s), _stream(stream)), fn)
    return q, s


def act_quant_int8(x: torch.Tensor, gran: int = GRAN_ROW, stream=None):
    """-> (int8 codes [R][C], float32 scales in the layout of `gran`)."""
    return _act_quant("act_quant_int8", x, gran, torch.int8, stream)


def act_quant_fp8(x: torch.Tensor, gran: int = GRAN_ROW, stream=None):
    """-> (E4M3 bytes as uint8 [R][C], float32 scales in the layout of `gran`)."""
    return _act_quant("act_quant_fp8", x, gran, torch.uint8, stream)


def act_quant_int8_smooth(x: torch.Tensor, col_mul: torch.Tensor, gran: int = GRAN_ROW, stream=None):
    """INT8 codes and scales of X diag(col_mul) (the SmoothQuant fold: 1/s for
    activations, s for the weights)."""
    return _act_quant("act_quant_int8_smooth", x, gran, torch.int8, stream, col_mul)


def act_quant_fp8_smooth(x: torch.Tensor, col_mul: torch.Tensor, gran: int = GRAN_ROW, stream=None):
    """E4M3 codes and scales of X diag(col_mul)."""
    return _act_quant("act_quant_fp8_smooth", x, gran, torch.uint8, stream, col_mul)


_OUT_DT = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32, torch.int32: I32}


def act_quant_mxfp8(x: torch.Tensor, stream=None):
    """-> (E4M3 bytes as uint8 [R][C], E8M0 scale bytes uint8 [C/32][R rounded
    up to 16], K-block-major)."""
    R, C = x.shape
    dt = _TORCH_DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"act_quant_mxfp8: unsupported dtype {x.dtype}")
    q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    e = torch.empty((C // 32, (R + 15) // 16 * 16), dtype=torch.uint8, device=x.device)
    _check(lib().act_quant_mxfp8(_ptr(x), dt, R, C, _ptr(q), _ptr(e), _stream(stream)), "act_quant_mxfp8")
    return q, e


def gemm_mxfp8(a: torch.Tensor, a_e8m0: torch.Tensor, w: torch.Tensor, w_e8m0: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = (A X_a)(W X_w)^T for MXFP8 operands (act_quant_mxfp8 outputs)."""
    M, K = a.shape
    N, K2 = w.shape
    if K != K2:
        raise ValueError(f"gemm_mxfp8: K mismatch {K} vs {K2}")
    for t, rows in ((a_e8m0, M), (w_e8m0, N)):
        if t.dtype != torch.uint8 or tuple(t.shape) != (K // 32, (rows + 15) // 16 * 16):
            raise ValueError("gemm_mxfp8: scales must be uint8 [K/32][rows rounded up to 16]")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check(lib().gemm_mxfp8(_ptr(a), _ptr(a_e8m0), _ptr(w), _ptr(w_e8m0), M, N, K, _ptr(out), _OUT_DT[out.dtype],
                            _stream(stream)), "gemm_mxfp8")
    return out


def act_quant_mxfp4(x: torch.Tensor, stream=None):
    """-> (packed E2M1 bytes uint8 [R][C/2], element 2i in the low nibble;
    E8M0 scale bytes uint8 [C/32][R rounded up to 16], K-block-major)."""
    R, C = x.shape
    dt = _TORCH_DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"act_quant_mxfp4: unsupported dtype {x.dtype}")
    q = torch.empty((R, C // 2), dtype=torch.uint8, device=x.device)
    e = torch.empty((C // 32, (R + 15) // 16 * 16), dtype=torch.uint8, device=x.device)
    _check(lib().act_quant_mxfp4(_ptr(x), dt, R, C, _ptr(q), _ptr(e), _stream(stream)), "act_quant_mxfp4")
    return q, e


def gemm_mxfp4(a: torch.Tensor, a_e8m0: torch.Tensor, w: torch.Tensor, w_e8m0: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = (A X_a)(W X_w)^T for MXFP4 operands (act_quant_mxfp4 outputs:
    packed [rows][K/2] bytes)."""
    M, KH = a.shape
    N, KH2 = w.shape
    if KH != KH2:
        raise ValueError(f"gemm_mxfp4: K mismatch {2 * KH} vs {2 * KH2}")
    K = 2 * KH
    for t, rows in ((a_e8m0, M), (w_e8m0, N)):
        if t.dtype != torch.uint8 or tuple(t.shape) != (K // 32, (rows + 15) // 16 * 16):
            raise ValueError("gemm_mxfp4: scales must be uint8 [K/32][rows rounded up to 16]")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check(lib().gemm_mxfp4(_ptr(a), _ptr(a_e8m0), _ptr(w), _ptr(w_e8m0), M, N, K, _ptr(out), _OUT_DT[out.dtype],
                            _stream(stream)), "gemm_mxfp4")
    return out


def act_quant_outlier_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().act_quant_outlier_workspace_bytes(rows, cols))


def act_quant_int8_outlier(x: torch.Tensor, tau: float = 6.0, ws: torch.Tensor | None = None, stream=None):
    """The LLM.int8() split of X: its outlier channels (columns whose largest
    magnitude reaches tau) and the per-token INT8 codes of the other columns
    (outlier columns quantize to 0).  -> (q int8 [R][C], scales f32 [R], idx
    int32 [C] of which the first count entries are the outlier columns in
    increasing order, count int32 [1]); idx and count stay on the device."""
    R, C = x.shape
    dt = _TORCH_DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"act_quant_int8_outlier: unsupported dtype {x.dtype}")
    q = torch.empty((R, C), dtype=torch.int8, device=x.device)
    sc = torch.empty((R,), dtype=torch.float32, device=x.device)
    idx = torch.empty((C,), dtype=torch.int32, device=x.device)
    cnt = torch.empty((1,), dtype=torch.int32, device=x.device)
    if ws is None:
        ws = workspace(max(act_quant_outlier_workspace_bytes(R, C), 16), x.device)
    _check(lib().act_quant_int8_outlier(_ptr(x), dt, R, C, float(tau), _ptr(q), _ptr(sc), _ptr(idx), _ptr(cnt),
                                        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "act_quant_int8_outlier")
    return q, sc, idx, cnt


def gemm_w8a8_outlier(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                      w_gran: int, x: torch.Tensor, idx: torch.Tensor, count: torch.Tensor,
                      out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Y = s_a s_w (A W^T) + s_w (X_O W_O^T): the INT8 GEMM of the common
    channels plus the side path over the outlier channels idx[:count] (the
    act_quant_int8_outlier outputs), which multiplies the unquantized
    activations x by the INT8 weight columns, fused into the GEMM."""
    M, K = a.shape
    N, K2 = w.shape
    if K != K2 or tuple(x.shape) != (M, K):
        raise ValueError(f"gemm_w8a8_outlier: shapes a {tuple(a.shape)}, w {tuple(w.shape)}, x {tuple(x.shape)}")
    if a.dtype != torch.int8 or w.dtype != torch.int8:
        raise ValueError("gemm_w8a8_outlier: a and w must be int8 codes")
    if idx.dtype != torch.int32 or count.dtype != torch.int32 or idx.numel() < K:
        raise ValueError("gemm_w8a8_outlier: idx must be int32 with room for K entries, count int32")
    dt = _TORCH_DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"gemm_w8a8_outlier: unsupported dtype {x.dtype}")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check(lib().gemm_w8a8_outlier(_ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), w_gran, _ptr(x), dt, _ptr(idx),
                                   _ptr(count), M, N, K, _ptr(out), _OUT_DT[out.dtype], _stream(stream)),
           "gemm_w8a8_outlier")
    return out


def gemm_w8a8_workspace_bytes(M: int, N: int, K: int, fp8: bool = False, a_gran: int = GRAN_ROW,
                              algo: int = ALGO_AUTO) -> int:
    return int(lib().gemm_w8a8_workspace_bytes(M, N, K, FP8_E4M3 if fp8 else I8, a_gran, algo))


def gemm_w8a8(a: torch.Tensor, a_scales: torch.Tensor | None, a_gran: int, w: torch.Tensor,
              w_scales: torch.Tensor | None, w_gran: int, out_dtype: torch.dtype = torch.bfloat16,
              out: torch.Tensor | None = None, algo: int = ALGO_AUTO, ws: torch.Tensor | None | bool = None,
              stream=None) -> torch.Tensor:
    """Y = A W^T on the INT8 / FP8 matrix cores.  ws: a workspace tensor, None
    to use the cached per-device workspace (enables split-K of the large-M
    kernel), or False for none."""
    M, K = a.shape
    N, K2 = w.shape
    if K != K2:
        raise ValueError(f"gemm_w8a8: K mismatch {K} vs {K2}")
    if a.dtype == torch.int8 and w.dtype == torch.int8:
        in_dt = I8
    elif a.dtype == torch.uint8 and w.dtype == torch.uint8:
        in_dt = FP8_E4M3
    else:
        raise ValueError("gemm_w8a8: operands must both be int8 or both E4M3 bytes (uint8)")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    L = lib()
    if ws is False:
        _check(L.gemm_w8a8_ex(_ptr(a), _ptr(a_scales), a_gran, _ptr(w), _ptr(w_scales), w_gran, in_dt, M, N, K,
                              _ptr(out), _OUT_DT[out.dtype], algo, _stream(stream)), "gemm_w8a8")
        return out
    if ws is None:
        need = int(L.gemm_w8a8_workspace_bytes(M, N, K, in_dt, a_gran, algo))
        ws = workspace(need, a.device) if need > 0 else None
    _check(L.gemm_w8a8_ws(_ptr(a), _ptr(a_scales), a_gran, _ptr(w), _ptr(w_scales), w_gran, in_dt, M, N, K,
                          _ptr(out), _OUT_DT[out.dtype], _ptr(ws), 0 if ws is None else ws.numel(), algo,
                          _stream(stream)), "gemm_w8a8")
    return out


def gemm_w4a8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().gemm_w4a8_workspace_bytes(M, N, K))


def gemm_w4a8(a: torch.Tensor, a_scales: torch.Tensor, a_gran: int, packed: PackedW4,
              out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
              ws: torch.Tensor | None | bool = None, stream=None) -> torch.Tensor:
    """Y = (A s_a) W^T: INT8 activation codes (act_quant_int8 with GRAN_ROW or
    GRAN_TENSOR) times packed INT4 weights, on the INT8 matrix cores.  ws: a
    workspace tensor, None to use the cached per-device workspace (enables the
    K split when the output tiles do not fill the device), or False for none."""
    M, K = a.shape
    if a.dtype != torch.int8:
        raise ValueError(f"gemm_w4a8: activations must be int8 codes, got {a.dtype}")
    if K != packed.K:
        raise ValueError(f"gemm_w4a8: a has K={K}, weights K={packed.K}")
    if out is None:
        out = torch.empty((M, packed.N), dtype=out_dtype, device=a.device)
    if out.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise ValueError(f"gemm_w4a8: output must be bfloat16/float16/float32, got {out.dtype}")
    L = lib()
    if ws is False:
        _check(L.gemm_w4a8(_ptr(a), _ptr(a_scales), a_gran, M, K, _ptr(packed.qweight), _ptr(packed.scales),
                           _ptr(packed.zeros), packed.N, packed.group, _ptr(out), _OUT_DT[out.dtype],
                           _stream(stream)), "gemm_w4a8")
        return out
    if ws is None:
        need = gemm_w4a8_workspace_bytes(M, packed.N, K)
        ws = workspace(need, a.device) if need > 0 else None
    _check(L.gemm_w4a8_ws(_ptr(a), _ptr(a_scales), a_gran, M, K, _ptr(packed.qweight), _ptr(packed.scales),
                          _ptr(packed.zeros), packed.N, packed.group, _ptr(out), _OUT_DT[out.dtype], _ptr(ws),
                          0 if ws is None else ws.numel(), _stream(stream)), "gemm_w4a8")
    return out


def gemm_w8a8_algo(M: int, N: int, K: int, fp8: bool = False) -> int:
    return lib().gemm_w8a8_algo(M, N, K, FP8_E4M3 if fp8 else I8)


# ----------------------------------------------------------- KV cache --------

_KV_CACHE = struct.Struct("@PPPPqiiii")               # bg_kv_cache
_KV_ATTN = struct.Struct("@PPqqPqPPPPPqqqqqqiiif")    # bg_kv_attn
_KV_DIMS = (64, 128, 256)


@dataclass(frozen=True)
class KVCache:
    """A paged key/value cache in 8 or 4 bits: codes [pages][kv_heads][page_size][D]
    (int8 for I8, E4M3 bytes as uint8 for FP8_E4M3) or [...][D / 2] uint8 (U4,
    element 2i in the low nibble), and one record per token and head
    [pages][kv_heads][page_size]: a float32 scale, or for U4 a float16 pair
    (scale, zero-point) in a last axis of 2.  Slot n is token n % page_size of
    page n // page_size."""
    k: torch.Tensor
    v: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor
    format: int

    def __post_init__(self):
        if self.format not in (I8, FP8_E4M3, U4):
            raise ValueError(f"KVCache: format must be I8, FP8_E4M3 or U4, got {self.format}")
        code, tail = (torch.int8 if self.format == I8 else torch.uint8), ((2,) if self.format == U4 else ())
        record = torch.float16 if self.format == U4 else torch.float32
        if self.k.dim() != 4 or self.k.dtype != code or self.v.dtype != code or self.v.shape != self.k.shape:
            raise ValueError(f"KVCache: k and v must be {code} [pages][kv_heads][page_size][bytes of a row]")
        for t in (self.k_scales, self.v_scales):
            if t.dtype != record or tuple(t.shape) != (*self.k.shape[:3], *tail):
                raise ValueError(f"KVCache: scales must be {record} {(*self.k.shape[:3], *tail)}")
        pages, heads, page, width = self.k.shape
        dim = 2 * width if self.format == U4 else width
        if dim not in _KV_DIMS or pages < 1 or heads < 1 or page < 16 or page > 1024 or page & (page - 1):
            raise ValueError(f"KVCache: head size {dim} must be one of {_KV_DIMS}, page_size {page} a power of two in 16..1024")
        tensors = (self.k, self.v, self.k_scales, self.v_scales)
        if any(t.device != self.k.device for t in tensors):
            raise ValueError("KVCache: the tensors must be on one device")
        ptrs = [_ptr(t).value for t in tensors]
        desc = ctypes.create_string_buffer(_KV_CACHE.pack(*ptrs, pages, page, heads, dim, self.format), _KV_CACHE.size)
        for name, value in (("_desc", desc), ("address", ctypes.addressof(desc)), ("device", self.k.device),
                            ("pages", pages), ("page_size", page), ("kv_heads", heads), ("head_dim", dim)):
            object.__setattr__(self, name, value)

    # Copies and pickles carry the fields alone: the descriptor of the new tensors is their own.
    def __getstate__(self):
        return self.k, self.v, self.k_scales, self.v_scales, self.format

    def __setstate__(self, state):
        for name, value in zip(("k", "v", "k_scales", "v_scales", "format"), state):
            object.__setattr__(self, name, value)
        self.__post_init__()

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scales, self.v_scales))


def kv_cache(pages: int, page_size: int, kv_heads: int, head_dim: int, format: int, device="cuda") -> KVCache:
    """A cache of `pages` pages whose slots hold zeros."""
    if format not in (I8, FP8_E4M3, U4):
        raise ValueError(f"kv_cache: format must be I8, FP8_E4M3 or U4, got {format}")
    shape, u4 = (pages, kv_heads, page_size), format == U4
    codes = [torch.zeros((*shape, head_dim // 2 if u4 else head_dim), dtype=torch.int8 if format == I8 else torch.uint8,
                         device=device) for _ in range(2)]
    scales = [torch.zeros((*shape, 2), dtype=torch.float16, device=device) if u4
              else torch.zeros(shape, dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(*codes, *scales, format)


def _on_device(fn: str, cache: KVCache, *tensors):
    for t in tensors:
        if t is not None and t.device != cache.device:
            raise ValueError(f"{fn}: operands must be on the cache's device {cache.device}, got {t.device}")
    if cache.device.index != torch.cuda.current_device():
        raise ValueError(f"{fn}: the cache is on {cache.device}, the current device is {torch.cuda.current_device()}")


def _raw_stream(device: int) -> int:
    """The handle of the device's current stream (without the Stream object of
    torch.cuda.current_stream(), which costs a call of a few microseconds more)."""
    return torch._C._cuda_getCurrentRawStream(device)


def _on_stream(stream, tensors, call):
    """call() with `stream` current, so what it allocates belongs to that stream;
    the operands' memory is kept from reuse until the stream has passed."""
    with torch.cuda.stream(stream):
        r = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return r


def _kv_slots(fn: str, slots: torch.Tensor) -> int:
    if slots.dtype != torch.int64 or slots.dim() != 1 or not slots.is_contiguous():
        raise ValueError(f"{fn}: slots must be a contiguous int64 vector")
    return slots.shape[0]


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, slots: torch.Tensor, stream=None) -> None:
    """Quantize the keys and values of T new tokens ([T][kv_heads][D], the last
    axis contiguous, the others of any stride that is a multiple of 16 bytes:
    slices of a fused projection's rows need no copy) into cache slots int64 [T].
    A slot outside the cache (-1) skips its token."""
    fn = "kv_cache_write"
    if stream is not None:
        return _on_stream(stream, (k, v, slots, cache.k, cache.v, cache.k_scales, cache.v_scales),
                          lambda: kv_cache_write(k, v, cache, slots))
    T = _kv_slots(fn, slots)
    shape = (T, cache.kv_heads, cache.head_dim)
    if tuple(k.shape) != shape or tuple(v.shape) != shape:
        raise ValueError(f"{fn}: k {tuple(k.shape)} and v {tuple(v.shape)} must be {shape}")
    dt = _TORCH_DT.get(k.dtype)
    if dt is None or v.dtype != k.dtype:
        raise ValueError(f"{fn}: k and v must be of one type, float32, float16 or bfloat16 (got {k.dtype}, {v.dtype})")
    if T == 0:
        return
    ks, vs = k.stride(), v.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError(f"{fn}: the last axis of k and v must be contiguous")
    _on_device(fn, cache, k, v, slots)
    if T == 1 or cache.kv_heads == 1:        # an axis of one element may have any stride
        ks, vs = ((0 if T == 1 else s[0], 0 if cache.kv_heads == 1 else s[1]) for s in (ks, vs))
    _check(lib().kv_cache_write(cache.address, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], dt,
                                slots.data_ptr(), T, _raw_stream(cache.device.index)), fn)


def kv_cache_read(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, stream=None):
    """-> (k, v) of `dtype` [T][kv_heads][D]: the values of slots int64 [T].  A
    slot outside the cache reads as zeros."""
    fn = "kv_cache_read"
    if stream is not None:
        return _on_stream(stream, (slots, cache.k, cache.v, cache.k_scales, cache.v_scales),
                          lambda: kv_cache_read(cache, slots, dtype))
    T = _kv_slots(fn, slots)
    dt = _TORCH_DT.get(dtype)
    if dt is None:
        raise ValueError(f"{fn}: unsupported dtype {dtype}")
    _on_device(fn, cache, slots)
    k, v = (torch.empty((T, cache.kv_heads, cache.head_dim), dtype=dtype, device=cache.device) for _ in range(2))
    if T:
        _check(lib().kv_cache_read(cache.address, slots.data_ptr(), T, k.data_ptr(), v.data_ptr(), dt,
                                   _raw_stream(cache.device.index)), fn)
    return k, v


_kv_workspaces: dict = {}


def _kv_workspace(nbytes: int, device, stream: int) -> torch.Tensor:
    """A workspace of at least nbytes, cached per device and stream.  In a graph's
    capture it is the graph's own, from its memory pool: graphs captured on one
    stream may be replayed on several, beside eager work."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, stream)
    ws = _kv_workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        if ws is not None:
            _retired.append(ws)       # HIP graphs captured earlier may still use it
        ws = torch.empty(1 << (nbytes - 1).bit_length(), dtype=torch.uint8, device=device)
        _kv_workspaces[key] = ws
    return ws


def _kv_attn(fn, q, cache, block_table, kv_lens, cu_q, tree, max_q_len, max_kv_len, window, sinks, scale, out, lse, ws):
    if q.dim() != 3 or q.stride(2) != 1 or q.shape[2] != cache.head_dim:
        raise ValueError(f"{fn}: q must be [T][q_heads][{cache.head_dim}] with a contiguous last axis, got {tuple(q.shape)}")
    T, heads, dim = q.shape
    dt = _TORCH_DT.get(q.dtype)
    if dt not in (F16, BF16):
        raise ValueError(f"{fn}: q must be float16/bfloat16, got {q.dtype}")
    if max_q_len is None:
        max_q_len = 1 if cu_q is None else max(T, 1)
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError(f"{fn}: block_table must be a contiguous int32 matrix [batch][pages of a sequence]")
    B, max_pages = block_table.shape
    if kv_lens.dtype != torch.int32 or kv_lens.shape != (B,) or not kv_lens.is_contiguous():
        raise ValueError(f"{fn}: kv_lens must be a contiguous int32 vector of {B}")
    if cu_q is not None and (cu_q.dtype != torch.int32 or cu_q.shape != (B + 1,) or not cu_q.is_contiguous()):
        raise ValueError(f"{fn}: cu_q must be a contiguous int32 vector of {B + 1}")
    words = 0
    if tree is not None:
        if tree.dtype != torch.int64 or tree.dim() != 2 or tree.shape[0] != T or not tree.is_contiguous():
            raise ValueError(f"{fn}: tree must be a contiguous int64 matrix [{T}][words]")
        words = tree.shape[1]
    if out is None:
        new = torch.empty if T <= B * max_q_len else torch.zeros       # more rows than the call can write
        out = new((T, heads, dim), dtype=q.dtype, device=q.device)
    elif out.shape != (T, heads, dim) or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError(f"{fn}: out must be a contiguous {(T, heads, dim)} of {q.dtype}")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, heads) or not lse.is_contiguous()):
        raise ValueError(f"{fn}: lse must be a contiguous float32 {(T, heads)}")
    if T == 0 or B == 0:
        return out
    _on_device(fn, cache, q, block_table, kv_lens, cu_q, tree, out, lse, ws)
    L = lib()
    s = _raw_stream(cache.device.index)
    args = _KV_ATTN.pack(
        cache.address, q.data_ptr(), 0 if T == 1 else q.stride(0), 0 if heads == 1 else q.stride(1),
        block_table.data_ptr(), max_pages, kv_lens.data_ptr(), 0 if cu_q is None else cu_q.data_ptr(),
        0 if tree is None else tree.data_ptr(), out.data_ptr(),
        0 if lse is None else lse.data_ptr(), T, B, max_q_len, max_kv_len, window, sinks, heads, dt, words,
        dim ** -0.5 if scale is None else scale)
    if ws is None:
        need = L.kv_attn_workspace_bytes(args)
        ws = _kv_workspace(need, q.device, s) if need > 0 else None
    elif not ws.is_contiguous():
        raise ValueError(f"{fn}: the workspace must be contiguous")
    _check(getattr(L, fn)(args, None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size(), s), fn)
    return out


def kv_attn(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
            cu_q: torch.Tensor | None = None, max_q_len: int | None = None, *, max_kv_len: int = 0, window: int = 0, sinks: int = 0,
            scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
            ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of ragged queries [T][q_heads][D] over the cache -> [T][q_heads][D].

    Sequence b owns the queries cu_q[b] .. cu_q[b + 1] - 1 (cu_q None: one query
    per sequence), which are the last of its kv_lens[b] positions; position j
    lies in page block_table[b][j // page_size] (a page outside the cache, such
    as -1, holds nothing).  A query sees the positions up to its own; with a
    window only the last `window` of them and the first `sinks`.  A query that
    sees nothing gives zeros.  max_q_len and max_kv_len (0: the table's width)
    are host-side bounds of the lengths: a sequence's queries past max_q_len are
    left alone, and without it (None) every sequence may own all T, which with
    cu_q costs some speed.  scale None: D ** -0.5.  lse: float32
    [T][q_heads] that receives the log-sum-exp of the scaled scores.  ws: a
    workspace tensor (kv_attn_workspace_bytes), None for the one cached per stream
    (a captured graph: its own)."""
    if stream is not None:
        return _on_stream(stream, (q, cache.k, cache.v, cache.k_scales, cache.v_scales, block_table, kv_lens, cu_q, out, lse, ws),
                          lambda: kv_attn(q, cache, block_table, kv_lens, cu_q, max_q_len, max_kv_len=max_kv_len, window=window,
                                          sinks=sinks, scale=scale, out=out, lse=lse, ws=ws))
    return _kv_attn("kv_attn", q, cache, block_table, kv_lens, cu_q, None, max_q_len, max_kv_len, window, sinks, scale, out,
                    lse, ws)


def kv_attn_tree(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor, cu_q: torch.Tensor,
                 tree: torch.Tensor, max_q_len: int, *, max_kv_len: int = 0, scale: float | None = None,
                 out: torch.Tensor | None = None, lse: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """kv_attn for a tree of drafted tokens: a sequence's queries are its last
    positions (already written), each sees every position before them, and of
    the drafted ones exactly its bits of tree int64 [T][words] (bit e % 64 of word
    e // 64: drafted token e; a token's own bit among them)."""
    if stream is not None:
        return _on_stream(stream, (q, cache.k, cache.v, cache.k_scales, cache.v_scales, block_table, kv_lens, cu_q, tree, out,
                                   lse, ws),
                          lambda: kv_attn_tree(q, cache, block_table, kv_lens, cu_q, tree, max_q_len, max_kv_len=max_kv_len,
                                               scale=scale, out=out, lse=lse, ws=ws))
    return _kv_attn("kv_attn_tree", q, cache, block_table, kv_lens, cu_q, tree, max_q_len, max_kv_len, 0, 0, scale, out, lse, ws)


def kv_attn_workspace_bytes(q_shape, cache: KVCache, batch: int, max_pages: int, max_q_len: int | None = None, max_kv_len: int = 0,
                            window: int = 0, sinks: int = 0, tree_words: int = 0) -> int:
    """Bytes of the workspace that kv_attn (kv_attn_tree with tree_words > 0) needs for queries of q_shape;
    max_q_len None: with or without cu_q."""
    if max_q_len is None:
        bounds = {max(q_shape[0], 1)} | ({1} if q_shape[0] == batch else set())
        return max(kv_attn_workspace_bytes(q_shape, cache, batch, max_pages, n, max_kv_len, window, sinks, tree_words) for n in bounds)
    return int(lib().kv_attn_workspace_bytes(_KV_ATTN.pack(
        cache.address, 0, 0, 0, 0, max_pages, 0, 256, 0, 0, 0, q_shape[0], batch, max_q_len, max_kv_len, window, sinks,
        q_shape[1], BF16, tree_words, 1.0)))
