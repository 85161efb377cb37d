"""Binding of the single-token entry points (C ABI in ``include/qv_decode.h``): few-row linears with
4-bit weights, the append of keys and values to a paged cache, and the attention of one new token over
it.  As in the package's other entry points, every operand's shape, type and layout is checked before
the library is called (ValueError), a non-OK status raises QVError, and there is no fallback.

These calls take microseconds, so the checks are written out flat and work on plain Python values.
"""
from __future__ import annotations

import ctypes

import torch

from . import QV_EPI_NONE, QVError, lib

__all__ = [
    "qv_w4a16_gemv", "qv_w4a16_linear", "qv_w4a16_linear_workspace_size", "QVKVCache", "qv_kv_append",
    "qv_paged_attention", "qv_paged_attention_workspace_size", "QV_KV_BF16", "QV_KV_INT8",
]

QV_KV_BF16, QV_KV_INT8 = 0, 1

_F32, _BF16, _U8, _I8, _I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int8, torch.int32
_CODE = {_F32: 0, _BF16: 1}  # qv_dtype


class _Cache(ctypes.Structure):  # qv_kv_cache
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class _Heads(ctypes.Structure):  # qv_heads
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def bind(L):
    """Declare the C signatures of these entry points on a loaded library handle and return it."""
    P, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    L.qv_w4a16_gemv.argtypes = [P, i32, i64, i64, i64, P, P, i64, P, i64, i32, P, i32, i64, P]
    L.qv_w4a16_linear_workspace_size.argtypes = [i64, i64]
    L.qv_w4a16_linear_workspace_size.restype = sz
    L.qv_w4a16_linear.argtypes = [P, i32, i64, i64, i64, P, P, P, i64, P, i64, i32, P, i32, i64, P, sz, P]
    L.qv_kv_append.argtypes = [P, P, i64, i64, i64, P, P, i64, P, P, i32, P, P, i64, i64, P, P, P, i64, P]
    L.qv_paged_attention_workspace_size.argtypes = [i64, i64, i64, i64, i64]
    L.qv_paged_attention_workspace_size.restype = sz
    L.qv_paged_attention.argtypes = [P, i32, i64, i64, P, P, i64, i64, P, f32, i64, P, P, sz, P]
    for name in ("qv_w4a16_gemv", "qv_w4a16_linear", "qv_kv_append", "qv_paged_attention"):
        getattr(L, name).restype = i32
    return L


_bound = None


def _lib():
    global _bound
    if _bound is None:
        _bound = bind(lib())
    return _bound


def _stream(stream) -> int:
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _bad(what: str, name: str, t, wanted: str):
    if t is None:
        raise ValueError(f"{what}: {name} is required")
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: {name} must be a torch tensor")
    raise ValueError(f"{what}: {name} is {str(t.dtype).replace('torch.', '')} {tuple(t.shape)} with strides "
                     f"{tuple(t.stride())}, expected {wanted}")


def _dense(what: str, name: str, t, dtype, shape) -> int:
    """Address of a contiguous operand of this type and shape."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _bad(what, name, t, f"dense {str(dtype).replace('torch.', '')} {tuple(shape)}")
    return t.data_ptr()


def _rows(what: str, name: str, t, M: int, N: int) -> int:
    """Row stride of a float operand [M, N] with unit column stride."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _CODE or t.shape != (M, N):
        _bad(what, name, t, f"float32 or bfloat16 {(M, N)}")
    ld, unit = t.stride()
    if (unit != 1 and N > 1) or (ld < N and M > 1):
        _bad(what, name, t, f"unit column stride and a row stride of at least {N}")
    return ld if ld >= N else N


def _one_gpu(what: str, *tensors) -> None:
    on = -2
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != on:
                if d < 0:
                    raise ValueError(f"{what}: every operand must be a GPU tensor (got one on {t.device})")
                if on >= 0:
                    raise ValueError(f"{what}: operands are on different devices")
                on = d


def _done(status: int, what: str) -> None:
    if status != 0:
        raise QVError(status, what)


# ------------------------------------------------------------------------------------- few-row linears

def _w4a16_sizes(what, X, Wq, w_scale, group, bias):
    if not isinstance(X, torch.Tensor) or X.dim() != 2 or not isinstance(Wq, torch.Tensor) or Wq.dim() != 2:
        raise ValueError(f"{what}: X and Wq must be 2-D tensors")
    M, K = X.shape
    N = Wq.shape[0]
    _dense(what, "Wq", Wq, _U8, (N, K // 2))
    if group <= 0 or K % group:
        raise ValueError(f"{what}: group {group} must be positive and divide K = {K}")
    G = K // group
    if w_scale is None or w_scale.dim() != 1 or G != 1:
        _dense(what, "w_scale", w_scale, _F32, (N, G))
    else:
        _dense(what, "w_scale", w_scale, _F32, (N,))
    if bias is not None:
        _dense(what, "bias", bias, _F32, (N,))
    return M, K, N


def qv_w4a16_gemv(X, Wq, w_scale, group: int, bias, Y, epi: int = QV_EPI_NONE, stream=None) -> None:
    """Y [M, N] = X [M, K] . dequant(Wq)^T (+ bias) (+ GELU) for few rows of fp32/bf16 activations, taken as
    they are.  Wq [N, K/2] uint8 packed int4, w_scale [N, K/group] fp32 (or [N] where group == K)."""
    what = "qv_w4a16_gemv"
    M, K, N = _w4a16_sizes(what, X, Wq, w_scale, group, bias)
    ldx, ldy = _rows(what, "X", X, M, K), _rows(what, "Y", Y, M, N)
    _one_gpu(what, X, Wq, w_scale, bias, Y)
    _done(_lib().qv_w4a16_gemv(X.data_ptr(), _CODE[X.dtype], M, K, ldx, Wq.data_ptr(), w_scale.data_ptr(), group,
                               None if bias is None else bias.data_ptr(), N, epi, Y.data_ptr(), _CODE[Y.dtype], ldy,
                               _stream(stream)), what)


def qv_w4a16_linear_workspace_size(M: int, K: int) -> int:
    return int(_lib().qv_w4a16_linear_workspace_size(int(M), int(K)))


def qv_w4a16_linear(X, inv_smooth, Wq, w_scale, group: int, bias, Y, workspace, epi: int = QV_EPI_NONE,
                    stream=None) -> None:
    """The online layer for few rows: X rotated (K = 1024 or 4096), smoothed by inv_smooth [K] (or None) and
    multiplied as in ``qv_w4a16_gemv`` without being quantized.  ``workspace`` is a uint8 device tensor of at
    least ``qv_w4a16_linear_workspace_size(M, K)`` bytes."""
    what = "qv_w4a16_linear"
    M, K, N = _w4a16_sizes(what, X, Wq, w_scale, group, bias)
    ldx, ldy = _rows(what, "X", X, M, K), _rows(what, "Y", Y, M, N)
    if inv_smooth is not None:
        _dense(what, "inv_smooth", inv_smooth, _F32, (K,))
    L = _lib()
    size = _workspace(what, workspace, L.qv_w4a16_linear_workspace_size(M, K))
    _one_gpu(what, X, inv_smooth, Wq, w_scale, bias, Y, workspace)
    _done(L.qv_w4a16_linear(X.data_ptr(), _CODE[X.dtype], M, K, ldx,
                            None if inv_smooth is None else inv_smooth.data_ptr(), Wq.data_ptr(), w_scale.data_ptr(),
                            group, None if bias is None else bias.data_ptr(), N, epi, Y.data_ptr(), _CODE[Y.dtype],
                            ldy, workspace.data_ptr(), size, _stream(stream)), what)


def _workspace(what: str, workspace, need: int) -> int:
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != _U8 or not workspace.is_contiguous():
        _bad(what, "workspace", workspace, f"dense uint8 of at least {need} bytes")
    size = workspace.numel()
    if size < need:
        raise ValueError(f"{what}: workspace holds {size} bytes, needs {need}")
    return size


# ---------------------------------------------------------------------------------------- paged cache

class QVKVCache:
    """A paged cache of keys and values over the caller's tensors: k_pages, v_pages [pages, heads, page_size, D]
    (bf16, or int8 with k_scale, v_scale [pages, heads, page_size] fp32), D 64 or 128, unit channel stride,
    the same strides in both; a permuted [pages, page_size, heads, D] tensor fits.  Holds the tensors, checks
    them once and allocates nothing."""

    def __init__(self, k_pages, v_pages, k_scale=None, v_scale=None):
        what = "QVKVCache"
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not isinstance(t, torch.Tensor) or t.dtype not in (_BF16, _I8) or t.dim() != 4:
                _bad(what, name, t, "bfloat16 or int8 [pages, heads, page_size, D]")
        if v_pages.dtype != k_pages.dtype or v_pages.shape != k_pages.shape or v_pages.stride() != k_pages.stride():
            _bad(what, "v_pages", v_pages, "type, shape and strides of k_pages")
        if k_pages.stride(3) != 1:
            _bad(what, "k_pages", k_pages, "unit channel stride")
        pages, heads, size, dim = k_pages.shape
        # an extent of one has no stride of its own
        sp, sh, st = (max(s, dim) if n <= 1 else s for s, n in zip(k_pages.stride()[:3], k_pages.shape[:3]))
        if min(sp, sh, st) < dim:
            _bad(what, "k_pages", k_pages, "tokens that do not overlap")
        quantized = k_pages.dtype == _I8
        if quantized:
            _dense(what, "k_scale", k_scale, _F32, (pages, heads, size))
            _dense(what, "v_scale", v_scale, _F32, (pages, heads, size))
        elif k_scale is not None or v_scale is not None:
            raise ValueError(f"{what}: a bfloat16 cache has no scales")
        _one_gpu(what, k_pages, v_pages, k_scale, v_scale)
        unit = 16 if quantized else 8
        sp, sh, st = (-(-s // unit) * unit if n <= 1 else s for s, n in zip((sp, sh, st), k_pages.shape[:3]))
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.head_dim = pages, heads, size, dim
        self.device = k_pages.get_device()
        self.c = _Cache(k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr() if quantized else None,
                        v_scale.data_ptr() if quantized else None, pages, heads, size, dim, sp, sh, st,
                        QV_KV_INT8 if quantized else QV_KV_BF16)
        self.ref = ctypes.byref(self.c)


def _heads(what: str, name: str, t, shape, dtype=None):
    """A qv_heads of [T, heads, D] rows with unit channel stride."""
    if (not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype not in _CODE
            or (dtype is not None and t.dtype != dtype)):
        _bad(what, name, t, f"{'float32 or bfloat16' if dtype is None else str(dtype).replace('torch.', '')} {shape}")
    ts, hs, unit = t.stride()
    if unit != 1 or (hs < shape[2] and shape[1] > 1):
        _bad(what, name, t, "unit channel stride and heads that do not overlap")
    if shape[1] <= 1:
        hs = shape[2]
    return _Heads(t.data_ptr(), ts if shape[0] > 1 else 0, hs)


def _page_table(what: str, t, rows=None):
    if (not isinstance(t, torch.Tensor) or t.dtype != _I32 or t.dim() != 2 or (rows is not None and t.shape[0] != rows)
            or (t.stride(1) != 1 and t.shape[1] > 1) or (t.stride(0) < t.shape[1] and t.shape[0] > 1)):
        _bad(what, "page_table", t, f"int32 [{'sequences' if rows is None else rows}, pages] with unit column stride")
    return t.shape[0], t.shape[1], max(t.stride(0), t.shape[1])


def qv_kv_append(cache, page_table, token_seq, token_index, K, V, cos=None, sin=None, position=None, Q=None,
                 Q_out=None, stream=None) -> None:
    """Store the keys K and values V [T, heads, D] (fp32/bf16) of T new tokens in ``cache``, K turned by position.

    page_table [sequences, pages] int32; token_seq [T] int32 sequence of each token (None: token t is sequence t);
    token_index [T] int32 place of each token in its sequence; cos, sin [places, D / (2 axes)] fp32 (None: no
    rotation); position [T, axes] int32 with 1 or 2 axes (None: token_index).  Q [T, q_heads, D] is turned into
    Q_out (which may be Q)."""
    what = "qv_kv_append"
    if not isinstance(cache, QVKVCache):
        raise ValueError(f"{what}: cache must be a QVKVCache")
    seqs, pages, ld = _page_table(what, page_table)
    if not isinstance(K, torch.Tensor) or K.dim() != 3:
        _bad(what, "K", K, "[T, heads, D]")
    T, H, D = K.shape[0], cache.heads, cache.head_dim
    dt = K.dtype
    k, v = _heads(what, "K", K, (T, H, D)), _heads(what, "V", V, (T, H, D), dt)
    index = _dense(what, "token_index", token_index, _I32, (T,))
    seq = None
    if token_seq is not None:
        seq = _dense(what, "token_seq", token_seq, _I32, (T,))
    elif T > seqs:
        raise ValueError(f"{what}: {T} tokens of {seqs} sequences need token_seq")
    axes = places = 0
    c = s = p = q = qo = None
    q_heads = 0
    if (cos is None) != (sin is None):
        raise ValueError(f"{what}: cos and sin come together")
    if position is not None:
        if not isinstance(position, torch.Tensor) or position.dim() != 2 or position.shape[1] not in (1, 2):
            _bad(what, "position", position, f"int32 {(T, 1)} or {(T, 2)}")
        axes = position.shape[1]
        p = _dense(what, "position", position, _I32, (T, axes))
    axes = axes or 1
    if cos is not None:
        places = cos.shape[0] if isinstance(cos, torch.Tensor) and cos.dim() == 2 else 0
        c = _dense(what, "cos", cos, _F32, (places, D // 2 // axes))
        s = _dense(what, "sin", sin, _F32, (places, D // 2 // axes))
    if (Q is None) != (Q_out is None):
        raise ValueError(f"{what}: Q and Q_out come together")
    if Q is not None:
        if not isinstance(Q, torch.Tensor) or Q.dim() != 3 or Q.shape[1] == 0:
            _bad(what, "Q", Q, "[T, q_heads, D]")
        q_heads = Q.shape[1]
        q = _heads(what, "Q", Q, (T, q_heads, D), dt)
        qo = _heads(what, "Q_out", Q_out, (T, q_heads, D), dt)
    _one_gpu(what, cache.k_pages, page_table, token_seq, token_index, K, V, cos, sin, position, Q, Q_out)
    ref = ctypes.byref
    _done(_lib().qv_kv_append(cache.ref, page_table.data_ptr(), seqs, pages, ld, seq, index, T, ref(k), ref(v),
                              _CODE[dt], c, s, places, axes, p, None if q is None else ref(q),
                              None if qo is None else ref(qo), q_heads, _stream(stream)), what)


def qv_paged_attention_workspace_size(B: int, q_heads: int, heads: int, head_dim: int, capacity: int) -> int:
    return int(_lib().qv_paged_attention_workspace_size(int(B), int(q_heads), int(heads), int(head_dim), int(capacity)))


def qv_paged_attention(Q, cache, page_table, lens, O, workspace, scale=None, window: int = 0, stream=None) -> None:
    """O [B, q_heads, D]: attention of one new token Q [B, q_heads, D] (fp32/bf16) of each sequence over the last
    ``window`` (0: all) of its lens[b] tokens in ``cache``; scale defaults to D ** -0.5.  ``workspace`` holds at
    least ``qv_paged_attention_workspace_size(B, q_heads, heads, D, page_table.shape[1] * page_size)`` bytes."""
    what = "qv_paged_attention"
    if not isinstance(cache, QVKVCache):
        raise ValueError(f"{what}: cache must be a QVKVCache")
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3 or Q.shape[1] == 0 or Q.shape[1] % cache.heads:
        _bad(what, "Q", Q, f"[B, a multiple of {cache.heads} heads, {cache.head_dim}]")
    B, Hq, D = Q.shape[0], Q.shape[1], cache.head_dim
    q = _heads(what, "Q", Q, (B, Hq, D))
    o = _heads(what, "O", O, (B, Hq, D), Q.dtype)
    _, pages, ld = _page_table(what, page_table, B)
    _dense(what, "lens", lens, _I32, (B,))
    if window < 0:
        raise ValueError(f"{what}: window {window} must not be negative")
    L = _lib()
    size = _workspace(what, workspace,
                      L.qv_paged_attention_workspace_size(B, Hq, cache.heads, D, pages * cache.page_size))
    _one_gpu(what, cache.k_pages, Q, page_table, lens, O, workspace)
    _done(L.qv_paged_attention(ctypes.byref(q), _CODE[Q.dtype], B, Hq, cache.ref, page_table.data_ptr(), pages, ld,
                               lens.data_ptr(), D ** -0.5 if scale is None else scale, window, ctypes.byref(o),
                               workspace.data_ptr(), size, _stream(stream)), what)
