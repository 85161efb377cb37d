"""Single-token entry points (C ABI in ``include/qv_decode.h``): few-row linears with 4-bit weights, the
append of keys and values to a paged cache, and the attention of one new token over it.

As in the package's other entry points, every operand's shape, type, layout and device is checked before
the library is called (ValueError), a non-OK status raises QVError, and there is no fallback.  The
checks live in the extension module ``_decode`` (``csrc/decode_binding.cpp``): these calls take a few
microseconds on the device, and checks written in Python would take longer.
"""
from __future__ import annotations

import ctypes

from . import QV_EPI_NONE, lib

__all__ = [
    "qv_w4a16_gemv", "qv_w4a16_linear", "qv_w4a16_linear_workspace_size", "QVKVCache", "qv_kv_append",
    "qv_paged_attention", "qv_paged_attention_workspace_size", "QV_KV_BF16", "QV_KV_INT8", "QV_KV_FP8",
]

QV_KV_BF16, QV_KV_INT8, QV_KV_FP8 = 0, 1, 2


class QVKVCacheStruct(ctypes.Structure):
    """qv_kv_cache of the C ABI."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class QVBlockCacheStruct(ctypes.Structure):
    """qv_kv_cache with its last field, the tokens of a scale, which only FP8 caches have."""
    _fields_ = QVKVCacheStruct._fields_ + [("scale_tokens", ctypes.c_int32)]


class QVHeadsStruct(ctypes.Structure):
    """qv_heads of the C ABI."""
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


class _Unloaded:
    """Stands for the extension module until the first call, and fails loudly if it is not built."""

    def __getattr__(self, name):
        global _native
        lib()  # libqv.so, or its ImportError
        try:
            import torch  # noqa: F401  (the extension module links against it)

            from . import _decode
        except ImportError as e:
            raise ImportError(f"{e}; the extension module _decode.so is built by __graft_entry__.build()") from e
        _native = _decode
        return getattr(_decode, name)


_native = _Unloaded()


# ------------------------------------------------------------------------------------- few-row linears

def qv_w4a16_gemv(X, Wq, w_scale, group: int, bias, Y, epi: int = QV_EPI_NONE, stream=None) -> None:
    """Y [M, N] = X [M, K] . dequant(Wq)^T (+ bias) (+ GELU) for few rows of fp32/bf16 activations, taken as
    they are.  Wq [N, K/2] uint8 packed int4, w_scale [N, K/group] fp32 (or [N] where group == K)."""
    _native.w4a16_gemv(X, Wq, w_scale, group, bias, Y, epi, stream)


def qv_w4a16_linear_workspace_size(M: int, K: int) -> int:
    return int(_lib().qv_w4a16_linear_workspace_size(int(M), int(K)))


def qv_w4a16_linear(X, inv_smooth, Wq, w_scale, group: int, bias, Y, workspace, epi: int = QV_EPI_NONE,
                    stream=None) -> None:
    """The online layer for few rows: X rotated (K = 1024 or 4096), smoothed by inv_smooth [K] (or None) and
    multiplied as in ``qv_w4a16_gemv`` without being quantized.  ``workspace`` is a uint8 device tensor of at
    least ``qv_w4a16_linear_workspace_size(M, K)`` bytes."""
    _native.w4a16_linear(X, inv_smooth, Wq, w_scale, group, bias, Y, workspace, epi, stream)


# ---------------------------------------------------------------------------------------- paged cache

class QVKVCache:
    """A paged cache of keys and values over the caller's tensors: k_pages, v_pages [pages, heads, page_size, D]
    (bf16; int8 with k_scale, v_scale [pages, heads, page_size] fp32; or float8_e4m3fn with k_scale, v_scale [pages,
    heads, blocks] fp32, one for each block of page_size / blocks tokens, a multiple of 16), D 64 or 128, unit channel
    stride, the same strides in both; a permuted [pages, page_size, heads, D] tensor fits.  Holds the tensors, checks
    them once and allocates nothing; a tensor put in another's place needs a new QVKVCache."""

    __slots__ = ("_k", "_v", "_ks", "_vs", "_handle", "pages", "heads", "page_size", "head_dim")

    def __init__(self, k_pages, v_pages, k_scale=None, v_scale=None):
        self._k, self._v, self._ks, self._vs = k_pages, v_pages, k_scale, v_scale
        self._handle, self.pages, self.heads, self.page_size, self.head_dim = _native.kv_cache(k_pages, v_pages, k_scale,
                                                                                               v_scale)

    k_pages = property(lambda self: self._k)
    v_pages = property(lambda self: self._v)
    k_scale = property(lambda self: self._ks)
    v_scale = property(lambda self: self._vs)


def qv_kv_append(cache, page_table, token_seq, token_index, K, V, cos=None, sin=None, position=None, Q=None,
                 Q_out=None, stream=None) -> None:
    """Store the keys K and values V [T, heads, D] (fp32/bf16) of T new tokens in ``cache``, K turned by position.

    page_table [sequences, pages] int32; token_seq [T] int32 sequence of each token (None: token t is sequence t);
    token_index [T] int32 place of each token in its sequence; cos, sin [places, D / (2 axes)] fp32 (None: no
    rotation); position [T, axes] int32 with 1 or 2 axes (None: token_index).  Q [T, q_heads, D] is turned into
    Q_out (which may be Q).  A float8_e4m3fn cache takes the tokens of a block in the order of their places, next to each
    other; a block that was begun by an earlier call keeps its scale or has its codes rounded again by a larger one."""
    _native.kv_append(getattr(cache, "_handle", None), page_table, token_seq, token_index, K, V, cos, sin, position, Q,
                      Q_out, stream)


def qv_paged_attention_workspace_size(B: int, q_heads: int, heads: int, head_dim: int, capacity: int) -> int:
    return int(_lib().qv_paged_attention_workspace_size(int(B), int(q_heads), int(heads), int(head_dim), int(capacity)))


def qv_paged_attention(Q, cache, page_table, lens, O, workspace, scale=None, window: int = 0, stream=None) -> None:
    """O [B, q_heads, D]: attention of one new token Q [B, q_heads, D] (fp32/bf16) of each sequence over the last
    ``window`` (0: all) of its lens[b] tokens in ``cache``; scale defaults to D ** -0.5.  ``workspace`` holds at
    least ``qv_paged_attention_workspace_size(B, q_heads, heads, D, page_table.shape[1] * page_size)`` bytes."""
    _native.paged_attention(Q, getattr(cache, "_handle", None), page_table, lens, O, workspace, scale, window, stream)
