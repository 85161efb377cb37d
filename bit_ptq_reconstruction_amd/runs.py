"""Entry points for runs of tokens (C ABI in ``include/qv_runs.h``): prompts, frames, chunks and guessed tokens of many
sequences at once, over the paged cache of ``decode``.  Page tables and slots are worked out on the GPU from the tokens
that join each sequence, and each sequence's new tokens attend to its cache, within a window and to its first tokens.

Operands are checked as in ``decode``: shapes, types, layouts and devices before the library is called (ValueError), a
non-OK status raises QVError, and there is no fallback.
"""
from __future__ import annotations

import ctypes

from . import decode, lib

__all__ = [
    "qv_page_tables", "qv_run_attention", "qv_run_attention_workspace_size", "QV_RUN_OK", "QV_RUN_NO_ROOM",
    "QV_RUN_NO_PAGES", "QV_RUN_NO_ROWS",
]

QV_RUN_OK, QV_RUN_NO_ROOM, QV_RUN_NO_PAGES, QV_RUN_NO_ROWS = range(4)


def bind(L):
    """Declare the C signatures of these entry points on a loaded library handle and return it."""
    P, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    L.qv_page_tables.argtypes = [P, P, i64, i64, P, i64, P, P, i64, i64, P, P, P, P, P, P, i64, P, P]
    L.qv_run_attention_workspace_size.argtypes = [i64] * 7
    L.qv_run_attention_workspace_size.restype = sz
    L.qv_run_attention.argtypes = [P, i32, i64, i64, P, i64, i64, P, P, i64, i64, P, f32, i64, i64, i32, P, P, sz, P]
    for name in ("qv_page_tables", "qv_run_attention"):
        getattr(L, name).restype = i32
    return L


_bound = None


def _lib():
    global _bound
    if _bound is None:
        _bound = bind(lib())
    return _bound


def qv_page_tables(runs, lens, free_pages, free_count, page_size: int, page_table, starts, lens_out, free_left, token_seq,
                   token_index, slots, status, stream=None) -> None:
    """Pages, places and slots for runs[b] new tokens of each sequence b, which has lens[b] ([B] int32 both).

    The first free_count [1] of free_pages [F] are free (int32 both) and are taken from the end; page_table [B, pages] int32
    gets the new ones.  Out: starts [B + 1] int32 (rows starts[b] to starts[b + 1] - 1 are those of sequence b), lens_out [B]
    (may be lens), free_left [1] (may be free_count), token_seq, token_index [T] int32 and slots [T] int64 (-1 in rows without
    a token that has a place), status [B] int32: QV_RUN_OK, or why a sequence is refused as a whole (QV_RUN_NO_ROOM in the
    table, QV_RUN_NO_PAGES, QV_RUN_NO_ROWS: its rows pass T)."""
    decode._native.page_tables(runs, lens, free_pages, free_count, page_size, page_table, starts, lens_out, free_left,
                               token_seq, token_index, slots, status, stream)


def qv_run_attention_workspace_size(T: int, B: int, max_run: int, q_heads: int, heads: int, head_dim: int,
                                    capacity: int) -> int:
    return int(_lib().qv_run_attention_workspace_size(int(T), int(B), int(max_run), int(q_heads), int(heads), int(head_dim),
                                                      int(capacity)))


def qv_run_attention(Q, starts, max_run: int, cache, page_table, lens, O, workspace, scale=None, window: int = 0,
                     sinks: int = 0, causal: bool = True, stream=None) -> None:
    """O [T, q_heads, D]: attention of each sequence's new tokens, its last ones, over its lens[b] tokens in ``cache``.

    Rows starts[b] to starts[b + 1] - 1 of Q [T, q_heads, D] (fp32/bf16) are those of sequence b (starts [B + 1] int32; None:
    row b is sequence b's one token), up to ``max_run`` of them (a longer run is its first ``max_run`` rows, taken for the
    sequence's last tokens).  A token sees those up to itself (``causal``) or all of its
    sequence, and of these the last ``window`` up to itself (0: all) and the first ``sinks``; scale defaults to D ** -0.5.
    ``workspace`` holds at least ``qv_run_attention_workspace_size(T, B, max_run, q_heads, heads, D, page_table.shape[1] *
    page_size)`` bytes."""
    decode._native.run_attention(Q, starts, max_run, getattr(cache, "_handle", None), page_table, lens, O, workspace, scale,
                                 window, sinks, causal, stream)
