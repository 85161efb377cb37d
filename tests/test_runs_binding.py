"""The binding of the entry points for runs of tokens, and of FP8 caches, checks every tensor before the C call (CPU only: each case
fails in the checks, so nothing reaches the library or the GPU)."""
import pytest

torch = pytest.importorskip("torch")

import bit_ptq_reconstruction_amd as qv  # noqa: E402
from test_decode_binding import Handle, bf, built, i32, refused, u8  # noqa: E402,F401

i64 = lambda *s: torch.zeros(s, dtype=torch.int64)


def attend(**kw):
    a = dict(Q=bf(7, 6, 64), starts=i32(4), max_run=5, cache=Handle(), page_table=i32(3, 4), lens=i32(3), O=bf(7, 6, 64),
             workspace=u8(1 << 20))
    a.update(kw)
    qv.qv_run_attention(**a)


@pytest.mark.parametrize("match,change", [
    ("must be a QVKVCache", dict(cache=None)), ("Q is bfloat16", dict(Q=bf(7, 5, 64))), ("Q is bfloat16", dict(Q=bf(7, 6, 128))),
    ("Q is float16", dict(Q=bf(7, 6, 64).half())), ("Q is required", dict(Q=None)), ("O is float32", dict(O=torch.zeros(7, 6, 64))),
    ("O is bfloat16", dict(O=bf(6, 6, 64))), ("do not overlap", dict(O=bf(1, 6, 64).expand(7, 6, 64))),
    ("starts is int32", dict(starts=i32(3))), ("starts is int64", dict(starts=i64(4))), ("page_table is int64", dict(page_table=i64(3, 4))),
    ("lens is int32", dict(lens=i32(4))), ("max_run 8 of 7 rows", dict(max_run=8)), ("max_run -1 of 7 rows", dict(max_run=-1)),
    ("7 rows of 3 sequences in runs of up to 5 need starts", dict(starts=None)),
    ("3 rows of 3 sequences in runs of up to 2 need starts", dict(starts=None, Q=bf(3, 6, 64), O=bf(3, 6, 64), max_run=2)),
    ("window -1", dict(window=-1)), ("sinks -2", dict(sinks=-2)), ("workspace holds", dict(workspace=u8(255))),
    ("workspace is required", dict(workspace=None)), ("GPU tensor", {}), ("GPU tensor", dict(scale=0.3, window=7, sinks=2, causal=False)),
    ("GPU tensor", dict(starts=None, Q=bf(3, 6, 64), O=bf(3, 6, 64), max_run=1)),
])
def test_attention(match, change):
    refused(attend, match, **change)


def test_attention_types():
    for bad in (dict(max_run="5"), dict(max_run=2.0), dict(window=None), dict(sinks=1.5), dict(scale="x")):
        with pytest.raises(TypeError):
            attend(**bad)


def tables(**kw):
    a = dict(runs=i32(3), lens=i32(3), free_pages=i32(9), free_count=i32(1), page_size=16, page_table=i32(3, 4), starts=i32(4),
             lens_out=i32(3), free_left=i32(1), token_seq=i32(20), token_index=i32(20), slots=i64(20), status=i32(3))
    a.update(kw)
    qv.qv_page_tables(**a)


@pytest.mark.parametrize("match,change", [
    ("runs is int32", dict(runs=i32(2))), ("runs is int64", dict(runs=i64(3))), ("lens is int32", dict(lens=i32(3, 1))),
    ("free_pages is int64", dict(free_pages=i64(9))), ("free_pages is int32", dict(free_pages=i32(3, 3))),
    ("free_pages is int32", dict(free_pages=i32(18)[::2])), ("free_count is int32", dict(free_count=i32(2))),
    ("page_size 0", dict(page_size=0)), ("page_size -16", dict(page_size=-16)), ("page_table is int32", dict(page_table=i32(12))),
    ("page_table is int32", dict(page_table=i32(4, 3).t())), ("page_table is int32", dict(page_table=i32(1, 4).expand(3, 4))),
    ("starts is int32", dict(starts=i32(3))), ("lens_out is int32", dict(lens_out=i32(4))), ("free_left is int32", dict(free_left=i32(0))),
    ("token_seq is int64", dict(token_seq=i64(20))), ("token_index is int32", dict(token_index=i32(19))), ("slots is int32", dict(slots=i32(20))),
    ("status is int32", dict(status=i32(2))), ("status is required", dict(status=None)), ("GPU tensor", {}),
    ("GPU tensor", dict(free_pages=i32(0))), ("GPU tensor", dict(token_seq=i32(0), token_index=i32(0), slots=i64(0))),
])
def test_tables(match, change):
    refused(tables, match, **change)


def test_fp8_cache():
    f8 = lambda *s: torch.zeros(s).to(torch.float8_e4m3fn)
    k, s = f8(4, 2, 64, 64), torch.zeros(4, 2, 2)
    for match, args in (("k_scale is required", (k, k)), ("v_scale is required", (k, k, s)), ("v_pages is int8", (k, k.view(torch.int8))),
                        ("k_scale is float32", (k, k, torch.zeros(4, 2, 3), s)), ("k_scale is float32", (k, k, torch.zeros(4, 2, 8), s)),
                        ("k_scale is float32", (k, k, torch.zeros(4, 2), s)), ("k_scale is float32", (k, k, torch.zeros(4, 2, 0), s)),
                        ("k_scale is float64", (k, k, s.double(), s)), ("v_scale is float32", (k, k, s, torch.zeros(4, 2, 4))),
                        ("k_scale is float32", (k, k, torch.zeros(3, 2, 2), s)),
                        ("k_pages is float8_e5m2", (k.to(torch.float8_e5m2), k.to(torch.float8_e5m2), s, s)),
                        ("GPU tensor", (k, k, s, s)), ("GPU tensor", (k, k, torch.zeros(4, 2, 4), torch.zeros(4, 2, 4)))):
        with pytest.raises(ValueError, match=match):
            qv.QVKVCache(*args)


def test_names():
    assert qv.QV_KV_FP8 == 2 and [qv.QV_RUN_OK, qv.QV_RUN_NO_ROOM, qv.QV_RUN_NO_PAGES, qv.QV_RUN_NO_ROWS] == [0, 1, 2, 3]


def test_stream_block_of_two_caches():
    """Refused before anything is allocated."""
    from bit_ptq_reconstruction_amd.stream import StreamBlock

    with pytest.raises(ValueError, match="int8 or FP8"):
        StreamBlock(None, {}, 1, 16, "cpu", int8_cache=True, fp8_cache=True)
