"""The binding of the single-token entry points checks every tensor before the C call (CPU only: each case
fails in the checks, so nothing reaches the library or the GPU)."""
import os

import pytest

torch = pytest.importorskip("torch")

import bit_ptq_reconstruction_amd as qv  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_ptq_reconstruction_amd import build

    if not (os.path.exists(build.LIB) and os.path.exists(build.BINDING)):
        build.build_library()


M, K, N = 3, 1024, 40
u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)


def refused(f, match, **change):
    with pytest.raises(ValueError, match=match):
        f(**change)


def gemv(**kw):
    a = dict(X=bf(M, K), Wq=u8(N, K // 2), w_scale=torch.ones(N, 8), group=128, bias=None, Y=bf(M, N))
    a.update(kw)
    qv.qv_w4a16_gemv(**a)


def linear(**kw):
    a = dict(X=bf(M, K), inv_smooth=torch.ones(K), Wq=u8(N, K // 2), w_scale=torch.ones(N, 8), group=128, bias=None,
             Y=bf(M, N), workspace=u8(M * K * 4))
    a.update(kw)
    qv.qv_w4a16_linear(**a)


@pytest.mark.parametrize("call", [gemv, linear])
@pytest.mark.parametrize("match,change", [
    ("X is required", dict(X=None)), ("X must be a torch tensor", dict(X=[1])),
    ("X is float16", dict(X=torch.zeros((M, K), dtype=torch.float16))), ("X is bfloat16", dict(X=bf(M * K))),
    ("X is bfloat16", dict(X=bf(K, M).t())), ("Wq is uint8", dict(Wq=u8(N, K // 2 - 16))),
    ("Wq is int8", dict(Wq=u8(N, K // 2).view(torch.int8))), ("Wq is uint8", dict(Wq=u8(N, K)[:, ::2])),
    ("w_scale is float32", dict(w_scale=torch.ones(N, 7))), ("w_scale is float32", dict(w_scale=torch.ones(N))),
    ("w_scale is required", dict(w_scale=None)), ("w_scale is float64", dict(w_scale=torch.ones(N, 8).double())),
    ("group 100", dict(group=100)), ("group 0", dict(group=0)), ("group -128", dict(group=-128)),
    ("bias is float32", dict(bias=torch.ones(N - 1))), ("bias is bfloat16", dict(bias=bf(N))),
    ("Y is bfloat16", dict(Y=bf(M, N + 1))), ("Y is bfloat16", dict(Y=bf(N, M).t())),
    ("Y is float64", dict(Y=torch.zeros((M, N), dtype=torch.float64))), ("Y is required", dict(Y=None)),
    ("GPU tensor", {}), ("GPU tensor", dict(X=bf(M, K + 8)[:, :K], Y=bf(M, N + 3)[:, :N])),
    ("GPU tensor", dict(w_scale=torch.ones(N), group=K)), ("GPU tensor", dict(w_scale=torch.ones(N, 1), group=K)),
])
def test_linears(call, match, change):
    refused(call, match, **change)


def test_linear_own():
    refused(linear, "inv_smooth is float32", inv_smooth=torch.ones(K - 1))
    refused(linear, "workspace holds", workspace=u8(M * K * 4 - 1))
    refused(linear, "workspace is required", workspace=None)
    refused(linear, "workspace is int8", workspace=u8(M * K * 4).view(torch.int8))
    with pytest.raises(TypeError):
        gemv(group="128")
    with pytest.raises(TypeError):
        gemv(epi=0.5)


def test_cache():
    kv = lambda **kw: torch.zeros((4, 2, 16, 64), **{"dtype": torch.bfloat16, **kw})
    i8 = kv(dtype=torch.int8)
    s = torch.zeros((4, 2, 16))
    for match, args in (("k_pages is required", (None, kv())), ("k_pages is float32", (kv().float(), kv().float())),
                        ("v_pages is int8", (kv(), i8)), ("v_pages is bfloat16", (kv(), kv()[:3])),
                        ("v_pages is bfloat16", (kv(), torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16).transpose(1, 2))),
                        ("k_pages is bfloat16", (kv().transpose(2, 3), kv().transpose(2, 3))),
                        ("k_scale is required", (i8, i8)), ("v_scale is required", (i8, i8, s)),
                        ("v_scale is float32", (i8, i8, s, s[:3])), ("no scales", (kv(), kv(), s, s)),
                        ("do not overlap", (kv()[:1].expand(4, 2, 16, 64),) * 2),
                        ("GPU tensor", (kv(), kv())), ("GPU tensor", (i8, i8, s, s))):
        with pytest.raises(ValueError, match=match):
            qv.QVKVCache(*args)


class Handle:
    """A cache's handle over no memory, of 2 heads, 16 slots and 64 channels: the checks see no more of it."""

    def __init__(self, device=-1):
        import ctypes

        from bit_ptq_reconstruction_amd.decode import QVKVCacheStruct

        class Bound(ctypes.Structure):
            _fields_ = [("c", QVKVCacheStruct), ("device", ctypes.c_int)]

        c = QVKVCacheStruct(None, None, None, None, 0, 2, 16, 64, 2048, 1024, 64, 0)
        self._handle = bytes(Bound(c, device))


def append(**kw):
    a = dict(cache=Handle(), page_table=i32(3, 4), token_seq=i32(5), token_index=i32(5), K=bf(5, 2, 64), V=bf(5, 2, 64),
             cos=torch.zeros(9, 32), sin=torch.zeros(9, 32), position=i32(5, 1), Q=bf(5, 6, 64), Q_out=bf(5, 6, 64))
    a.update(kw)
    qv.qv_kv_append(**a)


@pytest.mark.parametrize("match,change", [
    ("must be a QVKVCache", dict(cache=None)), ("must be a QVKVCache", dict(cache=bf(4, 2, 16, 64))),
    ("page_table is int64", dict(page_table=i32(3, 4).long())), ("page_table is int32", dict(page_table=i32(12))),
    ("page_table is int32", dict(page_table=i32(4, 3).t())), ("token_index is int32", dict(token_index=i32(4))),
    ("token_index is required", dict(token_index=None)), ("token_seq is int64", dict(token_seq=i32(5).long())),
    ("5 tokens of 3 sequences", dict(token_seq=None)), ("K is bfloat16", dict(K=bf(5, 3, 64))),
    ("K is float16", dict(K=bf(5, 2, 64).half())), ("V is float32", dict(V=bf(5, 2, 64).float())),
    ("V is bfloat16", dict(V=bf(4, 2, 64))), ("K is bfloat16", dict(K=bf(5, 64, 2).transpose(1, 2))),
    ("K is bfloat16", dict(K=bf(5, 1, 64).expand(5, 2, 64))), ("cos and sin", dict(sin=None)),
    ("cos is float32", dict(cos=torch.zeros(9, 16))), ("sin is float32", dict(sin=torch.zeros(8, 32))),
    ("cos is bfloat16", dict(cos=bf(9, 32))), ("position is int32", dict(position=i32(5, 3))),
    ("position is int32", dict(position=i32(4, 1))), ("cos is float32", dict(position=i32(5, 2))),
    ("Q and Q_out", dict(Q=None)), ("Q and Q_out", dict(Q_out=None)), ("Q is bfloat16", dict(Q=bf(5, 384))),
    ("Q_out is bfloat16", dict(Q_out=bf(5, 5, 64))), ("Q is float32", dict(Q=torch.zeros(5, 6, 64))),
    ("GPU tensor", {}), ("GPU tensor", dict(K=bf(5, 10, 64)[:, 6:8], V=bf(5, 10, 64)[:, 8:])),
    ("GPU tensor", dict(position=i32(5, 2), cos=torch.zeros(9, 16), sin=torch.zeros(9, 16))),
    ("GPU tensor", dict(position=None, cos=None, sin=None, Q=None, Q_out=None)),
    ("GPU tensor", dict(page_table=i32(3, 9)[:, 2:6])),
])
def test_append(match, change):
    refused(append, match, **change)


def attend(**kw):
    a = dict(Q=bf(3, 6, 64), cache=Handle(), page_table=i32(3, 4), lens=i32(3), O=bf(3, 6, 64), workspace=u8(1 << 16))
    a.update(kw)
    qv.qv_paged_attention(**a)


@pytest.mark.parametrize("match,change", [
    ("must be a QVKVCache", dict(cache=None)), ("Q is bfloat16", dict(Q=bf(3, 5, 64))),
    ("Q is bfloat16", dict(Q=bf(3, 6, 128))), ("Q is float16", dict(Q=bf(3, 6, 64).half())),
    ("O is float32", dict(O=torch.zeros(3, 6, 64))), ("O is bfloat16", dict(O=bf(3, 4, 64))),
    ("page_table is int32", dict(page_table=i32(2, 4))), ("lens is int64", dict(lens=i32(3).long())),
    ("lens is int32", dict(lens=i32(4))), ("window -1", dict(window=-1)), ("workspace holds", dict(workspace=u8(255))),
    ("workspace is required", dict(workspace=None)), ("GPU tensor", {}), ("GPU tensor", dict(scale=0.3, window=7)),
])
def test_attention(match, change):
    refused(attend, match, **change)


def test_names():
    for name in qv.__all__:
        assert getattr(qv, name) is not None
    with pytest.raises(AttributeError):
        qv.qv_no_such_call
