"""Further calls that the single-token entry points refuse on the host (CPU only: nothing reaches the GPU)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import bit_ptq_reconstruction_amd as qv  # noqa: E402
from bit_ptq_reconstruction_amd.decode import QVKVCacheStruct  # noqa: E402
from test_decode_binding import append, attend, bf, built, refused  # noqa: E402,F401


def handle(heads=2, device=-1):
    """A cache's handle over no memory, of 16 slots and 64 channels."""
    class Bound(ctypes.Structure):
        _fields_ = [("c", QVKVCacheStruct), ("device", ctypes.c_int)]

    class Cache:
        _handle = bytes(Bound(QVKVCacheStruct(None, None, None, None, 0, heads, 16, 64, 2048, 1024, 64, 0), device))

    return Cache()


@pytest.mark.parametrize("shape", [(4, 0, 16, 64), (4, 2, 0, 64), (4, 2, 16, 0)])
def test_cache_without_heads(shape):
    """No heads, tokens or channels: refused where the cache is made, and again where its heads divide the queries'."""
    k = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="at least one head"):
        qv.QVKVCache(k, k)
    none = handle(heads=0)
    refused(attend, "no heads", cache=none)
    refused(attend, "no heads", cache=none, Q=bf(3, 0, 64), O=bf(3, 0, 64))
    refused(append, "GPU tensor", cache=none, K=bf(5, 0, 64), V=bf(5, 0, 64))
