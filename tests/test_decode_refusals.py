"""Further calls that the single-token entry points refuse on the host (CPU only: nothing reaches the GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

import bit_ptq_reconstruction_amd as qv  # noqa: E402
from bit_ptq_reconstruction_amd.decode import QVKVCacheStruct  # noqa: E402
from test_decode_abi import ROOT, SHAPE, UNSUPPORTED, WORKSPACE, L, gemv, linear  # noqa: E402,F401
from test_decode_abi import append as abi_append, attend as abi_attend, heads as abi_heads  # noqa: E402
from test_decode_binding import append, attend, bf, built, i32, refused  # noqa: E402,F401


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


def overlap(T, ts, H, hs, D):
    """Rows of D elements at t ts + h hs, counted out."""
    seen = set()
    for t in range(T):
        for h in range(H):
            row = set(range(t * ts + h * hs, t * ts + h * hs + D))
            if row & seen:
                return True
            seen |= row
    return False


def test_overlapping_outputs():
    """Outputs expanded along the tokens, or laid out so that rows share memory, are refused; inputs may be."""
    same = torch.zeros((1, 6, 64), dtype=torch.bfloat16)
    refused(attend, "O is bfloat16 .* do not overlap", O=same.expand(3, 6, 64))
    refused(append, "Q_out is bfloat16 .* do not overlap", Q_out=same.expand(5, 6, 64))
    refused(attend, "GPU tensor", Q=same.expand(3, 6, 64))
    refused(append, "GPU tensor", Q=same.expand(5, 6, 64))
    flat = bf(1 << 14)
    refused(attend, "O is bfloat16 .* do not overlap", O=flat.as_strided((3, 6, 64), (64, 64, 1)))
    refused(attend, "O is bfloat16 .* do not overlap", O=flat.as_strided((3, 6, 64), (192, 128, 1)))
    refused(attend, "GPU tensor", O=flat.as_strided((3, 6, 64), (64, 192, 1)))     # heads outside tokens
    refused(attend, "GPU tensor", O=flat.as_strided((2, 2, 64), (192, 128, 1)), Q=bf(2, 2, 64), page_table=i32(2, 4),
            lens=i32(2))                                                          # 0, 128, 192, 320


def test_overlapping_outputs_of_the_library(L):
    """Every small layout, against the rows counted out."""
    for T, H in ((1, 2), (2, 2), (2, 4), (3, 2), (5, 4)):
        for ts in range(0, 449, 64):
            for hs in range(64, 449, 64):
                bad = overlap(T, ts, H, hs, 64)
                got = abi_attend(L, O=abi_heads(ts=ts, hs=hs), Q=abi_heads(ts=256), B=T, q_heads=H, size=0)
                assert got == (SHAPE if bad else WORKSPACE), (T, H, ts, hs)
    assert abi_append(L, Q_out=abi_heads(ts=0)) == SHAPE and abi_append(L, Q_out=abi_heads(ts=64, hs=256)) == SHAPE


def test_sizes_that_no_launch_holds(L):
    """A launch holds fewer than 2^32 threads along a dimension: what passes that is refused before the first one."""
    most = (1 << 29) - 64
    assert gemv(L, N=most + 1, ldy=1 << 40) == UNSUPPORTED and linear(L, N=most + 1, ldy=1 << 40) == UNSUPPORTED
    assert linear(L, N=most, ldy=1 << 40, work=None) == WORKSPACE
    size = L.qv_paged_attention_workspace_size
    short = dict(q_heads=4, pages=4)                          # 64 tokens: no join; two blocks of 256 threads a sequence
    assert abi_attend(L, B=1 << 23, **short) == UNSUPPORTED and size(1 << 23, 4, 2, 64, 64) == 0
    assert abi_attend(L, B=(1 << 23) - 1, work=None, **short) == WORKSPACE and size((1 << 23) - 1, 4, 2, 64, 64) == 256
    long = dict(q_heads=32, pages=16, ld=16, O=abi_heads(ts=2048))  # 256 tokens: a join of 128 threads a query head
    assert abi_attend(L, B=1 << 20, **long) == UNSUPPORTED and size(1 << 20, 32, 2, 64, 256) == 0
    assert abi_attend(L, B=(1 << 20) - 1, work=None, **long) == WORKSPACE and size((1 << 20) - 1, 32, 2, 64, 256) > 256


def test_parts_of_any_batch_have_room(tmp_path):
    """The attention's cut into parts against the room that the workspace has for them."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    stubs, exe = os.path.join(ROOT, "tests", "sanitize"), str(tmp_path / "parts_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", stubs, "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "bit_ptq_reconstruction_amd", "csrc"),
                    os.path.join(stubs, "parts_check.cpp"), "-o", exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_append_of_no_tokens(L):
    """No tokens, no positions: accepted with two axes as well."""
    assert abi_append(L, T=0, axes=2, position=None) == 0 and abi_append(L, T=1, axes=2, position=None) == 1
