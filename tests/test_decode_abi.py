"""The C ABI of the single-token entry points on the CPU: every call that include/qv_decode.h declares is
exported and rejects bad arguments on the host before any HIP call (no device is touched by these calls).
QV_DECODE_ABI_TEST_LIB names a host-only build with stub launchers, made by the last test here under
AddressSanitizer and UndefinedBehaviorSanitizer; there, a rejected call is also checked to have launched
nothing, and the calls that are accepted to have launched once."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

from bit_ptq_reconstruction_amd import decode  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qv_decode.h")
STUB_LIB = os.environ.get("QV_DECODE_ABI_TEST_LIB")

OK, NULL, SHAPE, UNSUPPORTED, ALIGN, DTYPE, WORKSPACE, HIP = range(8)
F32, BF16 = 0, 1
P = 0x100000  # an aligned dummy address: never dereferenced, because validation fails first
MIS = P + 4


@pytest.fixture(scope="module")
def L():
    if STUB_LIB:
        return decode.bind(ctypes.CDLL(STUB_LIB))
    import bit_ptq_reconstruction_amd as qv

    if not os.path.exists(qv.library_path()):
        from bit_ptq_reconstruction_amd.build import build_library

        build_library()
    return decode.bind(qv.lib())


@pytest.fixture(autouse=True)
def launches(request):
    if not STUB_LIB or "L" not in request.fixturenames:
        yield
        return
    L_ = request.getfixturevalue("L")
    L_.qv_stub_reset()
    yield
    assert L_.qv_stub_launches() == getattr(request.node, "accepted", 0)


def test_library_exports_every_declared_symbol(L):
    names = re.findall(r"^(?:qv_status|size_t)\s+(qv_\w+)\s*\(", open(HEADER).read(), re.M)
    assert len(names) == 6
    for name in names:
        assert hasattr(L, name), name


def gemv(L, X=P, xt=BF16, M=4, K=1024, ldx=1024, Wq=P, ws=P, group=128, bias=None, N=33, epi=0, Y=P, yt=BF16, ldy=33):
    return L.qv_w4a16_gemv(X, xt, M, K, ldx, Wq, ws, group, bias, N, epi, Y, yt, ldy, None)


def linear(L, inv=None, work=P, size=1 << 20, X=P, xt=BF16, M=4, K=1024, ldx=4096, Wq=P, ws=P, group=128, bias=None,
           N=33, epi=0, Y=P, yt=BF16, ldy=33):
    return L.qv_w4a16_linear(X, xt, M, K, ldx, inv, Wq, ws, group, bias, N, epi, Y, yt, ldy, work, size, None)


@pytest.mark.parametrize("call", [gemv, linear])
def test_few_row_linear_refusals(L, call):
    assert call(L, M=0, X=None) == OK and call(L, N=0, ldy=0, Y=None) == OK
    for name in ("X", "Wq", "ws", "Y"):
        assert call(L, **{name: None}) == NULL, name
        assert call(L, **{name: MIS}) == ALIGN, name
    assert call(L, bias=MIS) == ALIGN
    assert call(L, ldx=4100) == ALIGN                       # 8200 bytes
    assert call(L, M=-1) == SHAPE and call(L, N=-1) == SHAPE and call(L, K=0) == SHAPE
    assert call(L, ldx=1016) == SHAPE and call(L, ldy=32) == SHAPE
    assert call(L, ldx=1 << 62) == SHAPE and call(L, ldy=1 << 62) == SHAPE
    assert call(L, K=1000) == UNSUPPORTED
    for group in (64, 0, -128, 384, 2048):
        assert call(L, group=group) == UNSUPPORTED, group
    assert call(L, M=1 << 40) == UNSUPPORTED and call(L, N=1 << 31, ldy=1 << 31) == UNSUPPORTED
    assert call(L, xt=2) == DTYPE and call(L, yt=-1) == DTYPE and call(L, epi=2) == DTYPE


def test_few_row_linear_sizes(L):
    assert gemv(L, K=1 << 17, ldx=1 << 17) == UNSUPPORTED
    assert linear(L, K=2048) == UNSUPPORTED                 # a Hadamard width
    assert linear(L, inv=MIS) == ALIGN and linear(L, work=P + 16) == ALIGN
    assert linear(L, work=None) == WORKSPACE
    assert linear(L, size=4 * 1024 * 4 - 1) == WORKSPACE
    assert L.qv_w4a16_linear_workspace_size(3, 1024) == 3 * 4096
    assert L.qv_w4a16_linear_workspace_size(0, 1024) == 0
    assert L.qv_w4a16_linear_workspace_size(-1, 1024) == 0
    assert L.qv_w4a16_linear_workspace_size(1 << 40, 1 << 38) == 0


def cache(**kw):
    f = dict(k_pages=P, v_pages=P, k_scale=P, v_scale=P, num_pages=8, heads=2, page_size=16, head_dim=64,
             page_stride=2048, head_stride=1024, token_stride=64, dtype=0)
    f.update(kw)
    return ctypes.byref(decode.QVKVCacheStruct(*[f[n] for n, _ in decode.QVKVCacheStruct._fields_]))


def heads(data=P, ts=128, hs=64):
    return ctypes.byref(decode.QVHeadsStruct(data, ts, hs))


def append(L, cache_=None, table=P, seqs=3, pages=4, ld=4, seq=P, index=P, T=5, K=0, V=0, xt=BF16, cos=P, sin=P,
           places=9, axes=1, position=P, Q=0, Q_out=0, q_heads=2):
    k, v, q, o = (heads() if x == 0 else x for x in (K, V, Q, Q_out))
    return L.qv_kv_append(cache_ or cache(), table, seqs, pages, ld, seq, index, T, k, v, xt, cos, sin, places, axes,
                          position, q, o, q_heads, None)


def attend(L, cache_=None, Q=0, O=0, qt=BF16, B=3, q_heads=4, table=P, pages=4, ld=4, lens=P, window=0, work=P,
           size=1 << 20):
    q, o = (heads(ts=256) if x == 0 else x for x in (Q, O))
    return L.qv_paged_attention(q, qt, B, q_heads, cache_ or cache(), table, pages, ld, lens, 0.125, window, o, work,
                                size, None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_refusals(L, call):
    for f in ("k_pages", "v_pages"):
        assert call(L, cache(**{f: None})) == NULL and call(L, cache(**{f: MIS})) == ALIGN
    int8 = dict(dtype=1)
    for f in ("k_scale", "v_scale"):
        assert call(L, cache(**int8, **{f: None})) == NULL and call(L, cache(**int8, **{f: MIS})) == ALIGN
    assert call(L, cache(dtype=2)) == DTYPE
    for f in ("num_pages", "heads", "page_size", "head_dim"):
        assert call(L, cache(**{f: -1})) == SHAPE, f
    assert call(L, cache(heads=0)) == SHAPE
    assert call(L, cache(head_dim=96, token_stride=96)) == UNSUPPORTED
    assert call(L, cache(page_size=24)) == UNSUPPORTED and call(L, cache(page_size=1 << 17)) == UNSUPPORTED
    for f in ("page_stride", "head_stride", "token_stride"):
        assert call(L, cache(**{f: 32})) == SHAPE, f
        assert call(L, cache(**{f: 1 << 32})) == SHAPE, f
        assert call(L, cache(**{f: 1028})) == ALIGN, f
    assert call(L, cache(dtype=1, token_stride=72)) == ALIGN     # 72 bytes
    assert call(L, pages=5) == SHAPE                             # ld_table is 4
    assert call(L, pages=1 << 28, ld=1 << 28) == UNSUPPORTED     # 2^32 places
    assert call(L, table=None) == NULL and call(L, table=P + 2) == ALIGN


def test_append_refusals(L):
    assert append(L, T=0, K=None, V=None, index=None, Q=None, Q_out=None, q_heads=0) == OK
    assert append(L, T=-1) == SHAPE and append(L, xt=3) == DTYPE
    assert append(L, K=None) == NULL and append(L, V=None) == NULL and append(L, index=None) == NULL
    assert append(L, K=heads(None)) == NULL and append(L, V=heads(MIS)) == ALIGN
    assert append(L, K=heads(hs=56)) == SHAPE and append(L, Q=heads(ts=-8)) == SHAPE
    assert append(L, K=heads(ts=132)) == ALIGN and append(L, Q_out=heads(hs=68)) == ALIGN
    assert append(L, seq=None, seqs=4) == SHAPE                  # five tokens of four sequences
    assert append(L, axes=0) == UNSUPPORTED and append(L, axes=3) == UNSUPPORTED
    assert append(L, cos=None) == NULL and append(L, sin=None) == NULL
    assert append(L, axes=2, position=None) == NULL
    assert append(L, places=-1) == SHAPE
    assert append(L, cos=MIS) == ALIGN and append(L, position=P + 1) == ALIGN and append(L, index=P + 2) == ALIGN
    assert append(L, Q_out=None) == NULL and append(L, q_heads=0) == NULL and append(L, Q=None, Q_out=None) == NULL


def test_attention_refusals(L):
    assert attend(L, B=0, Q=None, O=None, lens=None) == OK
    assert attend(L, B=-1) == SHAPE and attend(L, q_heads=3) == SHAPE and attend(L, q_heads=0) == SHAPE
    assert attend(L, window=-1) == SHAPE and attend(L, qt=2) == DTYPE
    assert attend(L, Q=None) == NULL and attend(L, O=None) == NULL and attend(L, lens=None) == NULL
    assert attend(L, Q=heads(MIS)) == ALIGN and attend(L, lens=P + 1) == ALIGN
    assert attend(L, B=1 << 30) == UNSUPPORTED
    assert attend(L, work=None) == WORKSPACE and attend(L, size=255) == WORKSPACE
    assert attend(L, work=P + 16) == ALIGN
    size = L.qv_paged_attention_workspace_size
    assert size(1, 4, 2, 64, 0) == 256 and size(0, 4, 2, 64, 100) >= 256
    assert size(1, 4, 2, 64, 4096) > 256
    for bad in ((-1, 4, 2, 64, 64), (1, 3, 2, 64, 64), (1, 4, 0, 64, 64), (1, 4, 2, 80, 64), (1, 4, 2, 64, -1),
                (1, 4, 2, 64, 1 << 40), (1 << 40, 4, 2, 64, 64)):
        assert size(*bad) == 0, bad


@pytest.mark.skipif(not STUB_LIB, reason="only meaningful in the host-only stub build")
def test_stub_counts_valid_calls(L, request):
    """Valid calls pass the checks and reach a (stub) launcher, whose failure is reported."""
    calls = [gemv(L), linear(L), append(L), append(L, Q=None, Q_out=None, q_heads=0, cos=None, sin=None, position=None),
             append(L, seq=None, T=3), append(L, axes=2), attend(L), attend(L, cache(num_pages=0, k_pages=None)),
             attend(L, pages=0, ld=0, table=None), gemv(L, group=1024), linear(L, K=4096, group=4096)]
    assert calls == [HIP] * len(calls)
    request.node.accepted = len(calls)


def test_checks_under_sanitizers(tmp_path):
    import sys

    from test_sanitizers import SAN, _env, _runtime

    if STUB_LIB:
        return
    _runtime()
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    csrc, stubs = os.path.join(ROOT, "bit_ptq_reconstruction_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    so = str(tmp_path / "libqv_decode_stub.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", *SAN, "-I", stubs, "-I",
                    os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "qv_decode_abi.cpp"),
                    os.path.join(stubs, "decode_stubs.cpp"), "-o", so], check=True, capture_output=True, text=True)
    logs = tmp_path / "logs"
    logs.mkdir()
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", __file__], cwd=ROOT,
                       env=_env(logs, QV_DECODE_ABI_TEST_LIB=so), capture_output=True, text=True, timeout=600)
    reports = "".join(open(os.path.join(logs, f)).read() for f in sorted(os.listdir(logs)))
    assert not reports, reports[-3000:]
    assert r.returncode == 0 and " passed" in r.stdout and "skipped" not in r.stdout, (r.stdout + r.stderr)[-3000:]
