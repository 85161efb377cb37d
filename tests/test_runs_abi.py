"""The C ABI of the entry points for runs of tokens, and of FP8 caches, on the CPU: bad arguments are rejected on the host before
any HIP call.  QV_RUNS_ABI_TEST_LIB names a host-only build with stub launchers, made by the last test here under AddressSanitizer
and UndefinedBehaviorSanitizer; there, a rejected call is also checked to have launched nothing."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest

pytest.importorskip("torch")

from bit_ptq_reconstruction_amd import decode, runs  # noqa: E402
from test_decode_abi import append as abi_append, attend as abi_attend  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STUB_LIB = os.environ.get("QV_RUNS_ABI_TEST_LIB")
OK, NULL, SHAPE, UNSUPPORTED, ALIGN, DTYPE, WORKSPACE, HIP = range(8)
F32, BF16 = 0, 1
P = 0x100000  # an aligned dummy address: never dereferenced, because validation fails first
MIS = P + 2


@pytest.fixture(scope="module")
def L():
    if STUB_LIB:
        return runs.bind(ctypes.CDLL(STUB_LIB))
    import bit_ptq_reconstruction_amd as qv

    if not os.path.exists(qv.library_path()):
        from bit_ptq_reconstruction_amd.build import build_library

        build_library()
    return runs.bind(decode.bind(qv.lib()))


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
    names = re.findall(r"^(?:qv_status|size_t)\s+(qv_\w+)\s*\(", open(os.path.join(ROOT, "include", "qv_runs.h")).read(), re.M)
    assert len(names) == 3
    for name in names:
        assert hasattr(L, name), name


def cache(**kw):
    f = dict(k_pages=P, v_pages=P, k_scale=P, v_scale=P, num_pages=8, heads=2, page_size=32, head_dim=64, page_stride=4096,
             head_stride=2048, token_stride=64, dtype=0, scale_tokens=0)
    f.update(kw)
    return ctypes.byref(decode.QVBlockCacheStruct(*[f[n] for n, _ in decode.QVBlockCacheStruct._fields_]))


def heads(data=P, ts=256, hs=64):
    return ctypes.byref(decode.QVHeadsStruct(data, ts, hs))


def attend(L, Q=0, qt=BF16, T=12, q_heads=4, starts=P, B=3, max_run=5, cache_=None, table=P, pages=4, ld=4, lens=P, window=0,
           sinks=0, causal=1, O=0, work=P, size=1 << 24):
    q, o = (heads() if x == 0 else x for x in (Q, O))
    return L.qv_run_attention(q, qt, T, q_heads, starts, B, max_run, cache_ or cache(), table, pages, ld, lens, 0.125, window,
                              sinks, causal, o, work, size, None)


def tables(L, runs_=P, lens=P, B=3, page=16, free=P, F=9, count=P, table=P, pages=4, ld=4, starts=P, after=P, left=P, seq=P,
           index=P, slots=P, T=20, status=P):
    return L.qv_page_tables(runs_, lens, B, page, free, F, count, table, pages, ld, starts, after, left, seq, index, slots, T,
                            status, None)


def test_fp8_cache_refusals(L):
    calls = [attend] if STUB_LIB else [attend, abi_append, abi_attend]
    for call in calls:
        fp8 = lambda **kw: cache(dtype=2, scale_tokens=16, **kw) if "scale_tokens" not in kw else cache(dtype=2, **kw)
        assert call(L, cache_=fp8(scale_tokens=0)) == DTYPE
        for n in (-16, 8, 24, 64):
            assert call(L, cache_=fp8(scale_tokens=n)) == UNSUPPORTED, n
        for f in ("k_scale", "v_scale"):
            assert call(L, cache_=fp8(**{f: None})) == NULL and call(L, cache_=fp8(**{f: MIS})) == ALIGN
        assert call(L, cache_=fp8(token_stride=72)) == ALIGN
        assert call(L, cache_=cache(dtype=3)) == DTYPE


def test_attention_refusals(L):
    assert attend(L, T=0, max_run=0, Q=None, O=None, lens=None) == OK
    assert attend(L, B=0, lens=None, table=None, pages=0, ld=0) == OK and attend(L, max_run=0) == OK
    assert attend(L, T=-1) == SHAPE and attend(L, B=-1) == SHAPE and attend(L, max_run=-1) == SHAPE and attend(L, max_run=13) == SHAPE
    assert attend(L, q_heads=3) == SHAPE and attend(L, q_heads=0) == SHAPE and attend(L, window=-1) == SHAPE
    assert attend(L, sinks=-1) == SHAPE and attend(L, qt=2) == DTYPE
    assert attend(L, starts=None) == SHAPE                                    # 12 rows of 3 sequences
    assert attend(L, starts=None, T=3, B=3, max_run=2) == SHAPE
    for name in ("Q", "O", "lens"):
        assert attend(L, **{name: None}) == NULL, name
    assert attend(L, table=None) == NULL and attend(L, table=MIS + 1) == ALIGN
    assert attend(L, starts=MIS + 1) == ALIGN and attend(L, lens=MIS + 1) == ALIGN and attend(L, Q=heads(MIS)) == ALIGN
    assert attend(L, O=heads(ts=0)) == SHAPE and attend(L, O=heads(ts=64, hs=64)) == SHAPE   # rows that share memory
    assert attend(L, work=None) == WORKSPACE and attend(L, work=P + 64) == ALIGN
    assert attend(L, pages=1 << 27, ld=1 << 27) == UNSUPPORTED                # 2^32 places
    assert attend(L, pages=(1 << 26) - 1, ld=1 << 26) == UNSUPPORTED          # 2^31 - 32: the last step passes 2^31
    assert attend(L, T=1 << 31, B=1 << 31, max_run=1) == UNSUPPORTED
    assert attend(L, T=1 << 30, B=1 << 30, max_run=1) == UNSUPPORTED
    assert attend(L, T=1 << 28, max_run=1 << 28) == UNSUPPORTED               # rows of a join


@pytest.mark.parametrize("T,B,max_run,q_heads,pages", [(12, 3, 5, 4, 4), (40, 3, 16, 4, 300), (80, 3, 30, 4, 300),
                                                       (200, 3, 100, 4, 3000), (9, 3, 5, 64, 300)])
def test_workspace(L, T, B, max_run, q_heads, pages):
    size = L.qv_run_attention_workspace_size(T, B, max_run, q_heads, 2, 64, pages * 32)
    assert size >= 256 and size % 256 == 0
    call = lambda n: attend(L, T=T, B=B, max_run=max_run, q_heads=q_heads, pages=pages, ld=pages, size=n, Q=heads(ts=4096),
                            O=heads(ts=4096), work=None if n is None else P)
    assert call(size - 1) == WORKSPACE


def test_workspace_sizes(L):
    size = L.qv_run_attention_workspace_size
    assert size(0, 0, 0, 4, 2, 64, 0) == size(5, 3, 0, 4, 2, 64, 100) == 256
    for bad in ((-1, 3, 1, 4, 2, 64, 64), (5, -1, 1, 4, 2, 64, 64), (5, 3, 6, 4, 2, 64, 64), (5, 3, -1, 4, 2, 64, 64),
                (5, 3, 1, 3, 2, 64, 64), (5, 3, 1, 4, 0, 64, 64), (5, 3, 1, 4, 2, 80, 64), (5, 3, 1, 4, 2, 64, -1),
                (5, 3, 1, 4, 2, 64, 1 << 40), (1 << 40, 3, 1, 4, 2, 64, 64), (1 << 20, 1 << 40, 1, 4, 2, 64, 64)):
        assert size(*bad) == 0, bad


def test_table_refusals(L):
    assert tables(L, B=-1) == SHAPE and tables(L, T=-1) == SHAPE and tables(L, F=-1) == SHAPE and tables(L, page=0) == SHAPE
    assert tables(L, pages=-1) == SHAPE and tables(L, ld=3) == SHAPE and tables(L, ld=1 << 41) == SHAPE
    assert tables(L, pages=1 << 27, ld=1 << 27) == UNSUPPORTED and tables(L, T=1 << 31) == UNSUPPORTED
    assert tables(L, B=1 << 31) == UNSUPPORTED and tables(L, F=1 << 31) == UNSUPPORTED and tables(L, page=1 << 31, pages=1) == UNSUPPORTED
    for name in ("runs_", "lens", "free", "count", "table", "starts", "after", "left", "seq", "index", "slots", "status"):
        assert tables(L, **{name: None}) == NULL, name
        assert tables(L, **{name: MIS + 1}) == ALIGN, name
    assert tables(L, slots=P + 4) == ALIGN


@pytest.mark.skipif(not STUB_LIB, reason="only meaningful in the host-only stub build")
def test_stub_counts_valid_calls(L, request):
    """Valid calls pass the checks and reach a (stub) launcher, whose failure is reported."""
    calls = [attend(L), attend(L, T=3, B=3, max_run=1, starts=None), attend(L, window=7, sinks=4, causal=0),
             attend(L, cache_=cache(num_pages=0, k_pages=None)), attend(L, cache_=cache(dtype=2, scale_tokens=32)),
             attend(L, pages=0, ld=0, table=None), attend(L, T=200, max_run=200), tables(L), tables(L, F=0, free=None),
             tables(L, T=0, seq=None, index=None, slots=None), tables(L, pages=0, ld=0, table=None),
             tables(L, B=0, runs_=None, lens=None, after=None, status=None, table=None)]
    assert calls == [HIP] * len(calls)
    request.node.accepted = len(calls)


@pytest.mark.skipif(not STUB_LIB, reason="only the stub build shows the cut into parts")
def test_parts_have_room(L):
    """Whatever window a call has, its parts are no more than the workspace was sized for, and its items cover every tile."""
    L.qv_stub_parts.argtypes, L.qv_stub_parts.restype = [ctypes.c_int64] * 6, ctypes.c_int64
    L.qv_stub_items.argtypes, L.qv_stub_items.restype = [ctypes.c_int64] * 4, ctypes.c_int64
    for T in (33, 129, 1000, 5000, 70000):
        for B in (1, 3, 40):
            for heads_, share in ((1, 1), (2, 5), (16, 1), (8, 4)):
                for capacity in (0, 64, 4000, 100000):
                    room = L.qv_stub_parts(T, B, heads_ * share, heads_, capacity, 64)
                    assert 1 <= room <= 64
                    for seen in (1, 200, 3000, capacity):
                        assert 1 <= L.qv_stub_parts(T, B, heads_ * share, heads_, seen, room) <= room
                # any cut of the rows into runs: a sequence's tiles begin at floor(row * share / 128) + number
                for step in (1, 7, 128, T):
                    starts = [min(T, i * step) for i in range(B)] + [T]
                    first = [s * share // 128 + b for b, s in enumerate(starts)]
                    for b in range(B):
                        assert first[b + 1] - first[b] >= -(-(starts[b + 1] - starts[b]) * share // 128)
                    assert first[B] == L.qv_stub_items(T, B, heads_ * share, heads_)


def test_checks_under_sanitizers(tmp_path):
    from test_sanitizers import SAN, _env, _runtime

    if STUB_LIB:
        return
    _runtime()
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    csrc, stubs = os.path.join(ROOT, "bit_ptq_reconstruction_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    so = str(tmp_path / "libqv_runs_stub.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", *SAN, "-I", stubs, "-I",
                    os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "qv_runs_abi.cpp"),
                    os.path.join(stubs, "runs_stubs.cpp"), "-o", so], check=True, capture_output=True, text=True)
    logs = tmp_path / "logs"
    logs.mkdir()
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", __file__], cwd=ROOT,
                       env=_env(logs, QV_RUNS_ABI_TEST_LIB=so), capture_output=True, text=True, timeout=600)
    reports = "".join(open(os.path.join(logs, f)).read() for f in sorted(os.listdir(logs)))
    assert not reports, reports[-3000:]
    assert r.returncode == 0 and " passed" in r.stdout and "skipped" not in r.stdout, (r.stdout + r.stderr)[-3000:]
