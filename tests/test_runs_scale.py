"""A scale that is not finite is refused on the host, in the C ABI and in the binding (CPU only)."""
import pytest

pytest.importorskip("torch")

from bit_ptq_reconstruction_amd import decode, runs  # noqa: E402
from test_runs_abi import L, OK, P, SHAPE, cache, heads  # noqa: E402,F401
from test_runs_binding import attend, built, refused  # noqa: E402,F401

SCALES = [float("nan"), float("inf"), float("-inf"), 1e39, -1e39]


@pytest.mark.parametrize("scale", SCALES)
def test_abi(L, scale):
    call = lambda scale, T: L.qv_run_attention(heads(), 1, T, 4, P, 3, T and 5, cache(), P, 4, 4, P, scale, 0, 0, 1, heads(), P,
                                               1 << 24, None)
    assert call(scale, 12) == SHAPE and call(scale, 0) == SHAPE
    assert call(0.0, 0) == call(-3.4e38, 0) == OK


@pytest.mark.parametrize("scale", SCALES)
def test_binding(scale):
    refused(attend, "scale .* must be finite", scale=scale)
    refused(attend, "GPU tensor", scale=-3e38)
