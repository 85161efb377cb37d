"""StreamBlock's window and first tokens are checked on construction (CPU only)."""
import pytest

pytest.importorskip("torch")

from bit_ptq_reconstruction_amd.stream import StreamBlock  # noqa: E402


@pytest.mark.parametrize("change,match", [(dict(window=-1), "window -1"), (dict(sinks=-2), "sinks -2"), (dict(window=1.5), "window 1.5"),
                                          (dict(sinks=None), "sinks None"), (dict(window=1 << 63), "window 9223372036854775808")])
def test_window(change, match):
    """What the attention would refuse, after the call's tokens have joined the cache, is refused before anything is allocated."""
    with pytest.raises(ValueError, match=match):
        StreamBlock(None, {}, 1, 16, "cpu", **change)
