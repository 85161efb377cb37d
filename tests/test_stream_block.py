"""StreamBlock's checks on construction (CPU only)."""
import pytest

pytest.importorskip("torch")

from bit_ptq_reconstruction_amd.stream import StreamBlock  # noqa: E402


@pytest.mark.parametrize("heads", [0, 1, 4, 12, 32])
def test_heads(heads):
    """Heads of other than 64 or 128 channels are refused before anything is allocated."""
    with pytest.raises(ValueError, match=f"{heads} heads"):
        StreamBlock(None, {}, 1, 16, "cpu", heads=heads)
