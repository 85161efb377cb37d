"""What StreamBlock refuses leaves it as it was: lengths, pages, tables and cache, on the GPU and in the host's copies."""
import zlib

import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import dev, gen, qv  # noqa: E402,F401
from test_gpu_stream import make, places, rows, weights  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def state(block):
    torch.cuda.synchronize()
    pool = (block.count.tolist(), block.left) if block.pooled else ()
    return (block.lens.tolist(), list(block.held), block.table.tolist(), pool,
            [zlib.crc32(x.view(torch.uint8).cpu().numpy().tobytes()) for x in (block.cache.k_pages, block.cache.v_pages)])


def wrong_positions(n, g, dev):
    at = places(n, g, dev)
    return [at.long(), at[:-1], at[:, :1], at[:, 0], torch.cat((at, at), 1)[:, ::2], at.cpu(), at.float(), None, at.tolist()]


@pytest.mark.parametrize("pages", [None, 8])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_positions_of_another_kind(qv, dev, weights, pages, cache):
    """Positions of another type, shape, layout or device than int32 [T, axes] are refused before a sequence grows or a page is
    taken; the call with the right ones then gives what it gives in a block that never refused any."""
    g = gen(3)
    kw = dict(sequences=2, capacity=64, frame_tokens=40, pages=pages, fp8_cache=cache == "fp8")
    block, other = make(qv, dev, weights, **kw), make(qv, dev, weights, **kw)
    x, at = rows(40, g, dev), places(40, g, dev)
    frame, where = rows(7, g, dev), places(7, g, dev)
    one = rows(2, g, dev)
    for call, n in ((lambda b, p: b.take_runs(x, [25, 15], p), 40), (lambda b, p: b.take_frame(frame, 1, p), 7)):
        before = state(block)
        for wrong in wrong_positions(n, g, dev):
            with pytest.raises(ValueError, match="position"):
                call(block, wrong)
            assert state(block) == before
        out, expect = (call(b, at if n == 40 else where) for b in (block, other))
        assert out is expect is None or torch.equal(out, expect)
    for b in (block, other):
        b.position = places(2, gen(4), dev)
    right, before = block.position, state(block)
    for wrong in wrong_positions(2, g, dev):
        block.position = wrong
        with pytest.raises(ValueError, match="position"):
            block.step(one)
        assert state(block) == before
    block.position = right
    assert torch.equal(block.step(one), other.step(one)) and state(block) == state(other)


@pytest.mark.parametrize("pages", [None, 8])
def test_places_as_positions(qv, dev, weights, pages):
    """With one axis, no positions are the places in the sequence."""
    g = gen(5)
    kw = dict(sequences=2, capacity=64, frame_tokens=40, pages=pages, axes=1, positions=64)
    block, other = make(qv, dev, weights, **kw), make(qv, dev, weights, **kw)
    x = rows(40, g, dev)
    at = torch.tensor([*range(25), *range(15)], dtype=torch.int32, device=dev)[:, None]
    assert torch.equal(block.take_runs(x, [25, 15], None), other.take_runs(x, [25, 15], at))
    frame, at = rows(7, g, dev), torch.arange(25, 32, dtype=torch.int32, device=dev)[:, None]
    block.take_frame(frame, 0, None)
    other.take_frame(frame, 0, at)
    assert state(block) == state(other)


class Short:
    """The package, with an attention whose workspace no GPU holds."""

    def __init__(self, qv):
        self.qv = qv

    def __getattr__(self, name):
        return getattr(self.qv, name)

    def qv_run_attention_workspace_size(self, *sizes):
        return 1 << 50


@pytest.mark.parametrize("pages", [None, 8])
def test_no_memory(qv, dev, weights, pages):
    """A workspace that does not fit, or an argument that has no truth value, stops a call before its tokens have places."""
    g = gen(6)
    block = make(qv, dev, weights, capacity=64, frame_tokens=40, pages=pages)
    x, at = rows(40, g, dev), places(40, g, dev)
    before = state(block)
    block.qv = Short(qv)
    with pytest.raises(RuntimeError):
        block.take_runs(x, [25, 15], at)
    assert state(block) == before
    block.qv = qv
    with pytest.raises(RuntimeError):
        block.take_runs(x, [25, 15], at, causal=torch.zeros(2))
    assert state(block) == before
    assert bool(torch.isfinite(block.take_runs(x, [25, 15], at).float()).all()) and block.held == [25, 15]
