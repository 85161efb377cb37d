"""StreamBlock at the edges of its capacity, its frames and its positions."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import dev, gen, qv, turn32  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def weights(dev):
    from bit_ptq_reconstruction_amd import configs, synth

    return {lin.name: synth.weights_torch(lin.N, lin.K, lin.w_seed, dev) for lin in configs.block_linears()}


def make(qv, dev, weights, **kw):
    from bit_ptq_reconstruction_amd.stream import StreamBlock

    return StreamBlock(qv, weights, **{**dict(sequences=2, capacity=32, device=dev, axes=2, positions=40, base=100.0, page_size=16,
                                              frame_tokens=30), **kw})


def rows(n, g, dev):
    return torch.randn((n, 1024), generator=g).to(torch.bfloat16).to(dev)


def places(n, g, dev):
    return torch.randint(0, 40, (n, 2), generator=g, dtype=torch.int32).to(dev)


def test_no_room(qv, dev, weights):
    """A token or frame that no page has room for is refused before anything is launched; replays count as well."""
    g = gen(1)
    block = make(qv, dev, weights)
    block.take_frame(rows(30, g, dev), 1, places(30, g, dev))
    with pytest.raises(ValueError, match="sequence 1 holds 30 tokens .* 32"):
        block.take_frame(rows(3, g, dev), 1, places(3, g, dev))
    x = rows(2, g, dev)
    block.step(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x)
    assert block.held == [1, 31]
    block.reserve()
    graph.replay()
    assert block.lens.tolist() == block.held == [2, 32]
    before = block.cache.k_pages.clone()
    for call in (block.reserve, lambda: block.step(x)):
        with pytest.raises(ValueError, match="sequence 1 holds 32 tokens .* 32"):
            call()
    assert block.lens.tolist() == block.held == [2, 32]
    assert torch.equal(before.view(torch.int16), block.cache.k_pages.view(torch.int16))
