"""StreamBlock at the edges of its capacity, its frames and its positions."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import codes32, dev, gen, qv, turn32  # noqa: E402,F401

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


@pytest.mark.parametrize("int8", [False, True])
def test_frames_of_any_size(qv, dev, weights, int8):
    """Frames up to ``frame_tokens``: what they store, against the linear's own output turned by position; larger ones, and
    frames of a block that was made for none, are refused."""
    from bit_ptq_reconstruction_amd.stream import GROUP

    g = gen(3)
    block = make(qv, dev, weights, capacity=64, int8_cache=int8)
    expect = [[], []]
    for sequence, T in ((1, 30), (0, 7), (1, 1), (1, 13), (0, 0)):
        x, at = rows(T, g, dev), places(T, g, dev)
        block.take_frame(x, sequence, at)
        if T == 0:
            continue
        qkv = torch.empty((T, 3072), dtype=torch.bfloat16, device=dev)
        work = torch.empty(qv.qv_w4a4_linear_grouped_workspace_size(T, 1024, GROUP), dtype=torch.uint8, device=dev)
        qv.qv_w4a4_linear_grouped(torch.nn.functional.layer_norm(x, (1024,)), None, GROUP, block.Wq["qkv"], block.ws["qkv"],
                                  None, qkv, work)
        qkv = qkv.cpu().view(T, 3, 16, 64)
        expect[sequence].append((turn32(qkv[:, 1], block.cos.cpu(), block.sin.cpu(), at.cpu(), 2), qkv[:, 2].float()))
    assert block.lens.tolist() == block.held == [7, 44]
    for s in range(2):
        t = torch.arange(block.held[s])
        page, slot = block.table[s].cpu().long()[t // 16], t % 16
        for i, (pages, scales) in enumerate(((block.cache.k_pages, block.cache.k_scale), (block.cache.v_pages, block.cache.v_scale))):
            x = torch.cat([e[i] for e in expect[s]])
            got = pages.cpu()[page, :, slot]
            if int8:
                codes, scale = codes32(x)
                assert torch.equal(got, codes) and torch.equal(scales.cpu()[page, :, slot], scale)
            else:
                assert torch.equal(got, x.to(torch.bfloat16))
    with pytest.raises(ValueError, match="a frame of 31 tokens, the block was made for frames of up to 30"):
        block.take_frame(rows(31, g, dev), 0, places(31, g, dev))
    with pytest.raises(ValueError, match="sequence 2 of 2"):
        block.take_frame(rows(1, g, dev), 2, places(1, g, dev))
    none = make(qv, dev, weights, frame_tokens=0)
    with pytest.raises(ValueError, match="a frame of 5 tokens, the block was made for frames of up to 0"):
        none.take_frame(rows(5, g, dev), 0, places(5, g, dev))
    assert block.held == [7, 44] and none.held == [0, 0]


def test_eight_heads(qv, dev, weights):
    """The other number of heads that the attention takes."""
    g = gen(6)
    block = make(qv, dev, weights, heads=8)
    block.take_frame(rows(9, g, dev), 0, places(9, g, dev))
    assert bool(torch.isfinite(block.step(rows(2, g, dev)).float()).all()) and block.lens.tolist() == [10, 1]


@pytest.mark.parametrize("int8", [False, True])
def test_position_outside(qv, dev, weights, int8):
    """A position without an angle shows as NaN in its sequence, then and in the steps behind it, whose past lacks the token; the
    other sequence is untouched."""
    g = gen(5)
    frame, at = rows(20, g, dev), places(20, g, dev)
    x = [rows(2, g, dev) for _ in range(3)]
    p = [places(2, g, dev) for _ in range(3)]
    outs = []
    for bad in (False, True):
        block = make(qv, dev, weights, int8_cache=int8)
        for s in range(2):
            block.take_frame(frame, s, at)
        got = []
        for i in range(3):
            block.position.copy_(p[i])
            if bad and i == 1:
                block.position[0, 1] = 40
            got.append(block.step(x[i]).float().cpu())
        outs.append(got)
    clean, spoilt = outs
    assert torch.equal(spoilt[0], clean[0])
    for i in (1, 2):
        assert bool(torch.isnan(spoilt[i][0]).all()) and torch.equal(spoilt[i][1], clean[i][1])
