"""StreamBlock's runs of tokens, shared pages, window and first tokens: tables, append and attention together."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import BF, dev, gen, qv, turn32  # noqa: E402,F401
from test_gpu_runs import held, runs64, sums  # noqa: E402
from test_gpu_stream import make, places, rows, weights  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def attended(block, b, runs, before, causal, window, sinks):
    """The attention of a call from the block's own queries and cache, in 64 bits, against what the block has formed."""
    T = sum(runs)
    Q = b["q"][:T].cpu()
    lens = [n + m for n, m in zip(runs, before)]
    o, mag, root = runs64(Q, sums(runs), block.cache, block.table.cpu(), lens, window, sinks, causal, block.dim ** -0.5)
    err = (b["o"][:T].double().cpu() - o).abs()
    # probabilities and results in bf16, 2^-8 each; the rest of test_gpu_runs' bound
    worst = (err / ((1e-5 + BF) * mag + 1.01 * BF * o.abs() + 1e-38)).max().item()
    assert worst <= 1.0, f"{worst:.2f} of the bound"


@pytest.mark.parametrize("cache", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("window,sinks,causal", [(0, 0, True), (0, 0, False), (20, 3, True)])
def test_runs_of_many_sequences(qv, dev, weights, cache, window, sinks, causal):
    """Prompts, chunks and single tokens of three sequences over shared pages: keys, values and attention of every call, and the
    same outputs where each sequence has pages of its own."""
    calls = [([30, 0, 47], causal), ([1, 64, 1], True), ([17, 5, 0], causal)]
    kw = dict(sequences=3, capacity=128, frame_tokens=90, int8_cache=cache == "int8", fp8_cache=cache == "fp8", window=window,
              sinks=sinks)
    shared, own = make(qv, dev, weights, pages=16, **kw), make(qv, dev, weights, **kw)
    g = gen(7)
    before = [0, 0, 0]
    for runs, how in calls:
        T = sum(runs)
        x, at = rows(T, g, dev), places(T, g, dev)
        out = shared.take_runs(x, runs, at, how)
        assert torch.equal(out, own.take_runs(x, runs, at, how)) and bool(torch.isfinite(out.float()).all())
        qkv = shared.frame["qkv"][:T].cpu().view(T, 3, 16, 64)
        turned = turn32(qkv[:, 0], shared.cos.cpu(), shared.sin.cpu(), at.cpu(), 2).to(torch.bfloat16)
        assert torch.equal(shared.frame["q"][:T].cpu(), turned)
        attended(shared, shared.frame, runs, before, how, window, sinks)
        if cache == "bf16":
            k = turn32(qkv[:, 1], shared.cos.cpu(), shared.sin.cpu(), at.cpu(), 2).to(torch.bfloat16)
            row = 0
            for s, n in enumerate(runs):
                t = torch.arange(before[s], before[s] + n)
                page, slot = shared.table[s].cpu().long()[t // 16], t % 16
                assert torch.equal(shared.cache.k_pages.cpu()[page, :, slot], k[row:row + n])
                assert torch.equal(shared.cache.v_pages.cpu()[page, :, slot], qkv[row:row + n, 2])
                row += n
        before = [n + m for n, m in zip(runs, before)]
        assert shared.lens.tolist() == own.lens.tolist() == before == shared.held
        assert int(shared.count) == shared.left == 16 - sum(-(-n // 16) for n in before)
    x = rows(3, g, dev)
    for block in (shared, own):
        block.position.zero_()
    out = shared.step(x)
    assert torch.equal(out, own.step(x))
    attended(shared, shared.one, [1, 1, 1], before, True, window, sinks)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_replayed_steps_over_shared_pages(qv, dev, weights, cache):
    """A captured step takes pages as its sequences grow: replays, with the host's own work between them, give what eager steps
    give."""
    kw = dict(sequences=2, capacity=64, frame_tokens=40, pages=7, fp8_cache=cache == "fp8", window=24, sinks=2)
    eager, graphed = make(qv, dev, weights, **kw), make(qv, dev, weights, **kw)
    g = gen(4)
    x0, at = rows(40, g, dev), places(40, g, dev)
    xs = [rows(2, g, dev) for _ in range(18)]
    for block in (eager, graphed):
        block.take_runs(x0, [30, 10], at)
        block.step(xs[0])
    x = xs[1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = graphed.step(x)
    for i in range(1, 18):
        x.copy_(xs[i])
        graphed.reserve()
        graph.replay()
        assert torch.equal(out, eager.step(xs[i])), i
        assert graphed.lens.tolist() == graphed.held == eager.held and int(graphed.count) == graphed.left == eager.left
    assert eager.held == [48, 28] and eager.left == 7 - 3 - 2


def test_pages_come_back(qv, dev, weights):
    """What passes the pool, or a sequence's room, is refused before anything is launched; a sequence that ends gives its pages
    back."""
    block = make(qv, dev, weights, sequences=3, capacity=64, frame_tokens=64, pages=4)
    g = gen(2)
    feed = lambda runs: block.take_runs(rows(sum(runs), g, dev), runs, places(sum(runs), g, dev))
    feed([33, 0, 5])  # four pages
    state = lambda: (block.lens.tolist(), block.held, int(block.count), block.left, block.table.tolist())
    full = state()
    for runs in ([0, 1, 0], [16, 0, 0], [0, 0, 12]):
        with pytest.raises(ValueError, match="1 pages needed, 0 of 4 are free"):
            feed(runs)
    with pytest.raises(ValueError, match="sequence 0 holds 33 tokens .* 32 more in 64"):
        feed([32, 0, 0])
    with pytest.raises(ValueError, match="pages needed"):
        block.step(rows(3, g, dev))
    with pytest.raises(ValueError, match="pages needed"):
        block.take_frame(rows(3, g, dev), 1, places(3, g, dev))
    assert state() == full
    block.end(0)
    assert block.held == [0, 0, 5] and int(block.count) == block.left == 3
    feed([0, 33, 11])
    block.take_frame(rows(15, g, dev), 1, places(15, g, dev))
    taken = block.table[1].tolist()[:3] + block.table[2].tolist()[:1]
    assert sorted(taken) == [0, 1, 2, 3] and block.lens.tolist() == [0, 48, 16]
    for runs in ([1, 2], [1, 2, -1], [1, 1, 1]):
        with pytest.raises(ValueError, match="runs"):
            block.take_runs(rows(4, g, dev), runs, places(4, g, dev))
    with pytest.raises(ValueError, match="65 tokens, the block was made for"):
        block.take_runs(rows(65, g, dev), [65, 0, 0], places(65, g, dev))
    with pytest.raises(ValueError, match="int8 or FP8"):
        make(qv, dev, weights, int8_cache=True, fp8_cache=True)


@pytest.mark.parametrize("flags", [["--attend"], ["--fp8", "--attend", "--window", "1500", "--sinks", "5"], ["--fp8"]])
def test_example(dev, flags):
    import sys

    from test_decode_abi import ROOT

    sys.path.insert(0, ROOT + "/examples")
    import stream_block

    block, out = stream_block.main(["--frames", "2", "--sequences", "2", "--tokens", "6", *flags])
    # one eager step and six replays behind two frames
    assert block.lens.tolist() == [2 * 1374 + 7] * 2 == block.held and bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("cache", ["bf16", "int8", "fp8"])
def test_position_outside_in_a_run(qv, dev, weights, cache):
    """A token at a place without an angle: its output and those behind it in its sequence are NaN, those before it and the other
    sequence's are what they are without it."""
    g = gen(9)
    x, at = rows(50, g, dev), places(50, g, dev)
    outs = []
    for bad in (False, True):
        block = make(qv, dev, weights, sequences=2, capacity=48, frame_tokens=50, int8_cache=cache == "int8", fp8_cache=cache == "fp8")
        if bad:
            at[20, 0] = 40
        outs.append(block.take_runs(x, [35, 15], at).float())
    clean, spoilt = outs
    assert bool(torch.isnan(spoilt[20:35]).all()) and bool(torch.isfinite(clean).all())
    if cache != "fp8":  # where the other tokens of the page share its scale
        assert torch.equal(spoilt[:20], clean[:20])
    assert torch.equal(spoilt[35:], clean[35:]) and bool(torch.isfinite(spoilt[:20]).all())


@pytest.mark.parametrize("pages", [None, 6])
@pytest.mark.parametrize("cache", ["bf16", "int8", "fp8"])
def test_position_outside_on_pages_used_before(qv, dev, weights, cache, pages):
    """A token at a place without an angle is not stored: it and those behind it in its sequence are NaN, whatever sequence had the
    pages before; those before it and the other sequence are not."""
    block = make(qv, dev, weights, sequences=2, capacity=48, frame_tokens=60, int8_cache=cache == "int8", fp8_cache=cache == "fp8",
                 pages=pages)
    g = gen(8)
    block.take_runs(rows(60, g, dev), [40, 20], places(60, g, dev))
    for s in range(2):
        block.end(s)
    at = places(50, g, dev)
    at[20] = torch.tensor([40, 3])
    out = block.take_runs(rows(50, g, dev), [35, 15], at).float()
    assert bool(torch.isnan(out[20:35]).all()) and bool(torch.isfinite(out[:20]).all()) and bool(torch.isfinite(out[35:]).all())
    block.position.zero_()
    out = block.step(rows(2, g, dev)).float()
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1]).all())
    assert block.lens.tolist() == block.held == [36, 16]
