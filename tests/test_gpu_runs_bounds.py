"""Runs of tokens: what the probabilities' pieces leave of them, what tokens that no row sees cost, runs longer than said, and which
sequences ask for pages.

The probabilities of a bf16 query are two bf16 pieces, each to the nearest: one in [1, 2) leaves at most 2^-8 to the second,
whose last place is then 2^-16, so that 2^-17 of it is lost at most.  With the rest of test_gpu_runs' bound an element is held to
(1e-5 + 2^-17) sum p |v|, plus 2^-8 |o| for the result's own rounding."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import BF, dev, gen, qv, shuffled_table  # noqa: E402,F401
from test_gpu_runs import attend, make, runs64, sums  # noqa: E402

pytestmark = pytest.mark.gpu

LOST = 2.0 ** -17


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("runs,before,heads,share,dim,window,sinks,causal", [
    ([129], [0], 2, 1, 64, 0, 0, True),
    ([150, 1, 70], [900, 0, 33], 1, 4, 128, 128, 16, True),
    ([257, 64], [0, 333], 2, 2, 64, 0, 0, False),
    ([33, 40], [5000, 16], 1, 3, 128, 0, 0, True),  # in parts
])
def test_probabilities_of_bf16_queries(qv, dev, kind, runs, before, heads, share, dim, window, sinks, causal):
    """Long runs lose no more of their probabilities than short ones, so that a query's precision does not depend on its run."""
    g = gen(sum(runs) + dim)
    lens = [n + m for n, m in zip(runs, before)]
    table, pages = shuffled_table(lens, 16, g)
    cache = make(qv, dev, pages, heads, 16, dim, kind, 6)
    Q = (2 * torch.randn((sum(runs), heads * share, dim), generator=g)).to(torch.bfloat16)
    starts = sums(runs)
    O = attend(qv, dev, Q.to(dev), starts, max(runs), cache, table, lens, window, sinks, causal).double().cpu()
    o, mag, _ = runs64(Q, starts, cache, table, lens, window, sinks, causal, dim ** -0.5)
    worst = ((O - o).abs() / ((1e-5 + LOST) * mag + 1.01 * BF * o.abs() + 1e-38)).max().item()
    assert worst <= 1.0, f"{worst:.2f} of the bound"


def fastest(call, times=30):
    """ms of a call among others."""
    best = float("inf")
    for _ in range(times):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(4):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 4)
    return best


@pytest.mark.parametrize("seqs,before,run,window,causal", [(1, 0, 5502, 0, False), (64, 1003, 128, 900, True)])
@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_scales_that_no_row_needs(qv, dev, kind, seqs, before, run, window, causal):
    """Scales of NaN behind a sequence's end, as a new cache has them, and before its window change neither the result nor the
    time."""
    heads, dim, page, n = 16, 64, 32, before + run
    each = -(-n // page)
    cache = make(qv, dev, seqs * each, heads, page, dim, kind, 6)
    table = torch.arange(seqs * each, dtype=torch.int32, device=dev).view(seqs, each)
    lens = torch.full((seqs,), n, dtype=torch.int32, device=dev)
    starts = torch.arange(seqs + 1, dtype=torch.int32, device=dev) * run
    Q = torch.randn((seqs * run, heads, dim), generator=gen(1)).to(torch.bfloat16).to(dev)
    work = torch.empty(qv.qv_run_attention_workspace_size(seqs * run, seqs, run, heads, heads, dim, each * page),
                       dtype=torch.uint8, device=dev)

    def timed():
        O = torch.empty_like(Q)
        call = lambda: qv.qv_run_attention(Q, starts, run, cache, table, lens, O, work, window=window, causal=causal)
        call()
        return O, fastest(call)

    clean, clean_ms = timed()
    step = 1 if kind == "int8" else 16  # tokens of a scale
    for scales in (cache.k_scale, cache.v_scale):
        per = scales.view(seqs, each, heads, page // step).transpose(2, 3).reshape(seqs, -1, heads)  # a copy, by place
        per[:, -(-n // step):] = float("nan")
        if window:  # the first row sees places n - run - window + 1 onwards
            per[:, :(n - run - window + 1) // step] = float("nan")
        scales.copy_(per.view(seqs, each, page // step, heads).transpose(2, 3).reshape(scales.shape))
    got, ms = timed()
    assert torch.equal(got, clean) and bool(torch.isfinite(got.float()).all())
    print(f"{kind} {seqs} x {run}: {clean_ms * 1e3:.1f} us, with scales of NaN {ms * 1e3:.1f}")
    assert ms <= 1.35 * clean_ms, f"{ms * 1e3:.1f} us, {clean_ms * 1e3:.1f} with finite scales"


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("run,max_run,window,causal", [(7, 4, 0, True), (20, 9, 11, True), (150, 130, 0, True), (150, 90, 40, False)])
def test_run_longer_than_said(qv, dev, kind, run, max_run, window, causal):
    """A run of more than max_run rows is its first max_run, as if there were no others: their places are those of a run of that many.
    The rows behind them stay."""
    g = gen(run)
    lens, starts = [run + 60, run], [0, run, 2 * run]
    table, pages = shuffled_table(lens, 16, g)
    cache = make(qv, dev, pages, 2, 16, 64, kind, 7)
    Q = torch.randn((2 * run, 4, 64), generator=g).to(torch.bfloat16)
    O = attend(qv, dev, Q.to(dev), starts, max_run, cache, table, lens, window, 3 if window else 0, causal)
    for b in range(2):
        part = Q[b * run:b * run + max_run].to(dev).contiguous()
        one = attend(qv, dev, part, [0, max_run], max_run, cache, table[b:b + 1], lens[b:b + 1], window, 3 if window else 0, causal)
        # the two calls may cut the tokens differently: each is held to its bound
        got = O[b * run:b * run + max_run].double().cpu()
        o, mag, _ = runs64(Q[b * run:b * run + max_run], [0, max_run], cache, table[b:b + 1], lens[b:b + 1], window,
                           3 if window else 0, causal, 0.125)
        for x in (got, one.double().cpu()):
            assert ((x - o).abs() / ((1e-5 + LOST) * mag + 1.01 * BF * o.abs() + 1e-38)).max().item() <= 1.0
        assert bool(torch.isnan(O[b * run + max_run:(b + 1) * run].float()).all())


@pytest.mark.parametrize("T,last", [(200, 3), (3000, 2)])  # the last run: its rows pass T, or there are no pages
def test_who_asks_for_pages(qv, dev, T, last):
    """A sequence without room asks for no pages, so that the next one gets some; one that lacks pages has asked for them."""
    runs = [20, 60, 10, 30, 40, 16, 3, 50, 0]
    lens = [0, 5, 20, 16, 0, 16, 33, 0, 64]  # in tables of 4 pages of 16
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    empty = lambda n, dtype=torch.int32: torch.full((n,), -7, dtype=dtype, device=dev)
    B = len(runs)
    table = torch.full((B, 4), 99, dtype=torch.int32, device=dev)
    starts, after, left, seq, index, slots, status = (empty(B + 1), empty(B), empty(1), empty(T), empty(T),
                                                      empty(T, torch.int64), empty(B))
    qv.qv_page_tables(i32(runs), i32(lens), i32([5, 9, 3, 8, 1, 7]), i32([5]), 16, table, starts, after, left, seq, index,
                      slots, status)
    assert status.tolist() == [0, 1, 0, 0, 2, 2, 0, last, 0] and left.tolist() == [1]
    assert after.tolist() == [20, 5, 30, 46, 0, 16, 36, 0, 64]
    expect = [[99] * 4 for _ in runs]
    expect[0][:2], expect[3][1:3] = [1, 8], [3, 9]  # from the end of the five that count
    assert table.tolist() == expect
