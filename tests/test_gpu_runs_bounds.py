"""Attention of runs of tokens: what the probabilities' pieces leave of them.

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
