"""Appends at the edges of what the entry point takes."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import dev, gen, make_cache, qv  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_append_with_empty_tables(qv, dev):
    """Tables without a place have no position inside: nothing is stored, and queries are NaN."""
    g = gen(2)
    cache = make_cache(qv, dev, 2, 2, 16, 64, "bf16", 0)
    K, V, Q = (torch.randn((5, 2, 64), generator=g).to(dev) for _ in range(3))
    i = torch.arange(5, dtype=torch.int32, device=dev)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=dev)
    none = torch.empty((0, 32), device=dev)
    out = torch.zeros_like(Q)
    qv.qv_kv_append(cache, table, torch.zeros_like(i), i, K, V, none, none, None, Q, out)
    assert bool(torch.isnan(cache.k_pages).all()) and bool(torch.isnan(cache.v_pages).all())
    assert bool(torch.isnan(out).all())
