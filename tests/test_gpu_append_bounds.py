"""Appends at the edges of what the entry point takes."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import DT, codes32, dev, gen, make_cache, qv, turn32  # noqa: E402,F401

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


@pytest.mark.parametrize("T,heads,q_heads,dim,axes,xt,kind,rotate", [
    (5600, 16, 16, 64, 2, "bf16", "bf16", True), (9003, 3, 9, 128, 1, "fp32", "int8", True), (14001, 4, 11, 64, 1, "bf16", "int8", True),
    (16500, 2, 5, 128, 2, "fp32", "bf16", True), (16391, 4, 0, 128, 1, "bf16", "bf16", False), (9001, 5, 20, 128, 1, "bf16", "int8", True),
    (22001, 3, 7, 64, 1, "fp32", "int8", True), (11003, 8, 9, 64, 1, "fp32", "bf16", True),
])
def test_long_appends(qv, dev, T, heads, q_heads, dim, axes, xt, kind, rotate):
    """2^20 threads' worth of tokens and more, where a thread takes two heads; even and odd numbers of them."""
    g = gen(T)
    size = 64
    table = torch.randperm(-(-T // size) + 3, generator=g, dtype=torch.int32)[None, :-(-T // size)].contiguous()
    cache = make_cache(qv, dev, table.shape[1] + 3, heads, size, dim, kind, 0, "slot")
    K, V = (torch.randn((T, heads, dim), generator=g).to(DT[xt]) for _ in range(2))
    Q = torch.randn((T, q_heads, dim), generator=g).to(DT[xt]) if q_heads else None
    i = torch.arange(T, dtype=torch.int32)
    places = 300
    position = torch.randint(places, (T, axes), generator=g, dtype=torch.int32)
    angle = torch.arange(places)[:, None] * 100.0 ** (-torch.arange(0, dim // axes, 2) / (dim // axes))
    cos, sin = angle.cos(), angle.sin()
    d = lambda t: None if t is None else t.to(dev)
    out = None if Q is None else torch.full((T + 1, q_heads, dim), float("nan"), dtype=DT[xt], device=dev)
    qv.qv_kv_append(cache, d(table), torch.zeros(T, dtype=torch.int32, device=dev), d(i), d(K), d(V),
                    *((d(cos), d(sin), d(position)) if rotate else (None, None, None)), d(Q), None if Q is None else out[:T])
    turned = lambda x: turn32(x, cos, sin, position, axes) if rotate else x.float()
    pg, slot = table[0, (i // size).long()].long(), (i % size).long()
    for pages, scales, x in ((cache.k_pages, cache.k_scale, turned(K)), (cache.v_pages, cache.v_scale, V.float())):
        got = pages.cpu()[pg, :, slot]
        if kind == "bf16":
            assert torch.equal(got, x.to(torch.bfloat16))
            assert int((~torch.isnan(pages.float())).sum()) == T * heads * dim
        else:
            codes, scale = codes32(x)
            assert torch.equal(got, codes) and torch.equal(scales.cpu()[pg, :, slot], scale)
            assert int((~torch.isnan(scales)).sum()) == T * heads
    if Q is not None:
        assert torch.equal(out[:T].cpu(), turned(Q).to(DT[xt])) and bool(torch.isnan(out[T:].float()).all())


def test_append_of_no_tokens_on_two_axes(qv, dev):
    """An empty run of tokens, whose empty tensors have no address, is a call like any other."""
    cache = make_cache(qv, dev, 2, 2, 16, 64, "bf16", 0)
    e = lambda *s: torch.empty(s, device=dev)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    qv.qv_kv_append(cache, i(1, 2), i(0), i(0), e(0, 2, 64), e(0, 2, 64), e(9, 16), e(9, 16), i(0, 2), e(0, 4, 64), e(0, 4, 64))
    assert bool(torch.isnan(cache.k_pages).all())
