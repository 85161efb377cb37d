"""The attention where a result is far smaller than its terms, and where it is not a number."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import DT, U, attend, attention64, check_attention, codes32, dev, fill, gen, make_cache, qv, shuffled_table  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("kind,dim,share", [("bf16", 64, 2), ("bf16", 128, 4), ("int8", 64, 4), ("int8", 128, 2),
                                            ("bf16", 64, 1), ("int8", 128, 1)])
def test_probabilities_keep_their_bits(qv, dev, xt, kind, dim, share):
    """One token of probability p = exp(t) and value -1 against tokens of probability 1 whose values sum to p.

    A score of up to 4 bits is off by 2 roundings of u each, times ln 2; exp2 by 2 u; products and sums of five tokens by
    a dozen more: 32 u of the sum of p |v|, and twice that for sums that the matrix cores cut."""
    B = 24
    t = -torch.linspace(0.1, 2.7, B).to(torch.bfloat16).double()  # a score: channel 0 of the token's key
    table = torch.arange(B, dtype=torch.int32)[:, None]
    cache = make_cache(qv, dev, B, 1, 16, dim, kind, 0)
    p = torch.exp(t)
    zero = torch.zeros(dim, device=dev)
    value = torch.zeros((B, 5), dtype=torch.float64)
    for b in range(B):
        rest = p[b].item()
        for i in range(5):
            code = -1.0 if i == 0 else 0.0
            scale = 1.0
            if 0 < i < 4:  # a third of p at a time, in as many bits as the cache has
                part = rest / (4 - i)
                if kind == "bf16":
                    code = torch.tensor(rest).to(torch.bfloat16).item()
                else:
                    code, scale = 3.0, torch.tensor(part / 3).float().item()
                rest -= code * scale
            value[b, i] = code * scale
            key = zero.clone()
            if kind == "bf16":
                key[0] = t[b] if i == 0 else 0.0
            else:
                key[0] = -1 if i == 0 else 0
                cache.k_scale[b, 0, i] = -t[b] if i == 0 else 1.0
                cache.v_scale[b, 0, i] = scale
            cache.k_pages[b, 0, i] = key.to(cache.k_pages.dtype)
            cache.v_pages[b, 0, i] = (zero + code).to(cache.v_pages.dtype)
    Q = torch.zeros((B, share, dim))
    Q[:, :, 0] = 1.0
    O = attend(qv, dev, Q.to(DT[xt]).to(dev), cache, table.to(dev), [5] * B, scale=1.0).double().cpu()
    weight = torch.cat((p[:, None], torch.ones((B, 4), dtype=torch.float64)), 1)
    o = ((weight * value).sum(1) / weight.sum(1))[:, None, None]
    terms = ((weight * value.abs()).sum(1) / weight.sum(1))[:, None, None]
    worst = ((O - o).abs() / (64 * U * terms + 2.0 ** -8 * o.abs())).max().item()
    assert worst <= 1.0, f"{worst:.2f} of the bound"


@pytest.mark.parametrize("xt,kind,dim,share", [("bf16", "bf16", 64, 1), ("fp32", "bf16", 128, 3), ("bf16", "int8", 128, 8),
                                               ("fp32", "int8", 64, 1), ("bf16", "bf16", 128, 17)])
@pytest.mark.parametrize("longest", [40, 3000])
def test_what_is_not_a_number_stays_so(qv, dev, xt, kind, dim, share, longest):
    """A query, a key or a value of NaN gives NaN, in its own rows only; what no row attends to has no effect, and a sequence
    without tokens still gives zeros."""
    g = gen(longest + dim)
    lens = [longest, 0, longest - 3, 20, longest, 31]
    table, pages = shuffled_table(lens, 16, g)
    cache = make_cache(qv, dev, pages, 2, 16, dim, kind, 0)  # NaN behind every sequence's end
    fill(cache, table, lens, g)
    Q = torch.randn((6, 2 * share, dim), generator=g).to(DT[xt]).to(dev)
    clean = attend(qv, dev, Q, cache, table.to(dev), lens).clone()
    assert bool(torch.isfinite(clean.float()).all()) and bool((clean[1] == 0).all())

    def spoil(pages_, scales, b, t, head, channel):
        page, slot = int(table[b, t // 16]), t % 16
        if scales is None:
            pages_[page, head, slot, channel] = float("nan")
        else:
            scales[page, head, slot] = float("nan")

    Q[0, share] = float("nan")  # one query of the second head
    Q[1, 0, 3] = float("nan")   # of a sequence without tokens
    spoil(cache.k_pages, cache.k_scale, 2, longest - 10, 0, 5)
    spoil(cache.v_pages, cache.v_scale, 3, 7, 1, 9)
    O = attend(qv, dev, Q, cache, table.to(dev), lens).float().cpu()
    bad = torch.zeros(O.shape, dtype=torch.bool)
    bad[0, share] = True
    bad[2, :share] = True
    bad[3, share:, slice(9, 10) if kind == "bf16" else slice(None)] = True
    assert bool(torch.isnan(O[bad]).all())
    assert torch.equal(O[~bad], clean.float().cpu()[~bad])


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_int8_append_of_what_is_not_finite(qv, dev, xt, dim):
    """A token and head with a NaN or an infinity is stored with a scale of NaN and zero codes, its neighbours as they are; the
    attention that reads it gives NaN."""
    g = gen(dim)
    cache = make_cache(qv, dev, 2, 3, 16, dim, "int8", 0)
    K, V = (torch.randn((20, 3, dim), generator=g) for _ in range(2))
    V[3, 1, dim - 1], V[7, 0, 0], V[7, 2, 17], K[11, 2, 8] = float("nan"), float("inf"), float("-inf"), float("nan")
    K, V = K.to(DT[xt]), V.to(DT[xt])
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=dev)
    i = torch.arange(20, dtype=torch.int32, device=dev)
    qv.qv_kv_append(cache, table, torch.zeros_like(i), i, K.to(dev), V.to(dev))
    for pages, scales, x, bad in ((cache.k_pages, cache.k_scale, K, [(11, 2)]),
                                  (cache.v_pages, cache.v_scale, V, [(3, 1), (7, 0), (7, 2)])):
        codes, scale = codes32(x.float())
        for t, h in bad:
            codes[t, h], scale[t, h] = 0, float("nan")
        order = lambda p: torch.cat((p[1], p[0]), 1)[:, :20].transpose(0, 1).cpu()
        assert torch.equal(order(pages), codes)
        assert torch.equal(torch.isnan(order(scales)), torch.isnan(scale))
        assert torch.equal(torch.nan_to_num(order(scales)), torch.nan_to_num(scale))
    Q = torch.randn((1, 3, dim), generator=g).to(DT[xt]).to(dev)
    n = lambda *lens: torch.isnan(attend(qv, dev, Q, cache, table, list(lens)).float()).all(2).tolist()
    assert n(3) == [[False, False, False]] and n(4) == [[False, True, False]] and n(20) == [[True, True, True]]


@pytest.mark.parametrize("xt,kind,dim,heads,share", [("bf16", "bf16", 128, 8, 4), ("bf16", "bf16", 64, 16, 1), ("fp32", "int8", 128, 5, 8),
                                                     ("bf16", "int8", 128, 8, 4), ("fp32", "bf16", 128, 20, 2)])
def test_join_of_many_heads(qv, dev, xt, kind, dim, heads, share):
    """More than 512 query heads in all, over sequences of many parts, of one and of none."""
    g = gen(dim + heads)
    lens = ([2500, 0, 1, 700, 128, 1900, 129, 33, 16, 1000] * 4)[:512 // (heads * share) + 1]
    table, pages = shuffled_table(lens, 16, g)
    cache = make_cache(qv, dev, pages, heads, 16, dim, kind, 0)
    kv = fill(cache, table, lens, g)
    Q = torch.randn((len(lens), heads * share, dim), generator=g).to(DT[xt])
    O = attend(qv, dev, Q.to(dev), cache, table.to(dev), lens)
    o, mag = attention64(Q, kv, lens, 0, dim ** -0.5)
    check_attention(O, o, mag, xt, f"{len(lens)} sequences")
    assert bool((O[[n == 0 for n in lens]] == 0).all())
