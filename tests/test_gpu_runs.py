"""Page tables, the FP8 cache and the attention of runs of tokens against plain implementations.

Tolerances, with 2^-24 and 2^-8 the rounding errors of fp32 and bf16:

* Page tables: whole numbers, equal.
* FP8 append: codes and scales are equal to the formula's, evaluated step by step in fp32 (powers of two multiply exactly, so a
  code is rounded once when it is made and once more when its block's scale grows).
* Attention with probabilities that are not rounded: 1e-5 sum p |v| as for single tokens (a score below 17 in bits is rounded
  about four times, exp2 and sums add a few 2^-24), plus 2^-8 |o| for bf16 results.
* Attention with probabilities in bf16: at most 2^-8 of each term more, 2^-8 sum p |v| for an element; those roundings are
  random, so the whole result (2-norm) is held to 2^-8 of the 2-norm of sqrt(sum (p v)^2)."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_decode import BF, DT, dev, gen, qv, shuffled_table, turn32  # noqa: E402,F401

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------ page tables

def tables64(runs, lens, free, count, page, table, T):
    """By hand, a sequence at a time; ``free`` and ``table`` are lists."""
    count = max(0, min(count, len(free)))
    table = [list(row) for row in table]
    starts, after, status, asked, taken = [0], [], [], 0, 0
    seq, index, slots = [-1] * T, [-1] * T, [-1] * T
    for b, (n, l) in enumerate(zip(runs, lens)):
        n, l = max(0, n), max(0, l)
        at = starts[-1]
        starts.append(min(at + n, 2 ** 31 - 1))
        held, need = -(-l // page), max(0, -(-(l + n) // page) - -(-l // page))
        why = 1 if l + n > len(table[b]) * page else 3 if n and at + n > T else 0
        if not why:
            if need and asked + need > count:
                why = 2
            else:
                for j in range(need):
                    table[b][held + j] = free[count - 1 - asked - j]
                taken += need
            asked += need
        status.append(why)
        after.append(l if why else l + n)
        for i in range(0 if why else n):
            e, s = divmod(l + i, page)
            seq[at + i], index[at + i] = b, l + i
            slots[at + i] = -1 if table[b][e] < 0 else table[b][e] * page + s
    return dict(table=table, starts=starts, after=after, left=[count - taken], seq=seq, index=index, slots=slots,
                status=status)


class Tables:
    """The operands of one call, with guards behind every output."""

    def __init__(self, qv, dev, runs, lens, free, count, page, width, T, in_place=False, pad=0):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        B = len(runs)
        self.qv, self.B, self.T, self.page = qv, B, T, page
        self.full = torch.full((B + 1, width + pad), -9, dtype=torch.int32, device=dev)
        self.table = self.full[:B, :width]
        for b, n in enumerate(lens):
            for e in range(min(width, -(-max(0, n) // page))):
                self.table[b, e] = 1000 * b + e
        self.runs, self.lens, self.free, self.count = i32(runs), i32(lens), i32(free), i32([count])
        self.expect = tables64(runs, lens, free, count, page, self.table.tolist(), T)
        guarded = lambda n, dtype=torch.int32: torch.full((n + 7,), -77, dtype=dtype, device=dev)
        self.out = dict(starts=guarded(B + 1), after=guarded(B), left=guarded(1), seq=guarded(T), index=guarded(T),
                        slots=guarded(T, torch.int64), status=guarded(B))
        self.view = {n: t[:len(t) - 7] for n, t in self.out.items()}
        if in_place:
            self.view["after"], self.view["left"] = self.lens, self.count

    def call(self, **kw):
        o = self.view
        self.qv.qv_page_tables(self.runs, self.lens, self.free, self.count, self.page, self.table, o["starts"], o["after"],
                               o["left"], o["seq"], o["index"], o["slots"], o["status"], **kw)

    def check(self):
        torch.cuda.synchronize()
        for name, t in self.view.items():
            assert t.tolist() == self.expect[name], name
        assert self.table.tolist() == self.expect["table"]
        assert bool((self.full[:, self.table.shape[1]:] == -9).all()) and bool((self.full[self.B:] == -9).all())
        assert all(bool((t[-7:] == -77).all()) for t in self.out.values())


TABLES = [  # runs, lens, free pages, count, page, width, T
    ([1], [0], 3, 3, 16, 4, 1),
    ([1, 1, 1, 1], [0, 15, 16, 17], 9, 9, 16, 2, 4),
    ([0, 0], [5, 0], 0, 0, 16, 2, 0),
    ([37, 0, 16, 1, 129], [3, 9, 0, 47, 16], 40, 33, 16, 12, 200),       # rows behind the last run
    ([20, 20, 0, 1, 20], [0, 0, 7, 5, 30], 3, 3, 16, 4, 61),             # too few pages: the second, and all behind it
    ([5, 40, 5], [0, 30, 0], 9, 9, 16, 4, 50),                           # no room in the table
    ([5, 40, 0, 5, 2], [0, 1, 2, 3, 4], 20, 20, 16, 4, 30),              # no rows
    ([-3, 7, 2], [4, -5, 2 ** 31 - 1], 9, 50, 7, 5, 9),                  # negative and far numbers, a count past the list
    ([2 ** 31 - 1, 2 ** 31 - 1, 1], [0, 1, 0], 9, -4, 1, 5, 3),
    ([1, 3], [16, 1], 2, 0, 16, 2, 4),                                   # no free pages, one place left
    ([5000, 1, 700], [100, 63, 0], 200, 180, 64, 90, 5800),              # many rows: several blocks
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("runs,lens,free,count,page,width,T", TABLES)
def test_page_tables(qv, dev, runs, lens, free, count, page, width, T, in_place):
    pool = torch.randperm(free + 50, generator=gen(free))[:free].tolist()
    t = Tables(qv, dev, runs, lens, pool, count, page, width, T, in_place, pad=3)
    t.call()
    t.check()


@pytest.mark.parametrize("B,longest,page", [(1024, 1, 16), (1025, 3, 16), (3000, 40, 64), (2500, 9, 128)])
def test_page_tables_of_many_sequences(qv, dev, B, longest, page):
    """More sequences than a block has threads, and sequences on both sides of a row that two blocks share."""
    g = gen(B)
    runs, lens = (torch.randint(0, n + 1, (B,), generator=g).tolist() for n in (longest, 300))
    pages = sum(-(-(n + m) // page) for n, m in zip(lens, runs))
    t = Tables(qv, dev, runs, lens, torch.randperm(pages, generator=g).tolist(), pages, page, 400 // page + 2, sum(runs) + 5)
    t.call()
    t.check()


def test_page_tables_replayed(qv, dev):
    """A captured step that takes its places in place, replayed: each replay goes on from the lengths and the list of the last."""
    free = torch.randperm(30, generator=gen(1)).tolist()
    t = Tables(qv, dev, [3, 1, 0], [0, 15, 2], free, 30, 16, 4, 4, in_place=True)
    t.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.call()
    for _ in range(6):
        t.expect = tables64([3, 1, 0], t.lens.tolist(), free, int(t.count), 16, t.table.tolist(), 4)
        graph.replay()
        t.check()
    assert t.lens.tolist() == [21, 22, 2]


def test_page_tables_of_nobody(qv, dev):
    t = Tables(qv, dev, [], [], [4, 2], 2, 16, 3, 5)
    t.call()
    t.check()


# --------------------------------------------------------------------------------------------- FP8 cache

def fp8_cache(qv, dev, pages, heads, size, dim, block, seed, order="head"):
    """Content of plausible sizes, scales of 2^-7 to 2^-5."""
    g = gen(seed)
    codes, scales = [], []
    for _ in range(2):
        c = (torch.randn((pages, heads, size, dim), generator=g) * 60).clamp(-448, 448).to(F8)
        if order == "slot":
            t = torch.empty((pages, size, heads, dim), dtype=F8, device=dev).transpose(1, 2)
            t.copy_(c)
            codes.append(t)
        else:
            codes.append(c.to(dev))
        scales.append(torch.exp2(torch.randint(-7, -4, (pages, heads, size // block), generator=g).float()).to(dev))
    return qv.QVKVCache(*codes, *scales)


def scale32(top):
    """The least power of two, 2^-126 or more, by which top is at most 448."""
    s = 2.0 ** -126
    while s * 448 < top:
        s *= 2
    return s


def store32(codes, scale, x, first, block):
    """x [n, D] at place ``first`` of a block ``codes`` [block, D] (any float type's values): the codes as fp32 numbers and the
    scale."""
    known = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    new = scale32(known.max().item())
    codes = codes.clone()
    if first:
        grown = max(scale, new) if scale == scale else new
        if grown != scale:
            codes[:first] = (codes[:first] * torch.tensor(scale / grown)).to(F8).float()
        new = grown
    y = (x / torch.tensor(new)).to(F8).float()
    codes[first:first + len(x)] = torch.where(torch.isfinite(x), y, torch.full_like(y, float("nan")))
    return codes, new


def append32(cache, table, runs, befores, K, V, block, stored=None):
    """(codes as fp32, scales) of keys and values after the append, a block at a time on the CPU."""
    out = []
    size = cache.page_size
    for pages, scales, x in ((cache.k_pages, cache.k_scale, K), (cache.v_pages, cache.v_scale, V)):
        codes, scales = pages.float().cpu(), scales.cpu().clone()
        at = 0
        for b, (n, before) in enumerate(zip(runs, befores)):
            i = 0
            while i < n:
                place = before + i
                page, slot = int(table[b, place // size]), place % size
                m = min(n - i, block - slot % block)
                rows = slice(slot - slot % block, slot - slot % block + block)
                for h in range(codes.shape[1]):
                    c, s = store32(codes[page, h, rows], scales[page, h, slot // block].item(), x[at + i:at + i + m, h],
                                   slot % block, block)
                    codes[page, h, rows], scales[page, h, slot // block] = c, s
                i += m
            at += n
        out.append((codes, scales))
    return out


def same(a, b):
    """Equal numbers, or NaN in the same places."""
    return torch.equal(torch.nan_to_num(a, nan=1e30), torch.nan_to_num(b, nan=1e30))


def check_cache(cache, expect, label=""):
    torch.cuda.synchronize()
    for name, codes, scales, (c, s) in (("keys", cache.k_pages, cache.k_scale, expect[0]),
                                        ("values", cache.v_pages, cache.v_scale, expect[1])):
        assert torch.equal(scales.cpu(), s), f"{label}: scales of the {name}"
        assert same(codes.float().cpu(), c), f"{label}: codes of the {name}"


FP8 = [  # tokens of each sequence, tokens before, heads, q_heads, dim, axes, page, block, x, order
    ([1], [0], 1, 1, 64, 1, 16, 16, "bf16", "head"),
    ([1, 1, 1, 1, 1], [0, 15, 16, 17, 100], 2, 6, 128, 1, 16, 16, "bf16", "head"),
    ([1, 1, 1], [31, 32, 77], 3, 5, 64, 2, 64, 32, "fp32", "slot"),
    ([37, 1, 0, 64], [3, 0, 9, 16], 3, 3, 64, 2, 16, 16, "fp32", "slot"),
    ([100, 33], [0, 31], 4, 16, 128, 2, 48, 48, "bf16", "head"),
    ([19, 200, 1], [1, 0, 63], 1, 5, 64, 1, 64, 64, "fp32", "slot"),
    ([300], [45], 2, 2, 128, 1, 256, 256, "bf16", "head"),
    ([1374], [0], 16, 16, 64, 2, 64, 32, "bf16", "head"),
    ([700, 3], [5, 129], 2, 2, 128, 1, 128, 16, "fp32", "head"),
]


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("new,before,heads,q_heads,dim,axes,page,block,xt,order", FP8)
def test_fp8_append(qv, dev, new, before, heads, q_heads, dim, axes, page, block, xt, order, rotate):
    g = gen(sum(new) * 31 + dim)
    table, pages = shuffled_table([n + m for n, m in zip(before, new)], page, g)
    cache = fp8_cache(qv, dev, pages, heads, page, dim, block, 5, order)
    T = sum(new)
    qkv = torch.randn((T, q_heads + 2 * heads, dim), generator=g)
    qkv *= torch.exp2(torch.randint(-9, 3, (T, 1, 1), generator=g).float())  # scales grow within a block
    qkv = qkv.to(DT[xt])
    seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(new)])
    index = torch.cat([torch.arange(m, m + n, dtype=torch.int32) for n, m in zip(new, before)])
    position = torch.randint(0, 50, (T, axes), generator=g, dtype=torch.int32)
    angle = torch.rand((50, dim // 2 // axes), generator=g) * 6
    cos, sin = (angle.cos(), angle.sin()) if rotate else (None, None)
    q, k, v = qkv.split((q_heads, heads, heads), 1)
    turned = (lambda x: turn32(x, cos, sin, position, axes)) if rotate else (lambda x: x.float())
    expect = append32(cache, table, new, before, turned(k), v.float(), block)
    full = torch.full((T + 2, q_heads, dim), float("nan"), dtype=DT[xt], device=dev)
    qd, kd, vd = qkv.to(dev).split((q_heads, heads, heads), 1)
    on = lambda x: None if x is None else x.to(dev)
    qv.qv_kv_append(cache, table.to(dev), seq.to(dev), index.to(dev), kd, vd, on(cos), on(sin), on(position if rotate else None),
                    qd, full[:T])
    check_cache(cache, expect)
    assert torch.equal(full[:T].cpu(), turned(q).to(DT[xt])) and bool(torch.isnan(full[T:].float()).all())


def test_fp8_append_token_by_token(qv, dev):
    """A block filled one token at a time, with values that grow and shrink, without token_seq."""
    g = gen(3)
    cache = fp8_cache(qv, dev, 4, 2, 32, 64, 32, 7)
    table = torch.tensor([[3], [1]], dtype=torch.int32)
    for i in range(32):
        k, v = (torch.randn((2, 2, 64), generator=g) * 2.0 ** float(torch.randint(-12, 9, (), generator=g)) for _ in range(2))
        expect = append32(cache, table, [1, 1], [i, i], k, v, 32)
        qv.qv_kv_append(cache, table.to(dev), None, torch.full((2,), i, dtype=torch.int32, device=dev), k.to(dev), v.to(dev))
        check_cache(cache, expect, f"token {i}")


def test_fp8_append_special_values(qv, dev):
    """Zeros, the least and largest numbers, what is not finite, and 448 times a power of two on both sides."""
    cases = [torch.zeros(64), torch.full((64,), 2.0 ** -140), torch.full((64,), 3.4e38), torch.full((64,), 448.0 * 2 ** -20),
             torch.full((64,), 448.0 * 2 ** -20 * (1 + 2.0 ** -22)), torch.full((64,), 448.0), torch.linspace(-5, 5, 64)]
    odd = torch.linspace(-1, 1, 64)
    odd[3], odd[7], odd[20] = float("inf"), float("-inf"), float("nan")
    cases += [odd, torch.full((64,), float("nan"))]
    x = torch.stack(cases)[:, None]
    n = len(cases)
    cache = fp8_cache(qv, dev, n, 1, 16, 64, 16, 2)
    table = torch.arange(n, dtype=torch.int32)[:, None].contiguous()
    expect = append32(cache, table, [1] * n, [0] * n, x, -x, 16)
    qv.qv_kv_append(cache, table.to(dev), None, torch.zeros(n, dtype=torch.int32, device=dev), x.to(dev), -x.to(dev))
    check_cache(cache, expect)


def test_fp8_append_rounds_to_nearest(qv, dev):
    """Every code, and the values halfway between neighbouring codes, a little more and a little less."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(F8).float()
    half = (codes[1:] + codes[:-1]) / 2
    near = torch.cat((codes, half, half * (1 + 2.0 ** -20), half * (1 - 2.0 ** -20)))
    x = torch.zeros(8 * 64)
    x[:len(near)] = near
    x = torch.cat((x, -x)).view(16, 1, 64)
    x[:, :, 63] = 448.0  # every token alone has the scale 1
    cache = fp8_cache(qv, dev, 1, 1, 16, 64, 16, 2)
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    index = torch.arange(16, dtype=torch.int32, device=dev)
    qv.qv_kv_append(cache, table, torch.zeros_like(index), index, x.to(dev), x.to(dev))
    torch.cuda.synchronize()
    assert cache.k_scale.item() == cache.v_scale.item() == 1.0
    assert torch.equal(cache.k_pages[0, 0].float().cpu(), x[:, 0].to(F8).float())
    assert torch.equal(cache.v_pages[0, 0].float().cpu(), x[:, 0].to(F8).float())


def test_fp8_append_out_of_place(qv, dev):
    """Tokens without a place, or with positions outside the tables, are not stored and do not count for a scale; queries of
    unknown positions are NaN; a block that follows another sequence's is told from it."""
    g = gen(9)
    cache = fp8_cache(qv, dev, 3, 2, 16, 64, 16, 4)
    table = torch.tensor([[0, 9], [2, -1]], dtype=torch.int32)
    seq = torch.tensor([0, 0, 0, 1, 1, 1, 7, -1, 0, 1], dtype=torch.int32)
    index = torch.tensor([3, 4, 5, 0, 1, 2, 3, 4, 16, 16], dtype=torch.int32)  # the last two: pages 9 and -1
    position = torch.tensor([[0], [5], [1], [2], [-1], [3], [0], [0], [0], [0]], dtype=torch.int32)
    k, v, q = (torch.randn((10, 2, 64), generator=g) for _ in range(3))
    k[1], v[1], v[4] = 1e6, 1e6, 1e6  # not stored
    angle = torch.rand((5, 32), generator=g)
    known = position[:, 0].clamp(0, 4)[:, None]
    turned = turn32(k, angle.cos(), angle.sin(), known, 1)
    out = torch.zeros((10, 2, 64), device=dev)
    expect = []
    for pages, scales, x in ((cache.k_pages, cache.k_scale, turned), (cache.v_pages, cache.v_scale, v)):
        codes, scales = pages.float().cpu(), scales.cpu().clone()
        for h in range(2):
            for page, first, rows in ((0, 3, (0, 2)), (2, 0, (3, 5))):
                held = codes[page, h].clone()
                both = torch.stack([x[t, h] for t in rows])
                codes[page, h], scales[page, h, 0] = store32(codes[page, h], scales[page, h, 0].item(), both, first, 16)
                new = codes[page, h, first:first + 2].clone()
                codes[page, h, first + 1] = held[first + 1]
                codes[page, h, first], codes[page, h, first + 2] = new[0], new[1]
        expect.append((codes, scales))
    qv.qv_kv_append(cache, table.to(dev), seq.to(dev), index.to(dev), k.to(dev), v.to(dev), angle.cos().to(dev),
                    angle.sin().to(dev), position.to(dev), q.to(dev), out)
    check_cache(cache, expect)
    q32 = turn32(q, angle.cos(), angle.sin(), known, 1)
    q32[[1, 4]] = float("nan")
    assert same(out.cpu(), q32)


# ---------------------------------------------------------------------------------------------- attention

def make(qv, dev, pages, heads, size, dim, kind, seed, order="head", block=16):
    """A cache with content and scales everywhere, on pages that no table names too."""
    if kind == "fp8":
        return fp8_cache(qv, dev, pages, heads, size, dim, block, seed, order)
    g = gen(seed)
    shape = (pages, size, heads, dim) if order == "slot" else (pages, heads, size, dim)
    data = []
    for _ in range(2):
        t = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8) if kind == "int8" else \
            torch.randn(shape, generator=g).to(torch.bfloat16)
        data.append(t.to(dev).transpose(1, 2) if order == "slot" else t.to(dev))
    if kind == "int8":
        data += [(0.01 + 0.01 * torch.rand((pages, heads, size), generator=g)).to(dev) for _ in range(2)]
    return qv.QVKVCache(*data)


def held(cache, pages, scales):
    """The cache's content in 64 bits [pages, heads, size, dim]."""
    x = pages.double().cpu() if pages.dtype != F8 else pages.float().cpu().double()
    if scales is None:
        return x
    s = scales.cpu().double()
    return x * s.repeat_interleave(cache.page_size // s.shape[2], 2)[..., None]


def runs64(Q, starts, cache, table, lens, window, sinks, causal, scale, max_run=1 << 30):
    """(o, sum p |v|, sqrt(sum (p v)^2)) [T, Hq, D] in 64 bits; NaN in rows that no sequence has."""
    T, Hq, D = Q.shape
    H = cache.heads
    k_all, v_all = held(cache, cache.k_pages, cache.k_scale), held(cache, cache.v_pages, cache.v_scale)
    out = [torch.full((T, Hq, D), float("nan"), dtype=torch.float64) for _ in range(3)]
    for b, n in enumerate(lens):
        n = max(0, min(n, table.shape[1] * cache.page_size))
        s0, s1 = starts[b], starts[b + 1]
        t = torch.arange(n)
        page = table[b].long()[t // cache.page_size]
        keep = (page >= 0) & (page < cache.pages)
        page, slot = page.clamp(0, cache.pages - 1), t % cache.page_size
        k, v = k_all[page, :, slot], v_all[page, :, slot]  # [n, H, D]
        for i in range(min(s1 - s0, max_run)):
            p = n - (s1 - s0 if s1 - s0 < max_run else max_run) + i
            use = keep & ((t <= p) if causal else (t < n))
            if window:
                use &= (t < sinks) | (t > p - window)
            for o in out:
                o[s0 + i] = 0
            if not bool(use.any()):
                continue
            s = Q[s0 + i].double().view(H, Hq // H, D) @ k[use].permute(1, 2, 0) * scale
            w = torch.softmax(s, -1)
            x = v[use].transpose(0, 1)
            out[0][s0 + i] = (w @ x).view(Hq, D)
            out[1][s0 + i] = (w @ x.abs()).view(Hq, D)
            out[2][s0 + i] = ((w ** 2) @ (x ** 2)).sqrt().view(Hq, D)
    return out


def rounds(max_run, share, xt, kind="bf16"):
    """Whether the probabilities of such a call are rounded to bf16."""
    return xt == "bf16" and max_run > 1 and max_run * share > (32 if kind == "bf16" else 64)


def check(O, expect, xt, rounded, label=""):
    o, mag, root = expect
    got = O.double().cpu()
    there = ~torch.isnan(o)
    if got.numel() == 0:
        return
    assert not bool(torch.isnan(got[there]).any()), f"{label}: NaN"
    err = torch.where(there, got - o, 0).abs()
    o, mag, root = (torch.nan_to_num(x) for x in (o, mag, root))
    tol = (1e-5 + (BF if rounded else 0)) * mag + (BF * 1.01 * o.abs() + 1e-38 if xt == "bf16" else 0)
    worst = (err / tol.clamp(min=1e-300)).max().item()
    assert worst <= 1.0, f"{label}: {worst:.2f} of the bound"
    if rounded:
        whole = err.norm().item() / (root.norm().item() + o.norm().item() + 1e-300)
        assert whole <= BF, f"{label}: {whole:.2e}"


def attend(qv, dev, Q, starts, max_run, cache, table, lens, window=0, sinks=0, causal=True, scale=None, pad=0):
    """O (its own rows are NaN before) with guards behind it, and a workspace with guard bytes."""
    T, Hq, D = Q.shape
    full = torch.full((T + 3, Hq, D + pad), float("nan"), dtype=Q.dtype, device=dev)
    size = qv.qv_run_attention_workspace_size(T, len(lens), max_run, Hq, cache.heads, D, table.shape[1] * cache.page_size)
    work = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device=dev)
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)
    qv.qv_run_attention(Q, i32(starts), max_run, cache, table.to(dev), i32(lens), full[:T, :, :D], work[:size], scale, window,
                        sinks, causal)
    torch.cuda.synchronize()
    assert bool((work[size:] == 0xFF).all())
    assert bool(torch.isnan(full[T:].float()).all()) and bool(torch.isnan(full[:, :, D:].float()).all())
    return full[:T, :, :D]


def sums(runs):
    out = [0]
    for n in runs:
        out.append(out[-1] + n)
    return out


RUNS = [  # tokens of each run, tokens before, heads, share, dim, page, window, sinks, causal, x, cache, order
    ([1], [0], 1, 1, 64, 16, 0, 0, True, "bf16", "bf16", "head"),
    ([1, 1, 1], [99, 16, 0], 2, 1, 64, 16, 20, 3, True, "bf16", "bf16", "head"),
    ([1, 1, 1, 1], [400, 31, 1000, 7], 2, 4, 128, 32, 64, 5, True, "fp32", "bf16", "slot"),
    ([1, 1], [500, 2000], 1, 8, 128, 16, 100, 33, True, "bf16", "fp8", "head"),
    ([3, 0, 5, 1], [40, 20, 0, 15], 2, 2, 64, 16, 0, 0, True, "bf16", "bf16", "head"),
    ([5, 2, 4], [300, 0, 77], 2, 3, 128, 64, 0, 0, False, "fp32", "int8", "head"),
    ([4, 7], [700, 63], 3, 2, 64, 16, 37, 4, True, "bf16", "int8", "slot"),
    ([2, 8, 3], [1200, 5, 16], 2, 4, 128, 32, 9, 70, True, "bf16", "fp8", "slot"),
    ([16, 1], [50, 3000], 4, 1, 64, 16, 5, 1, False, "fp32", "fp8", "head"),
    ([70, 1, 33], [0, 100, 15], 2, 1, 64, 16, 0, 0, True, "bf16", "bf16", "head"),
    ([128, 129, 0, 127], [0, 64, 5, 3], 1, 2, 128, 64, 0, 0, True, "bf16", "bf16", "slot"),
    ([200, 61], [37, 500], 2, 5, 128, 48, 0, 0, True, "bf16", "bf16", "head"),
    ([333], [0], 2, 1, 64, 32, 50, 7, True, "bf16", "bf16", "head"),
    ([150, 7], [900, 0], 1, 4, 128, 16, 128, 16, True, "bf16", "fp8", "head"),
    ([257, 64], [0, 333], 2, 2, 64, 128, 0, 0, False, "bf16", "int8", "head"),
    ([100, 90], [130, 0], 2, 2, 64, 16, 0, 0, True, "fp32", "bf16", "head"),
    ([65, 130], [20, 77], 1, 3, 128, 16, 40, 20, True, "fp32", "int8", "slot"),
    ([40, 300], [60, 0], 2, 1, 128, 64, 33, 2, False, "fp32", "fp8", "head"),
    ([64], [5000], 1, 1, 64, 16, 0, 0, True, "bf16", "bf16", "head"),
    ([33], [9000], 2, 1, 128, 64, 0, 0, True, "bf16", "fp8", "head"),
    ([48, 1], [3000, 4000], 1, 2, 64, 32, 1500, 100, True, "fp32", "bf16", "head"),
]


@pytest.mark.parametrize("runs,before,heads,share,dim,page,window,sinks,causal,xt,kind,order", RUNS)
def test_run_attention(qv, dev, runs, before, heads, share, dim, page, window, sinks, causal, xt, kind, order):
    g = gen(sum(runs) * 7 + sum(before) + dim)
    lens = [n + m for n, m in zip(runs, before)]
    table, pages = shuffled_table(lens, page, g, extra=1)
    cache = make(qv, dev, pages, heads, page, dim, kind, 11, order)
    Q = (2 * torch.randn((sum(runs) + 2, heads * share, dim), generator=g)).to(DT[xt])
    starts = sums(runs)
    O = attend(qv, dev, Q.to(dev), starts, max(runs), cache, table, lens, window, sinks, causal, pad=8)
    check(O, runs64(Q, starts, cache, table, lens, window, sinks, causal, dim ** -0.5), xt, rounds(max(runs), share, xt, kind))
    assert bool(torch.isnan(O[starts[-1]:].float()).all())  # rows that no sequence has
    if max(runs) == 1 and starts[-1] == len(runs):  # single tokens without starts
        again = attend(qv, dev, Q[:len(runs)].to(dev), None, 1, cache, table, lens, window, sinks, causal, pad=8)
        assert torch.equal(again, O[:len(runs)])


@pytest.mark.parametrize("lens,heads,share,dim,page,block,window,xt,order", [
    ([1], 1, 1, 64, 16, 16, 0, "bf16", "head"), ([0, 1, 15, 16, 17, 33, 200], 2, 1, 64, 32, 16, 0, "fp32", "slot"),
    ([47, 0, 200, 129], 3, 5, 128, 48, 48, 0, "bf16", "head"), ([700, 5, 64, 2000], 2, 4, 128, 64, 32, 37, "fp32", "head"),
    ([20011], 1, 8, 128, 256, 128, 0, "bf16", "head"), ([5003, 11], 2, 17, 64, 16, 16, 0, "bf16", "slot")])
def test_fp8_single_tokens(qv, dev, lens, heads, share, dim, page, block, window, xt, order):
    """qv_paged_attention over the FP8 cache."""
    g = gen(sum(lens) + dim)
    table, pages = shuffled_table(lens, page, g, extra=1)
    cache = make(qv, dev, pages, heads, page, dim, "fp8", 3, order, block)
    B = len(lens)
    Q = (2 * torch.randn((B, heads * share, dim), generator=g)).to(DT[xt])
    full = torch.full((B + 3, heads * share, dim), float("nan"), dtype=DT[xt], device=dev)
    size = qv.qv_paged_attention_workspace_size(B, heads * share, heads, dim, table.shape[1] * page)
    work = torch.empty(size, dtype=torch.uint8, device=dev)
    qv.qv_paged_attention(Q.to(dev), cache, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), full[:B], work,
                          window=window)
    expect = runs64(Q, list(range(B + 1)), cache, table, lens, window, 0, True, dim ** -0.5)
    check(full[:B], [torch.nan_to_num(x) for x in expect], xt, False)
    assert bool(torch.isnan(full[B:].float()).all())


def test_run_attention_as_single_tokens(qv, dev):
    """Runs of one without first tokens are what qv_paged_attention computes."""
    g = gen(2)
    lens = [700, 1, 64, 1500]
    table, pages = shuffled_table(lens, 16, g)
    for kind in ("bf16", "int8", "fp8"):
        cache = make(qv, dev, pages, 2, 16, 128, kind, 4)
        Q = torch.randn((4, 8, 128), generator=g).to(torch.bfloat16)
        O = attend(qv, dev, Q.to(dev), None, 1, cache, table, lens, window=200)
        check(O, runs64(Q, list(range(5)), cache, table, lens, 200, 0, True, 128 ** -0.5), "bf16", False, kind)


@pytest.mark.parametrize("xt,kind,dim,run,share", [
    ("bf16", "bf16", 64, 7, 2), ("fp32", "bf16", 128, 4, 1), ("bf16", "fp8", 128, 6, 5), ("fp32", "int8", 64, 5, 3),
    ("bf16", "bf16", 128, 90, 1), ("bf16", "fp8", 64, 150, 2), ("fp32", "bf16", 64, 70, 1), ("bf16", "int8", 128, 80, 3)])
@pytest.mark.parametrize("window", [0, 30])
def test_what_a_row_does_not_see(qv, dev, xt, kind, dim, run, share, window):
    """NaN and infinities in tokens that a row does not see leave it alone; those that see them show it."""
    g = gen(run + dim + window)
    before, page, heads, sinks = 45, 16, 2, 3
    n = before + run
    table, pages = shuffled_table([n], page, g, extra=1)
    cache = make(qv, dev, pages, heads, page, dim, kind, 8)
    Q = torch.randn((run, heads * share, dim), generator=g).to(DT[xt])
    clean = runs64(Q, [0, run], cache, table, [n], window, sinks, True, dim ** -0.5)
    odd = [before + 1, before + run // 2, before - 20, 10, n - 1]  # places
    for i, t in enumerate(odd):
        at = (int(table[0, t // page]), slice(None), t % page)
        if kind == "int8":
            (cache.k_scale if i % 2 else cache.v_scale)[at] = float("nan")
        else:
            what = float("nan") if kind == "fp8" else (float("inf"), float("nan"))[i % 2]
            for pages_ in ((cache.k_pages,) if i % 3 == 2 else (cache.v_pages,) if i % 3 else (cache.k_pages, cache.v_pages)):
                row = pages_[at].float()
                row[:, i::7] = what
                if kind == "fp8":
                    pages_.view(torch.uint8)[at] = row.to(F8).view(torch.uint8)
                else:
                    pages_[at] = row.to(pages_.dtype)
    for p in range(n, -(-n // page) * page):  # behind the end
        cache.v_pages.view(torch.uint8)[int(table[0, p // page]), :, p % page] = 0xFF
    O = attend(qv, dev, Q.to(dev), [0, run], run, cache, table, [n], window, sinks).double().cpu()
    for i in range(run):
        p = before + i
        seen = [t for t in odd if t <= p and (not window or t < sinks or t > p - window)]
        if seen:
            assert not bool(torch.isfinite(O[i]).all(-1).any()), f"row {i} sees {seen}"
        else:
            rounded = rounds(run, share, xt, kind)
            check(O[i:i + 1], [x[i:i + 1] for x in clean], xt, rounded, f"row {i}")


@pytest.mark.parametrize("share,run", [(1, 3), (4, 6), (1, 100), (3, 50)])
def test_rows_without_tokens(qv, dev, share, run):
    """Sequences without tokens, runs longer than their sequence, pages that are gone, and scores of minus infinity."""
    g = gen(share + run)
    lens = [0, run // 2, run + 40, run]
    starts = sums([run] * 4)
    table = torch.arange(4 * 10, dtype=torch.int32).view(4, 10)
    cache = make(qv, dev, 40, 2, 16, 64, "bf16", 1)
    table[2, 0] = 40       # outside the cache
    table[2, 1] = -1
    table[3] = -1          # all gone
    Q = torch.randn((4 * run, 2 * share, 64), generator=g).to(torch.bfloat16)
    for causal in (True, False):
        O = attend(qv, dev, Q.to(dev), starts, run, cache, table, lens, 0, 0, causal)
        check(O, runs64(Q, starts, cache, table, lens, 0, 0, causal, 0.125), "bf16", rounds(run, share, "bf16"))
        assert bool((O[:run] == 0).all()) and bool((O[3 * run:] == 0).all())
        if causal:
            assert bool((O[run:run + run - run // 2] == 0).all())


@pytest.mark.parametrize("runs,starts,max_run", [
    ([2, 3], [0, 2, 5], 2),                    # the second run is cut to its first two rows
    ([3, 3], [0, 3, 100], 3),                  # past the rows
    ([4, 0, 2], [0, 4, -5, 2], 4),             # falling and negative: cut
    ([90, 70], [0, 90, 160], 80),
])
def test_runs_are_cut(qv, dev, runs, starts, max_run):
    """Whatever the starts say, nothing outside the rows is read or written."""
    g = gen(sum(runs))
    T = 6 if max_run < 10 else 160
    lens = [50 + n for n in runs]
    table, pages = shuffled_table(lens, 16, g)
    cache = make(qv, dev, pages, 2, 16, 64, "bf16", 1)
    Q = torch.randn((T, 4, 64), generator=g).to(torch.bfloat16)
    O = attend(qv, dev, Q.to(dev), starts, max_run, cache, table, lens).double().cpu()
    s0 = [min(max(s, 0), T) for s in starts]
    cut = [(a, min(max(a, b), a + max_run)) for a, b in zip(s0[:-1], s0[1:])]
    for (a, b), n, row in zip(cut, lens, table):
        one = runs64(Q, [a, b], cache, row[None], [n], 0, 0, True, 0.125)
        if all(x == y or not (x < b and a < y) for x, y in cut if (x, y) != (a, b)):
            check(O[a:b], [x[a:b] for x in one], "bf16", rounds(max_run, 2, "bf16"))
    inside = torch.zeros(T, dtype=torch.bool)
    for a, b in cut:
        inside[a:b] = True
    assert bool(torch.isnan(O[~inside]).all())


@pytest.mark.parametrize("run", [5, 200])
def test_far_pages(qv, dev, run):
    """Pages past byte offset 2^32 of a cache."""
    page, heads, dim = 64, 16, 128
    pages = 2 ** 32 // (page * heads * dim * 2) + 40
    k = torch.empty((pages, heads, page, dim), dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    g = gen(run)
    n = run + 100
    need = -(-n // page)
    table = torch.arange(pages - need, pages, dtype=torch.int32)[None]
    for x in (k, v):
        x[pages - need:] = torch.randn((need, heads, page, dim), generator=g).to(torch.bfloat16).to(dev)
    small = qv.QVKVCache(k[pages - need:], v[pages - need:])
    cache = qv.QVKVCache(k, v)
    Q = torch.randn((run, heads, dim), generator=g).to(torch.bfloat16).to(dev)
    far = attend(qv, dev, Q, [0, run], run, cache, table, [n])
    near = attend(qv, dev, Q, [0, run], run, small, table - (pages - need), [n])
    assert torch.equal(far, near)
    check(near, runs64(Q.cpu(), [0, run], small, table - (pages - need), [n], 0, 0, True, dim ** -0.5), "bf16",
          rounds(run, 1, "bf16"))


@pytest.mark.parametrize("scale", [-0.4, 0.0, 3.0])
@pytest.mark.parametrize("xt,run", [("bf16", 4), ("bf16", 90), ("fp32", 70)])
def test_scales(qv, dev, scale, xt, run):
    """Scales of any sign, zero (the plain mean of what a row sees), and ones that leave a row one or two tokens."""
    g = gen(run)
    lens = [run + 100, run]
    table, pages = shuffled_table(lens, 16, g)
    cache = make(qv, dev, pages, 2, 16, 64, "bf16", 3)
    Q = torch.randn((2 * run, 2, 64), generator=g).to(DT[xt])
    starts = sums([run] * 2)
    O = attend(qv, dev, Q.to(dev), starts, run, cache, table, lens, 40, 2, scale=scale)
    # scores of up to about 150 bits lose four roundings of 150 * 2^-24 each: ten times the bound of scores below 17
    expect = runs64(Q, starts, cache, table, lens, 40, 2, True, scale)
    expect[1] = expect[1] * 10
    check(O, expect, xt, rounds(run, 1, xt))


class Serve:
    """Tables, append and attention of two calls of runs, as a serving loop makes them, into the same buffers."""

    def __init__(self, qv, dev, kind, run):
        self.qv, g = qv, gen(run)
        self.runs = torch.tensor([run, 0, 3], dtype=torch.int32, device=dev)
        self.T, self.run, H, D = run + 3, run, 2, 64
        self.cache = make(qv, dev, 80, H, 16, D, kind, 5)
        self.table = torch.full((3, 40), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(3, dtype=torch.int32, device=dev)
        self.free = torch.randperm(80, generator=g).to(torch.int32).to(dev)
        self.count = torch.full((1,), 80, dtype=torch.int32, device=dev)
        e = lambda n, t=torch.int32: torch.empty(n, dtype=t, device=dev)
        self.out = [e(4), e(self.T), e(self.T), e(self.T, torch.int64), e(3)]
        self.x = torch.randn((self.T, 4 * H, D), generator=g).to(torch.bfloat16).to(dev)
        self.o = torch.empty((self.T, 2 * H, D), dtype=torch.bfloat16, device=dev)
        self.work = e(qv.qv_run_attention_workspace_size(self.T, 3, run, 2 * H, H, D, 640), torch.uint8)

    def __call__(self, stream=None):
        qv, (starts, seq, index, slots, status) = self.qv, self.out
        qv.qv_page_tables(self.runs, self.lens, self.free, self.count, 16, self.table, starts, self.lens, self.count, seq, index,
                          slots, status, stream=stream)
        qv.qv_kv_append(self.cache, self.table, seq, index, self.x[:, 4:6], self.x[:, 6:], stream=stream)
        qv.qv_run_attention(self.x[:, :4], starts, self.run, self.cache, self.table, self.lens, self.o, self.work, window=150,
                            sinks=4, stream=stream)
        return self.o


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("run", [6, 100])
def test_served_in_a_graph_and_on_a_stream(qv, dev, kind, run):
    """The three calls captured and replayed, with other calls in between that use the workspace, and on a stream of their own,
    against the eager calls."""
    eager, graphed, aside = (Serve(qv, dev, kind, run) for _ in range(3))
    first = eager().clone()
    graphed.work, graphed.out = eager.work, eager.out  # shared by the two
    assert torch.equal(graphed(), first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    aside(stream)
    stream.synchronize()
    assert torch.equal(aside.o, first)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        got = graphed.o.clone()
        assert torch.equal(got, eager()), "replay"
        aside(stream)
        stream.synchronize()
        assert torch.equal(aside.o, got)
        assert eager.lens.tolist() == graphed.lens.tolist() == aside.lens.tolist()
        eager.work.fill_(0xFF)  # nothing in the workspace is kept
        for a, b in ((eager, graphed), (eager, aside)):
            assert torch.equal(a.table, b.table) and int(a.count) == int(b.count)
    assert eager.lens.tolist() == [5 * run, 0, 15] and eager.out[4].tolist() == [0, 0, 0]
    expect = runs64(eager.x[:, :4].cpu(), [0, run, run, run + 3], eager.cache, eager.table.cpu(), eager.lens.tolist(), 150, 4, True, 0.125)
    check(eager.o, expect, "bf16", rounds(run, 2, "bf16", kind))


def test_results_repeat(qv, dev):
    """Split runs give the same bits on every call."""
    g = gen(9)
    lens = [6000, 40]
    table, pages = shuffled_table(lens, 64, g)
    cache = make(qv, dev, pages, 2, 64, 128, "bf16", 1)
    Q = torch.randn((190, 4, 128), generator=g).to(torch.bfloat16).to(dev)
    first = attend(qv, dev, Q, [0, 150, 190], 150, cache, table, lens)
    for _ in range(3):
        assert torch.equal(first, attend(qv, dev, Q, [0, 150, 190], 150, cache, table, lens))


@pytest.mark.parametrize("run", [3, 120])
def test_pages_that_stand_twice(qv, dev, run):
    """A page that several entries name, and sequences that share their first pages."""
    g = gen(run)
    n = 16 * 20 + run
    entries = -(-n // 16)
    table = torch.randint(0, 5, (2, entries), generator=g, dtype=torch.int32)
    table[1, :10] = table[0, :10]
    cache = make(qv, dev, 5, 2, 16, 64, "bf16", 2)
    Q = torch.randn((2 * run, 2, 64), generator=g).to(torch.bfloat16)
    O = attend(qv, dev, Q.to(dev), [0, run, 2 * run], run, cache, table, [n, n])
    check(O, runs64(Q, [0, run, 2 * run], cache, table, [n, n], 0, 0, True, 0.125), "bf16", rounds(run, 1, "bf16"))


def test_many_sequences(qv, dev):
    """More sequences than a wave has lanes: few rows of each, and long runs with empty ones between."""
    g = gen(12)
    for longest in (4, 60):
        runs = [int(n) if i % 3 else 0 for i, n in enumerate(torch.randint(0, longest + 1, (200,), generator=g))]
        runs[17] = longest
        lens = [n + int(m) for n, m in zip(runs, torch.randint(0, 60, (200,), generator=g))]
        table, pages = shuffled_table(lens, 16, g)
        cache = make(qv, dev, pages, 1, 16, 64, "int8", 2)
        Q = torch.randn((sum(runs), 2, 64), generator=g).to(torch.bfloat16)
        starts = sums(runs)
        O = attend(qv, dev, Q.to(dev), starts, longest, cache, table, lens, 30, 1)
        check(O, runs64(Q, starts, cache, table, lens, 30, 1, True, 0.125), "bf16", rounds(longest, 2, "bf16", "int8"))


@pytest.mark.parametrize("share", [1, 3])
def test_runs_of_one_or_none(qv, dev, share):
    """Single tokens of some sequences, with and without tokens before them."""
    g = gen(share)
    runs, before = [1, 0, 1, 0, 1, 1], [0, 40, 700, 0, 15, 16]
    lens = [n + m for n, m in zip(runs, before)]
    table, pages = shuffled_table(lens, 16, g)
    for kind in ("bf16", "fp8"):
        cache = make(qv, dev, pages, 2, 16, 64, kind, 3)
        Q = torch.randn((5, 2 * share, 64), generator=g).to(torch.bfloat16)
        starts = sums(runs)
        for window, sinks in ((0, 0), (30, 2)):
            O = attend(qv, dev, Q.to(dev), starts, 1, cache, table, lens, window, sinks)
            check(O, runs64(Q, starts, cache, table, lens, window, sinks, True, 0.125), "bf16", False)
            assert bool(torch.isnan(O[4:].float()).all())


@pytest.mark.parametrize("run", [7, 150])
@pytest.mark.parametrize("window,sinks,causal", [(1, 0, True), (1, 1, True), (2, 0, False), (64, 64, True), (1 << 40, 3, True), (5, 1 << 40, True)])
def test_narrow_and_wide_windows(qv, dev, run, window, sinks, causal):
    g = gen(run)
    lens = [run + 77, run]
    table, pages = shuffled_table(lens, 16, g)
    cache = make(qv, dev, pages, 2, 16, 64, "bf16", 3)
    Q = torch.randn((2 * run, 2, 64), generator=g).to(torch.bfloat16)
    starts = sums([run] * 2)
    O = attend(qv, dev, Q.to(dev), starts, run, cache, table, lens, window, sinks, causal)
    check(O, runs64(Q, starts, cache, table, lens, window, sinks, causal, 0.125), "bf16", rounds(run, 1, "bf16"))
    if window == 1 and sinks == 0:  # a token sees itself alone
        t = torch.arange(lens[0] - run, lens[0])
        v = cache.v_pages.cpu()[table[0].long()[t // 16], :, t % 16]
        assert torch.equal(O[:run].cpu(), v)


def test_queries_that_are_not_numbers(qv, dev):
    """A query of NaN or infinity gives NaN in its row and nowhere else."""
    g = gen(4)
    for run, kind in ((9, "bf16"), (140, "bf16"), (140, "int8")):
        lens = [run + 50]
        table, pages = shuffled_table(lens, 16, g)
        cache = make(qv, dev, pages, 2, 16, 64, kind, 3)
        Q = torch.randn((run, 4, 64), generator=g).to(torch.bfloat16)
        clean = runs64(Q, [0, run], cache, table, lens, 0, 0, True, 0.125)
        Q[3, 1, 5], Q[run - 2, 2] = float("nan"), float("inf")
        O = attend(qv, dev, Q.to(dev), [0, run], run, cache, table, lens).cpu()
        for row, head in ((3, 1), (run - 2, 2)):
            assert bool(torch.isnan(O[row, head]).all())
            for x in clean:
                x[row, head] = float("nan")
            O[row, head] = 0
        check(O, clean, "bf16", rounds(run, 2, "bf16", kind))
