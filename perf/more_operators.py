"""Cases of the serving operators for runs of tokens: page tables and slot maps built from the tokens that join each
sequence, a cache in 8-bit floating point with a scale for each block of tokens and head (append and attention), and the
attention of runs of tokens with a sliding window and first tokens that stay visible.  With ``own`` the framework's entry
points run, without it their plain form in torch."""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2, "int8": 1, "fp8": 1}
FRAME = 1374  # tokens of one frame
TOP = 448.0   # largest value of the 8-bit format


# ------------------------------------------------------------------------------------------- cases

def tables_case(name, seqs, past, run, page):
    return dict(name=name, op="tables", seqs=seqs, past=past, run=run, page=page)


def append_case(name, seqs, tokens, past, heads, q_heads, dim, axes, page, block, x):
    return dict(name=name, op="append", seqs=seqs, tokens=tokens, past=past, heads=heads, q_heads=q_heads, dim=dim,
                axes=axes, page=page, block=block, x=x, cache="fp8")


def single_case(name, seqs, past, heads, q_heads, dim, page, block, window, x):
    return dict(name=name, op="single", seqs=seqs, past=past, run=1, heads=heads, q_heads=q_heads, dim=dim, page=page,
                block=block, window=window, sinks=0, causal=True, x=x, cache="fp8")


def runs_case(name, seqs, past, run, heads, q_heads, dim, page, block, window, sinks, causal, x, cache):
    return dict(name=name, op="runs", seqs=seqs, past=past, run=run, heads=heads, q_heads=q_heads, dim=dim, page=page,
                block=block, window=window, sinks=sinks, causal=causal, x=x, cache=cache)


def listed():
    return [
        # a serving step: one token joins each of 24 sequences, some of which need a page
        tables_case("tables 24 x 1", 24, 700, 1, 16),
        # prompts of up to a frame for 300 sequences at once, some of them without one
        tables_case("tables prompts", 300, 900, FRAME, 64),
        # one token of each of 24 sequences joins an open block, queries rotated on the way
        append_case("append 24 x 1", 24, 1, 60, 8, 32, 128, 1, 16, 16, "bf16"),
        # eight frames enter an empty cache, patches rotated by row and by column
        append_case("append 8 frames", 8, FRAME, 0, 16, 16, 64, 2, 64, 32, "bf16"),
        # one new token looks back on eight frames, a head of its own for every query
        single_case("attend 8 frames", 1, 8 * FRAME, 16, 16, 64, 64, 32, 0, "bf16"),
        # the largest served batch of long contexts, four queries to a head
        single_case("attend large batch", 48, 16384, 8, 32, 128, 64, 64, 0, "bf16"),
        # a stream that keeps its first tokens and a window: one token of each of 32 sequences
        runs_case("sinks 32 x 1", 32, 32768, 1, 8, 32, 128, 16, 16, 4096, 4, True, "bf16", "bf16"),
        # a few guessed tokens of 16 sequences are checked at once over the int8 cache
        runs_case("guesses 16 x 5", 16, 8192, 5, 4, 16, 128, 16, 16, 0, 0, True, "bf16", "int8"),
        # the tokens of a frame see each other and the seven frames before
        runs_case("frame of 8", 1, 7 * FRAME, FRAME, 16, 16, 64, 64, 32, 0, 0, False, "bf16", "bf16"),
        # fp32 prompts of uneven lengths with a window and first tokens, no past
        runs_case("prompts fp32 window", 3, 0, 1833, 8, 8, 64, 64, 32, 1000, 5, True, "fp32", "bf16"),
        # a chunk of two long prompts over the 8-bit cache, five queries to a head
        runs_case("chunk fp8", 2, 4001, 611, 4, 20, 128, 32, 16, 0, 0, True, "bf16", "fp8"),
        # the largest prompts, four queries to a head
        runs_case("prompts large", 4, 0, 8192, 8, 32, 128, 64, 64, 0, 0, True, "bf16", "bf16"),
    ]


def spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("tables", "append", "single", "runs", "runs"))
    x = rng.choice(("bf16", "bf16", "fp32"))
    dim, page = rng.choice((64, 128)), rng.choice((16, 32, 64, 128))
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    heads, share = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 1, 2, 4, 5, 8))
    if op == "tables":
        seqs = spread(rng, 1, 1000)
        c = tables_case("", seqs, spread(rng, 1, 2000), spread(rng, 1, max(1, min(4096, 400000 // seqs))), page)
    elif op == "append":
        seqs = spread(rng, 1, 64)
        tokens = 1 if rng.random() < 0.4 else spread(rng, 1, max(1, 16000 // seqs))
        c = append_case("", seqs, tokens, spread(rng, 1, 300), heads, heads * share, dim, rng.choice((1, 2)), page, block, x)
    elif op == "single":
        seqs = spread(rng, 1, 48)
        past = spread(rng, 1, min(100000, max(64, 12_000_000 // (seqs * heads * dim // 64))))
        window = spread(rng, 1, 4096) if rng.random() < 0.2 else 0
        c = single_case("", seqs, past, heads, heads * share, dim, page, block, window, x)
    else:
        seqs = spread(rng, 1, 32)
        run = rng.choice((1, spread(rng, 1, 16), spread(rng, 16, 8192), spread(rng, 16, 8192)))
        run = min(run, max(1, 16384 // seqs))
        # pairs of a query and a token, over all heads: no more than the largest listed case has
        most = 2_000_000_000 // (seqs * heads * share * run)
        past = spread(rng, 1, max(1, min(60000, 6_000_000 // (seqs * heads * dim // 64), most)))
        run = min(run, max(1, 2_000_000_000 // (seqs * heads * share * run)))
        window = spread(rng, 1, 4096) if rng.random() < 0.4 else 0
        c = runs_case("", seqs, past if rng.random() < 0.7 else 0, run, heads, heads * share, dim, page, block, window,
                      rng.choice((0, 1, 4, 5, 17, 70)) if window else 0, rng.random() < 0.75, x,
                      rng.choice(("bf16", "bf16", "int8", "fp8")))
    del c["name"]
    return c


def lengths(case):
    """(tokens in the cache before, tokens that join) of each sequence; the first one has the longest of both."""
    out = []
    for b in range(case["seqs"]):
        part = (0.618034 * b % 1.0) if b else 1.0
        past = int(case["past"] * part)
        if case["op"] == "append":
            out.append((int(case["past"] * (0.618034 * (b + 1) % 1.0)), case["tokens"]))
        elif case["run"] == 1:
            out.append((past, 1))
        else:  # every seventh sequence has none
            out.append((past, int(math.ceil(case["run"] * (0.754878 * b % 1.0 if b else 1.0))) if b % 7 != 3 else 0))
    return out


# ------------------------------------------------------------------------------------------ inputs

def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def ints(values):
    return torch.tensor(values, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = generator(seed)
    return {"tables": prepare_tables, "append": prepare_append, "single": prepare_attention,
            "runs": prepare_attention}[case["op"]](case, g)


def prepare_tables(case, g):
    both, page = lengths(case), case["page"]
    held = [-(-n // page) for n, _ in both]
    total = sum(-(-(n + m) // page) for n, m in both)
    pool = torch.randperm(total + 5, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((len(both), max(-(-(n + m) // page) for n, m in both) + 2), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = pool[at:at + n]
        at += n
    T = sum(m for _, m in both)
    empty = lambda *s, dtype=torch.int32: torch.empty(s, dtype=dtype, device="cuda")
    return {"case": case, "runs": ints([m for _, m in both]), "lens": ints([n for n, _ in both]),
            "free": pool[at:].contiguous(), "count": ints([total + 5 - at]), "table": table,
            "starts": empty(len(both) + 1), "after": empty(len(both)), "left": empty(1), "seq": empty(T),
            "index": empty(T), "slots": empty(T, dtype=torch.int64), "status": empty(len(both))}


def paged(case, rows, g):
    """(page table [seqs, most], number of pages): pages of a shuffled pool, -1 behind a sequence's last page."""
    need = [-(-n // case["page"]) for n in rows]
    pool = torch.randperm(sum(need) + 3, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((len(rows), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pool[at:at + n]
        at += n
    return table, len(pool)


def pages(case, count, g):
    """Key and value pages [pages, heads, page, dim] with plausible content, and the scales of an 8-bit cache."""
    shape = (count, case["heads"], case["page"], case["dim"])
    if case["cache"] == "bf16":
        k, v = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        return k, v, None, None
    if case["cache"] == "int8":
        k, v = (torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
        ks, vs = (0.01 + 0.015 * torch.rand(shape[:3], generator=g, device="cuda") for _ in range(2))
        return k, v, ks, vs
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(80).clamp_(-TOP, TOP)
            .to(torch.float8_e4m3fn) for _ in range(2))
    blocks = (count, case["heads"], case["page"] // case["block"])
    ks, vs = (torch.exp2(torch.randint(-7, -5, blocks, generator=g, device="cuda").float()) for _ in range(2))
    return k, v, ks, vs


def prepare_append(case, g):
    both, D = lengths(case), case["dim"]
    table, count = paged(case, [n + m for n, m in both], g)
    seq = torch.cat([torch.full((m,), b, dtype=torch.int32) for b, (_, m) in enumerate(both)]).cuda()
    index = torch.cat([torch.arange(n, n + m, dtype=torch.int32) for n, m in both]).cuda()
    T = len(seq)
    if case["axes"] == 1:
        position, places, base = index[:, None].contiguous(), max(n + m for n, m in both), 10000.0
    else:  # patches of a 37-wide image, by row and by column
        position, places, base = torch.stack((index % FRAME // 37, index % 37), 1).to(torch.int32).contiguous(), 38, 100.0
    w = D // case["axes"]
    angle = torch.arange(places, device="cuda")[:, None] * base ** (-torch.arange(0, w, 2, device="cuda") / w)
    qkv = torch.randn((T, case["q_heads"] + 2 * case["heads"], D), generator=g, device="cuda")
    qkv[:, :, torch.randperm(D, generator=g, device="cuda")[:3]] *= 8.0  # outlier channels
    q, kn, vn = qkv.to(DTYPES[case["x"]]).split((case["q_heads"], case["heads"], case["heads"]), 1)
    k, v, ks, vs = pages(case, count, g)
    page, slot = table[seq.long(), (index // case["page"]).long()].long(), (index % case["page"]).long()
    # every touched block of the cache, and the first place in it that a new token takes
    per = case["page"] // case["block"]
    first = torch.full((count * per,), case["block"], device="cuda")
    first.scatter_reduce_(0, page * per + slot // case["block"], slot % case["block"], "amin")
    s = {"case": case, "table": table, "seq": seq, "index": index, "position": position, "cos": angle.cos(),
         "sin": angle.sin(), "Q": q, "K": kn, "V": vn, "k": k, "v": v, "ks": ks, "vs": vs, "page": page, "slot": slot,
         "first": first, "Q_out": torch.empty((T, case["q_heads"], D), dtype=q.dtype, device="cuda")}
    if own:
        import bit_ptq_reconstruction_amd as qv

        s["cache"] = qv.QVKVCache(k, v, ks, vs)
    return s


def prepare_attention(case, g):
    both = lengths(case)
    table, count = paged(case, [n + m for n, m in both], g)
    k, v, ks, vs = pages(case, count, g)
    T = sum(m for _, m in both)
    Q = (1.5 * torch.randn((T, case["q_heads"], case["dim"]), generator=g, device="cuda")).to(DTYPES[case["x"]])
    starts = [0]
    for _, m in both:
        starts.append(starts[-1] + m)
    s = {"case": case, "table": table, "lens": ints([n + m for n, m in both]), "starts": ints(starts), "Q": Q, "k": k,
         "v": v, "ks": ks, "vs": vs, "O": torch.empty_like(Q)}
    if own:
        import bit_ptq_reconstruction_amd as qv

        s["cache"] = qv.QVKVCache(k, v, ks, vs)
        sizes = (case["q_heads"], case["heads"], case["dim"], table.shape[1] * case["page"])
        if case["op"] == "single":
            size = qv.qv_paged_attention_workspace_size(case["seqs"], *sizes)
        else:
            size = qv.qv_run_attention_workspace_size(T, case["seqs"], case["run"], *sizes)
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ passes

def run(s):
    return {"tables": run_tables, "append": run_append, "single": run_attention, "runs": run_attention}[s["case"]["op"]](s)


def run_tables(s):
    names = ("table", "starts", "after", "left", "seq", "index", "slots", "status")
    page = s["case"]["page"]
    if own:
        import bit_ptq_reconstruction_amd as qv

        qv.qv_page_tables(s["runs"], s["lens"], s["free"], s["count"], page, s["table"], s["starts"], s["after"],
                          s["left"], s["seq"], s["index"], s["slots"], s["status"])
        return {n: s[n] for n in names}
    runs, lens, T = s["runs"].long(), s["lens"].long(), len(s["seq"])
    starts = torch.nn.functional.pad(runs.cumsum(0), (1, 0))
    held = (lens + page - 1) // page
    need = (lens + runs + page - 1) // page - held
    before = need.cumsum(0) - need
    status = torch.where(lens + runs > s["table"].shape[1] * page, 1,
                         torch.where((need > 0) & (before + need > s["count"]), 2, torch.where(starts[1:] > T, 3, 0)))
    fits = status == 0
    column = torch.arange(s["table"].shape[1], device="cuda") - held[:, None]
    fresh = (column >= 0) & (column < need[:, None]) & fits[:, None]
    take = (s["count"] - 1 - before[:, None] - column).clamp(0, max(0, len(s["free"]) - 1))
    table = torch.where(fresh, s["free"][take.long()], s["table"])
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(starts[1:], t, right=True).clamp(max=len(runs) - 1)
    there = fits[seq] & (t < starts[-1])
    index = lens[seq] + t - starts[seq]
    slots = table[seq, (index // page).clamp(0, table.shape[1] - 1)].long() * page + index % page
    return {"table": table, "starts": starts.int(), "after": torch.where(fits, lens + runs, lens).int(),
            "left": (s["count"] - torch.where(fits, need, 0).sum()).int(), "seq": torch.where(there, seq, -1).int(),
            "index": torch.where(there, index, -1).int(), "slots": torch.where(there, slots, -1), "status": status.int()}


def rotated(x, s):
    """The position rotation of x [T, heads, dim] in 32 bits, every product and sum rounded by itself."""
    T, H, D = x.shape
    axes = s["case"]["axes"]
    x = x.float().view(T, H, axes, 2, D // axes // 2)
    c, n = s["cos"][s["position"].long()][:, None], s["sin"][s["position"].long()][:, None]  # [T, 1, axes, w / 2]
    a, b = x[:, :, :, 0], x[:, :, :, 1]
    return torch.stack((a * c - b * n, b * c + a * n), 3).view(T, H, D)


def scale_of(top):
    """The smallest power of two (2^-126 at least) by which ``top`` is no more than the 8-bit format's largest value."""
    part, power = torch.frexp(top)
    return torch.ldexp(torch.ones_like(top), (power - 9 + (part > TOP / 512)).clamp(min=-126))


def store_blocks(x, codes, scales, s):
    """x [T, heads, dim] into the cache: new scales of the touched blocks, older codes of a block whose scale grows."""
    case, pages, H = s["case"], codes.shape[0], codes.shape[1]
    block, per = case["block"], case["page"] // case["block"]
    at = s["page"] * per + s["slot"] // block
    top = torch.zeros((pages * per, H), device="cuda")
    top.scatter_reduce_(0, at[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    old = scales.transpose(1, 2).reshape(-1, H)
    touched, opened = s["first"] < block, s["first"] == 0
    new = torch.where(touched[:, None], torch.where(opened[:, None], scale_of(top), torch.maximum(old, scale_of(top))), old)
    older = (torch.arange(block, device="cuda") < s["first"][:, None]) & touched[:, None]  # [blocks, block]
    ratio = torch.where(older[:, :, None], (old / new)[:, None], 1.0)  # [blocks, block, heads]
    ratio = ratio.view(pages, case["page"], H).transpose(1, 2)[..., None]
    codes.copy_((codes.float() * ratio).to(codes.dtype))
    codes.view(torch.uint8)[s["page"], :, s["slot"]] = (x / new[at][..., None]).to(codes.dtype).view(torch.uint8)
    scales.copy_(new.view(pages, per, H).transpose(1, 2))


def values(codes, scales, s):
    """What the cache holds; codes times powers of two are exact in bf16."""
    shape = scales.shape + (s["case"]["block"], s["case"]["dim"])
    return codes.to(torch.bfloat16).view(shape).mul_(scales.to(torch.bfloat16)[..., None, None]).view(codes.shape)


def run_append(s):
    if own:
        import bit_ptq_reconstruction_amd as qv

        qv.qv_kv_append(s["cache"], s["table"], s["seq"], s["index"], s["K"], s["V"], s["cos"], s["sin"], s["position"],
                        s["Q"], s["Q_out"])
        Q = s["Q_out"]
    else:
        Q = rotated(s["Q"], s).to(s["Q"].dtype)
        store_blocks(rotated(s["K"], s), s["k"], s["ks"], s)
        store_blocks(s["V"].float(), s["v"], s["vs"], s)
    return {"k": values(s["k"], s["ks"], s), "v": values(s["v"], s["vs"], s), "q": Q}


def run_attention(s):
    case = s["case"]
    if own:
        import bit_ptq_reconstruction_amd as qv

        if case["op"] == "single":
            qv.qv_paged_attention(s["Q"], s["cache"], s["table"], s["lens"], s["O"], s["work"], window=case["window"])
        else:
            starts = None if case["run"] == 1 else s["starts"]
            qv.qv_run_attention(s["Q"], starts, case["run"], s["cache"], s["table"], s["lens"], s["O"], s["work"],
                                window=case["window"], sinks=case["sinks"], causal=case["causal"])
        return s["O"]
    B, Hq, H, D, n = case["seqs"], case["q_heads"], case["heads"], case["dim"], case["run"]
    r, L = Hq // H, s["table"].shape[1] * case["page"]
    T = len(s["Q"])
    out = torch.empty((T, Hq, D), dtype=s["O"].dtype, device="cuda")
    # sequences, and heads of one sequence, go in lots of about 2^28 scores
    heads = max(1, min(H, 2 ** 28 // (n * r * L)))
    lot = max(1, min(B, 2 ** 28 // (n * Hq * L)))
    t = torch.arange(L, device="cuda")
    i = torch.arange(n, device="cuda")
    for b in range(0, B, lot):
        lens, starts = s["lens"][b:b + lot].long(), s["starts"][b:b + lot + 1].long()
        counts = starts[1:] - starts[:-1]
        there = i < counts[:, None]  # [lot, n]
        row = (starts[:-1, None] + i).clamp(max=T - 1)
        place = (lens - counts)[:, None, None] + i[:, None]  # [lot, n, 1]
        sees = t < lens[:, None, None]
        if case["causal"]:
            sees = sees & (t <= place)
        if case["window"]:
            sees = sees & ((t < case["sinks"]) | (t > place - case["window"]))
        sees = sees[:, None, None]  # [lot, 1, 1, n, L]
        at = s["table"][b:b + lot].clamp(min=0).long()
        for h in range(0, H, heads):
            k, v = (s[name][at, h:h + heads].float() for name in ("k", "v"))  # [lot, pages, heads, page, D]
            if s["ks"] is not None:
                ks, vs = (s[name][at, h:h + heads].repeat_interleave(case["page"] // s[name].shape[2], -1)[..., None]
                          for name in ("ks", "vs"))
                k, v = k * ks, v * vs
            k, v = (x.transpose(1, 2).reshape(len(lens), -1, 1, L, D) for x in (k, v))
            q = s["Q"][row][:, :, h * r:(h + heads) * r].float().view(len(lens), n, -1, r, D).permute(0, 2, 3, 1, 4)
            p = torch.where(sees, (q @ k.transpose(-1, -2)) * D ** -0.5, -torch.inf)
            top = p.amax(-1, keepdim=True)
            p = torch.exp(p - torch.where(top > -torch.inf, top, 0))
            total = p.sum(-1, keepdim=True)
            o = (p @ v) / torch.where(total > 0, total, 1)  # [lot, heads, r, n, D]
            o = o.permute(0, 3, 1, 2, 4).reshape(len(lens), n, -1, D).to(out.dtype)
            out[row[there], h * r:(h + heads) * r] = o[there]
    return out


# -------------------------------------------------------------------------------------- work, exact

def visible(case, n, m):
    """(tokens that any query of a run sees, pairs of a query and a token that it sees) with n tokens before the run's m."""
    if m == 0:
        return 0, 0
    if not case["window"]:
        return n + m, (m * n + m * (m + 1) // 2 if case["causal"] else m * (n + m))
    w, sinks = case["window"], case["sinks"]
    pairs = 0
    for p in range(n, n + m):
        end = p + 1 if case["causal"] else n + m
        low = max(0, p - w + 1)
        pairs += end - low + min(sinks, low)
    low = max(0, n - w + 1)
    return n + m - low + min(sinks, low), pairs


def work(case):
    both = lengths(case)
    if case["op"] == "tables":
        T, page = sum(m for _, m in both), case["page"]
        fresh = sum(-(-(n + m) // page) - -(-n // page) for n, m in both)
        return {"bytes": 24 * len(both) + 8 * fresh + 16 * T, "flops": 0}
    D, H, Hq, x = case["dim"], case["heads"], case["q_heads"], BYTES[case["x"]]
    token = 2 * H * D * BYTES[case["cache"]]  # K and V of one token, with its scales
    token += {"bf16": 0, "int8": 8 * H, "fp8": 8 * H / case["block"]}[case["cache"]]
    if case["op"] == "append":
        T = len(both) * case["tokens"]
        return {"bytes": int(T * ((2 * Hq + 2 * H) * D * x + token + 8 + 4 * case["axes"] + D * 4)),
                "flops": T * (Hq + H) * D * 3 + T * H * D * 4}
    seen = [visible(case, n, m) for n, m in both]
    tokens, pairs, T = sum(a for a, _ in seen), sum(b for _, b in seen), sum(m for _, m in both)
    return {"bytes": int(tokens * token + tokens // case["page"] * 4 + 2 * T * Hq * D * x), "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": exact_tables, "append": exact_append, "single": exact_attention, "runs": exact_attention}[case["op"]](case, s)


def exact_tables(case, s):
    """By hand, a sequence at a time."""
    page, free = case["page"], s["free"].tolist()[:int(s["count"])]
    table, T = s["table"].cpu(), len(s["seq"])
    starts, after, status, used = [0], [], [], 0
    seq, index, slots = (torch.full((T,), -1, dtype=torch.int64) for _ in range(3))
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["runs"].tolist())):
        held, all_pages = -(-n // page), -(-(n + m) // page)
        at = starts[-1]
        starts.append(at + m)
        why = 1 if n + m > table.shape[1] * page else 2 if all_pages - held > len(free) else 3 if at + m > T else 0
        status.append(why)
        after.append(n if why else n + m)
        if not why:
            for j in range(held, all_pages):
                table[b, j] = free.pop()
            used += all_pages - held
            t = torch.arange(n, n + m)
            seq[at:at + m], index[at:at + m] = b, t
            slots[at:at + m] = table[b].long()[t // page] * page + t % page
    return {"table": table.cuda(), "starts": ints(starts), "after": ints(after), "left": ints([int(s["count"]) - used]),
            "seq": seq.int().cuda(), "index": index.int().cuda(), "slots": slots.cuda(), "status": ints(status)}


def exact_append(case, s):
    def turned(x):
        x = x.double()
        out = torch.empty_like(x)
        w = case["dim"] // case["axes"]
        for a in range(case["axes"]):
            at = s["position"][:, a].long()
            turn = torch.complex(s["cos"].double()[at], s["sin"].double()[at])[:, None]
            low, high = slice(a * w, a * w + w // 2), slice(a * w + w // 2, (a + 1) * w)
            z = torch.complex(x[..., low], x[..., high]) * turn
            out[..., low], out[..., high] = z.real, z.imag
        return out

    def nearest(x):
        """The 8-bit format's nearest value: 3 bits behind the leading one, steps of 2^-9 at least."""
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(x / step) * step

    def held(x, codes, scales):
        """Blocks [pages, blocks of a page, heads, tokens, dim] as they stand after the append."""
        block = case["block"]
        old = codes.double().view(codes.shape[0], codes.shape[1], -1, block, case["dim"]) * scales.double()[..., None, None]
        out = old.transpose(1, 2).clone()
        part, place = s["slot"] // block, s["slot"] % block
        raw = torch.zeros_like(out)
        raw[s["page"], part, :, place] = x
        new = torch.zeros(out.shape[:2] + (1, block, 1), dtype=torch.bool, device="cuda")
        new[s["page"], part, :, place] = True
        first = s["first"].view(out.shape[0], out.shape[1], 1, 1, 1)
        top = raw.abs().amax((3, 4), keepdim=True)
        step = torch.exp2(torch.ceil(torch.log2(top / TOP)).clamp(min=-126))
        before = scales.double().transpose(1, 2)[..., None, None]
        after = torch.where(first == block, before, torch.where(first == 0, step, torch.maximum(before, step)))
        older = torch.arange(block, device="cuda")[:, None] < first
        stale = out / before * after  # places behind the new tokens keep their codes
        out = torch.where(first == block, out, torch.where(older, nearest(out / after) * after, stale))
        out = torch.where(new, nearest(raw / after) * after, out)
        return out.transpose(1, 2).reshape(codes.shape)

    return {"k": held(turned(s["K"]), s["k"], s["ks"]), "v": held(s["V"].double(), s["v"], s["vs"]), "q": turned(s["Q"])}


def exact_attention(case, s):
    H, D, r = case["heads"], case["dim"], case["q_heads"] // case["heads"]
    out = torch.zeros((len(s["Q"]), H, r, D), dtype=torch.float64, device="cuda")
    start = 0
    for b, (n, m) in enumerate(lengths(case)):
        t = torch.arange(n + m, device="cuda")
        page, slot = s["table"][b].long()[t // case["page"]], t % case["page"]
        for h in range(H):
            k, v = s["k"][page, h, slot].double(), s["v"][page, h, slot].double()  # [tokens, D]
            if s["ks"] is not None:
                at = slot if case["cache"] == "int8" else slot // case["block"]
                k, v = k * s["ks"][page, h, at].double()[:, None], v * s["vs"][page, h, at].double()[:, None]
            for first in range(0, m, 2048):
                p = torch.arange(n + first, n + min(m, first + 2048), device="cuda")[:, None]
                hidden = (t > p) if case["causal"] else torch.zeros_like(t > p)
                if case["window"]:
                    hidden |= (t <= p - case["window"]) & (t >= case["sinks"])
                for g in range(r):
                    rows = slice(start + first, start + first + len(p))
                    scores = s["Q"][rows, h * r + g].double() @ k.t() / math.sqrt(D)
                    out[rows, h, g] = torch.softmax(scores.masked_fill_(hidden, -math.inf), -1) @ v
        start += m
    return out.view(len(s["Q"]), case["q_heads"], D)
