"""Cases of the single-token serving operators: the few-row linear with 4-bit weights, the append of
keys and values to a paged cache with the position rotation, and the attention of one new token over
that cache.  With ``own`` the framework's entry points run, without it their plain form in torch."""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2, "int8": 1}
FRAME = 1374  # tokens of one frame


# ------------------------------------------------------------------------------------------- cases

def linear_case(name, M, K, N, group, rotate, x, y, bias, gelu):
    return dict(name=name, op="linear", M=M, K=K, N=N, group=group, rotate=rotate, x=x, y=y, bias=bias, gelu=gelu)


def append_case(name, seqs, tokens, past, heads, q_heads, dim, axes, page, x, cache):
    return dict(name=name, op="append", seqs=seqs, tokens=tokens, past=past, heads=heads, q_heads=q_heads, dim=dim,
                axes=axes, page=page, x=x, cache=cache)


def attention_case(name, seqs, longest, ragged, heads, q_heads, dim, page, window, x, cache):
    return dict(name=name, op="attention", seqs=seqs, longest=longest, ragged=ragged, heads=heads, q_heads=q_heads,
                dim=dim, page=page, window=window, x=x, cache=cache)


def listed():
    return [
        # one token through the attention's output projection of a 1024-wide block: latency
        linear_case("linear 1 row", 1, 1024, 1024, 128, True, "bf16", "bf16", False, False),
        # three streams through the second linear of the MLP, rotated at width 4096
        linear_case("linear 3 rows wide", 3, 4096, 1024, 256, True, "bf16", "bf16", True, False),
        # fp32 activations, per-channel scales and GELU; an odd number of rows and of channels
        linear_case("linear 13 rows fp32", 13, 1024, 4099, 1024, True, "fp32", "fp32", True, True),
        # a batch of 16 through a large layer whose weights were not rotated
        linear_case("gemv 16 rows large", 16, 8192, 16384, 128, False, "bf16", "bf16", False, False),
        # one token of each of 24 sequences joins the cache, queries rotated on the way
        append_case("append 24 x 1", 24, 1, 700, 8, 32, 128, 1, 16, "bf16", "bf16"),
        # eight frames enter an empty cache, patches rotated by row and by column
        append_case("append 8 frames", 8, FRAME, 0, 16, 16, 64, 2, 64, "bf16", "bf16"),
        # a prompt of one odd length into the int8 cache, fp32 projections
        append_case("append int8", 3, 611, 37, 4, 16, 128, 1, 16, "fp32", "int8"),
        # one new token looks back on one frame, a head of its own for every query
        attention_case("attend 1 frame", 1, FRAME, False, 16, 16, 64, 16, 0, "bf16", "bf16"),
        # a served batch of uneven lengths, four queries to a head
        attention_case("attend ragged batch", 32, 4099, True, 8, 32, 128, 16, 0, "bf16", "bf16"),
        # fp32 queries that look back on a window of two frames
        attention_case("attend fp32 window", 5, 5 * FRAME, False, 16, 16, 64, 64, 2 * FRAME, "fp32", "bf16"),
        # two long contexts in the int8 cache, eight queries to a head
        attention_case("attend long int8", 2, 99991, False, 4, 32, 128, 64, 0, "bf16", "int8"),
        # the largest batch of long contexts
        attention_case("attend large batch", 48, 16384, True, 8, 32, 128, 64, 0, "bf16", "bf16"),
    ]


def spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("linear", "append", "attention"))
    x = rng.choice(("bf16", "bf16", "fp32"))
    if op == "linear":
        rotate = rng.random() < 0.6
        K = rng.choice((1024, 4096)) if rotate else 128 * spread(rng, 1, 96)
        group = rng.choice([g for g in (128, 256, 512, K) if K % g == 0])
        c = linear_case("", spread(rng, 1, 32), K, spread(rng, 65, 16384), group, rotate, x,
                        rng.choice(("bf16", "bf16", "fp32")), rng.random() < 0.5, rng.random() < 0.3)
    else:
        dim, page = rng.choice((64, 128)), rng.choice((16, 32, 64, 128))
        heads, share = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 1, 2, 4, 5, 8))
        cache = rng.choice(("bf16", "bf16", "int8"))
        if op == "append":
            seqs = spread(rng, 1, 64)
            tokens = 1 if rng.random() < 0.4 else spread(rng, 1, max(1, 16000 // seqs))
            c = append_case("", seqs, tokens, spread(rng, 1, 900), heads, heads * share, dim, rng.choice((1, 2)), page,
                            x, cache)
        else:
            seqs = spread(rng, 1, 48)
            longest = spread(rng, 1, min(100000, max(64, 12_000_000 // (seqs * heads * dim // 64))))
            window = spread(rng, 1, 4096) if rng.random() < 0.2 else 0
            c = attention_case("", seqs, longest, rng.random() < 0.6, heads, heads * share, dim, page, window, x, cache)
    del c["name"]
    return c


def lengths(case):
    """Tokens of each sequence: those in the cache before an append, or those that are attended."""
    if case["op"] == "append":
        return [int(case["past"] * (0.618034 * (b + 1) % 1.0)) for b in range(case["seqs"])]
    if not case["ragged"]:
        return [case["longest"]] * case["seqs"]
    return [case["longest"]] + [int(case["longest"] * (0.618034 * b % 1.0)) for b in range(1, case["seqs"])]


# ------------------------------------------------------------------------------------------ inputs

def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def hadamard_factor(n):
    """The n x n Sylvester matrix of +-1 (n a power of two)."""
    h = torch.ones((1, 1), device="cuda")
    while h.shape[0] < n:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h


def prepare(case, seed):
    g = generator(seed)
    return {"linear": prepare_linear, "append": prepare_append, "attention": prepare_attention}[case["op"]](case, g)


def prepare_linear(case, g):
    M, K, N, G = case["M"], case["K"], case["N"], case["K"] // case["group"]
    X = torch.randn((M, K), generator=g, device="cuda")
    X[:, torch.randperm(K, generator=g, device="cuda")[:8]] *= 20.0  # outlier channels
    codes = torch.randn((N, K), generator=g, device="cuda").mul_(2.3).round_().clamp_(-7, 7).to(torch.int8)
    Wq = ((codes[:, 0::2] & 15) | (codes[:, 1::2] << 4)).view(torch.uint8).contiguous()
    del codes
    ws = (0.004 + 0.008 * torch.rand((N, G), generator=g, device="cuda"))
    s = {"case": case, "X": X.to(DTYPES[case["x"]]), "Wq": Wq, "ws": ws[:, 0].contiguous() if G == 1 else ws,
         "bias": torch.randn((N,), generator=g, device="cuda") * 0.1 if case["bias"] else None,
         "inv": 0.5 + torch.rand((K,), generator=g, device="cuda") if case["rotate"] else None,
         "Y": torch.empty((M, N), dtype=DTYPES[case["y"]], device="cuda")}
    if case["rotate"]:
        s["h"] = hadamard_factor(math.isqrt(K))
        if own:
            import bit_ptq_reconstruction_amd as qv

            s["work"] = torch.empty(qv.qv_w4a16_linear_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    return s


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
    """Key and value pages [pages, heads, page, dim] with plausible content, and the int8 cache's scales."""
    shape = (count, case["heads"], case["page"], case["dim"])
    if case["cache"] == "bf16":
        k, v = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        return k, v, None, None
    k, v = (torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (0.01 + 0.015 * torch.rand(shape[:3], generator=g, device="cuda") for _ in range(2))
    return k, v, ks, vs


def prepare_append(case, g):
    before, T, D = lengths(case), case["seqs"] * case["tokens"], case["dim"]
    table, count = paged(case, [n + case["tokens"] for n in before], g)
    seq = torch.arange(case["seqs"], device="cuda", dtype=torch.int32).repeat_interleave(case["tokens"])
    index = (torch.tensor(before, device="cuda", dtype=torch.int32)[:, None]
             + torch.arange(case["tokens"], device="cuda", dtype=torch.int32)).reshape(-1).contiguous()
    if case["axes"] == 1:
        position, places, base = index[:, None].contiguous(), max(before) + case["tokens"], 10000.0
    else:  # patches of a 37-wide image, by row and by column
        position, places, base = torch.stack((index % FRAME // 37, index % 37), 1).to(torch.int32).contiguous(), 38, 100.0
    w = D // case["axes"]
    angle = torch.arange(places, device="cuda")[:, None] * base ** (-torch.arange(0, w, 2, device="cuda") / w)
    qkv = torch.randn((T, case["q_heads"] + 2 * case["heads"], D), generator=g, device="cuda").to(DTYPES[case["x"]])
    k, v, ks, vs = pages(case, count, g)
    q, kn, vn = qkv.split((case["q_heads"], case["heads"], case["heads"]), 1)
    s = {"case": case, "table": table, "seq": seq, "index": index, "position": position, "cos": angle.cos(),
         "sin": angle.sin(), "Q": q, "K": kn, "V": vn, "k": k, "v": v, "ks": ks, "vs": vs,
         "Q_out": torch.empty((T, case["q_heads"], D), dtype=qkv.dtype, device="cuda"),
         "page": table[seq.long(), (index // case["page"]).long()].long(), "slot": (index % case["page"]).long(),
         "levels": torch.full((), 127.0, device="cuda")}
    if own:
        import bit_ptq_reconstruction_amd as qv

        s["cache"] = qv.QVKVCache(k, v, ks, vs)
    return s


def prepare_attention(case, g):
    lens = lengths(case)
    table, count = paged(case, lens, g)
    k, v, ks, vs = pages(case, count, g)
    Q = torch.randn((case["seqs"], case["q_heads"], case["dim"]), generator=g, device="cuda").to(DTYPES[case["x"]])
    s = {"case": case, "table": table, "lens": torch.tensor(lens, device="cuda", dtype=torch.int32), "Q": Q, "k": k,
         "v": v, "ks": ks, "vs": vs, "O": torch.empty_like(Q)}
    if own:
        import bit_ptq_reconstruction_amd as qv

        s["cache"] = qv.QVKVCache(k, v, ks, vs)
        size = qv.qv_paged_attention_workspace_size(case["seqs"], case["q_heads"], case["heads"], case["dim"],
                                                    table.shape[1] * case["page"])
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ passes

def run(s):
    return {"linear": run_linear, "append": run_append, "attention": run_attention}[s["case"]["op"]](s)


def run_linear(s):
    case = s["case"]
    if own:
        import bit_ptq_reconstruction_amd as qv

        epi = qv.QV_EPI_GELU if case["gelu"] else qv.QV_EPI_NONE
        if case["rotate"]:
            qv.qv_w4a16_linear(s["X"], s["inv"], s["Wq"], s["ws"], case["group"], s["bias"], s["Y"], s["work"], epi)
        else:
            qv.qv_w4a16_gemv(s["X"], s["Wq"], s["ws"], case["group"], s["bias"], s["Y"], epi)
        return s["Y"]
    M, K, N = case["M"], case["K"], case["N"]
    x = s["X"].float()
    if case["rotate"]:  # H_K = H_n (x) H_n
        n = s["h"].shape[0]
        x = (s["h"] @ x.view(M, n, n) @ s["h"]).view(M, K) * (1.0 / n) * s["inv"]
    codes = torch.stack((s["Wq"] & 15, s["Wq"] >> 4), -1).view(N, -1, case["group"]).to(torch.int8)
    codes = torch.where(codes > 7, codes - 16, codes)
    w = (codes.float() * s["ws"].view(N, -1, 1)).view(N, K)
    y = x @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["gelu"]:
        y = 0.5 * y * torch.erfc(-y * math.sqrt(0.5))
    return y.to(s["Y"].dtype)


def rotated(x, s):
    """The position rotation of x [T, heads, dim] in 32 bits, every product and sum rounded by itself."""
    T, H, D = x.shape
    axes = s["case"]["axes"]
    x = x.float().view(T, H, axes, 2, D // axes // 2)
    c, n = s["cos"][s["position"].long()][:, None], s["sin"][s["position"].long()][:, None]  # [T, 1, axes, w / 2]
    a, b = x[:, :, :, 0], x[:, :, :, 1]
    return torch.stack((a * c - b * n, b * c + a * n), 3).view(T, H, D)


def coded(x, s):
    """(int8 codes, scales) of x [T, heads, dim], one scale to a token and head."""
    scale = x.abs().amax(-1) / s["levels"]
    q = (x / scale[..., None]).round().clamp(-128, 127)
    return torch.where(scale[..., None] > 0, q, 0).to(torch.int8), scale


def run_append(s):
    if own:
        import bit_ptq_reconstruction_amd as qv

        qv.qv_kv_append(s["cache"], s["table"], s["seq"], s["index"], s["K"], s["V"], s["cos"], s["sin"],
                        s["position"], s["Q"], s["Q_out"])
        Q = s["Q_out"]
    else:
        K, V, Q = rotated(s["K"], s), s["V"].float(), rotated(s["Q"], s).to(s["Q"].dtype)
        if s["ks"] is None:
            s["k"][s["page"], :, s["slot"]] = K.to(torch.bfloat16)
            s["v"][s["page"], :, s["slot"]] = V.to(torch.bfloat16)
        else:
            s["k"][s["page"], :, s["slot"]], s["ks"][s["page"], :, s["slot"]] = coded(K, s)
            s["v"][s["page"], :, s["slot"]], s["vs"][s["page"], :, s["slot"]] = coded(V, s)
    if s["ks"] is None:
        return {"k": s["k"], "v": s["v"], "q": Q}
    at = (s["page"], slice(None), s["slot"])  # codes as the values they stand for
    return {"k": s["k"][at].float() * s["ks"][at][..., None], "v": s["v"][at].float() * s["vs"][at][..., None], "q": Q}


def run_attention(s):
    case = s["case"]
    B, Hq, H, D = case["seqs"], case["q_heads"], case["heads"], case["dim"]
    if own:
        import bit_ptq_reconstruction_amd as qv

        qv.qv_paged_attention(s["Q"], s["cache"], s["table"], s["lens"], s["O"], s["work"], window=case["window"])
        return s["O"]
    at = s["table"].clamp(min=0).long()
    k, v = (s[n][at].float() for n in ("k", "v"))  # [B, pages, H, page, D]
    if s["ks"] is not None:
        k, v = k * s["ks"][at][..., None], v * s["vs"][at][..., None]
    t = torch.arange(at.shape[1] * case["page"], device="cuda")
    inside = t < s["lens"][:, None]
    if case["window"]:
        inside &= t >= s["lens"][:, None] - case["window"]
    k, v = (x.transpose(1, 2).reshape(B, H, -1, D) for x in (k, v))
    inside = inside[:, None, None]
    p = (s["Q"].float().view(B, H, Hq // H, D) @ k.transpose(-1, -2)) * D ** -0.5
    p = torch.where(inside, p, -torch.inf)
    top = p.amax(-1, keepdim=True)
    p = torch.where(inside, (p - torch.where(top > -torch.inf, top, 0)).exp(), 0)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, 1)
    return o.view(B, Hq, D).to(s["O"].dtype)


# -------------------------------------------------------------------------------------- work, exact

def work(case):
    x = BYTES[case["x"]]
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        extra = (4 * K if case["rotate"] else 0) + (4 * N if case["bias"] else 0)
        rotation = M * K * math.log2(K) if case["rotate"] else 0
        return {"bytes": N * K // 2 + 4 * N * (K // case["group"]) + M * K * x + M * N * BYTES[case["y"]] + extra,
                "flops": 2 * M * N * K + rotation}
    D, H, Hq = case["dim"], case["heads"], case["q_heads"]
    c = BYTES[case["cache"]]
    token = 2 * H * (D * c + (4 if case["cache"] == "int8" else 0))  # K and V of one token
    if case["op"] == "append":
        T = case["seqs"] * case["tokens"]
        return {"bytes": T * ((2 * Hq + 2 * H) * D * x + token + 8 + 4 * case["axes"] + D * 4), "flops": T * (Hq + H) * D * 3}
    n = sum(min(v, case["window"]) if case["window"] else v for v in lengths(case))
    return {"bytes": n * token + n // case["page"] * 4 + 2 * case["seqs"] * Hq * D * x, "flops": 4 * n * Hq * D}


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": exact_linear, "append": exact_append, "attention": exact_attention}[case["op"]](case, s)


def exact_linear(case, s):
    K, group = case["K"], case["group"]
    x = s["X"].double()
    if case["rotate"]:
        i = torch.arange(K, device="cuda")
        odd = i[:, None] & i[None, :]
        for shift in (8, 4, 2, 1):
            odd = odd ^ (odd >> shift)
        x = x @ (1.0 - 2.0 * (odd & 1).double()) / math.sqrt(K) * s["inv"].double()
    y = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device="cuda")
    low, high = s["Wq"].to(torch.int16) & 15, s["Wq"].to(torch.int16) >> 4
    low, high = low - 16 * (low >= 8), high - 16 * (high >= 8)
    scale = s["ws"].double().view(case["N"], -1)
    for g in range(K // group):
        half = slice(g * group // 2, (g + 1) * group // 2)
        even, odd = x[:, g * group:(g + 1) * group:2], x[:, g * group + 1:(g + 1) * group:2]
        y += (even @ low[:, half].double().t() + odd @ high[:, half].double().t()) * scale[:, g]
    if s["bias"] is not None:
        y += s["bias"].double()
    return y * torch.special.ndtr(y) if case["gelu"] else y


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

    K, V, Q = turned(s["K"]), s["V"].double(), turned(s["Q"])
    if s["ks"] is not None:
        def held(x):
            step = x.abs().amax(-1, keepdim=True) / 127
            return torch.round(x / step) * step
        return {"k": held(K), "v": held(V), "q": Q}
    k, v = s["k"].double(), s["v"].double()
    k[s["page"], :, s["slot"]], v[s["page"], :, s["slot"]] = K, V
    return {"k": k, "v": v, "q": Q}


def exact_attention(case, s):
    B, H, D, r = case["seqs"], case["heads"], case["dim"], case["q_heads"] // case["heads"]
    out = torch.zeros((B, H, r, D), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        t = torch.arange(first, n, device="cuda")
        page, slot = s["table"][b].long()[t // case["page"]], t % case["page"]
        q = s["Q"][b].double().view(H, r, D)
        k, v = s["k"][page, :, slot].double(), s["v"][page, :, slot].double()  # [t, H, D]
        if s["ks"] is not None:
            k, v = k * s["ks"][page, :, slot].double()[..., None], v * s["vs"][page, :, slot].double()[..., None]
        weight = torch.softmax(q @ k.permute(1, 2, 0) / math.sqrt(D), -1)
        out[b] = weight @ v.transpose(0, 1)
    return out.view(B, case["q_heads"], D)
