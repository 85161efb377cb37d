"""One transformer block that takes its tokens as they come: a frame's tokens at once, then one new token of every
sequence at a time, with 4-bit weights throughout and the keys and values of the past in a paged cache.

A frame runs through the W4A4 linears (tiles of 128 rows, activations rounded to 4 bits), single tokens through the
few-row linears (activations not rounded), both over the same packed weights with group scales.  Keys and queries
are turned by the tokens' positions on an image grid (row and column) or in a line.

    y = x + proj(attention(qkv(norm(x)))),   out = y + fc2(gelu(fc1(norm(y))))
"""
from __future__ import annotations

from . import configs

GROUP = 128


class StreamBlock:
    """``weights``: {"qkv", "proj", "fc1", "fc2"} -> [N, K] fp32/bf16 of a block of width 1024 with ``heads`` heads.

    ``cache`` holds bf16, int8 with a scale per token (``int8_cache``) or float8_e4m3fn with a scale per page
    (``fp8_cache``).  A token sees the last ``window`` tokens up to itself (0: all) and the first ``sinks``.  With ``pages`` the
    sequences share that many pages and take them as they grow (end() gives a sequence's back; a window gives none back, so that
    a sequence ends at ``capacity`` with one as well); else each has its own.

    The block has no biases, no weights in its norms and no smoothing.

    The cache for ``sequences`` sequences of up to ``capacity`` tokens (rounded up to whole pages), the workspaces and the
    linears' and the attention's outputs are allocated here, so a step can be captured in a graph.  The norms and residual
    sums are torch's and allocate theirs (under capture from the graph's pool), and so do take_frame()
    and take_runs(), which reads its runs on the host and is not for capture.

    ``positions`` places along each of ``axes`` axes have an angle; the output of a token at another one is NaN, and so is that of
    the tokens that attend to it: those that come after it in its sequence (or with it, where a run is not causal) as long as
    it is among the last ``window`` or first ``sinks`` tokens.  A frame, or the runs of one call, has up to ``frame_tokens`` tokens."""

    def __init__(self, qv, weights, sequences: int, capacity: int, device, heads: int = 16, axes: int = 1,
                 positions: int = 4096, base: float = 10000.0, int8_cache: bool = False, page_size: int = 64,
                 frame_tokens: int = 0, fp8_cache: bool = False, window: int = 0, sinks: int = 0, pages: int = None):
        import torch

        self.qv, self.B, self.heads, self.width = qv, sequences, heads, 1024
        if heads not in (8, 16):
            raise ValueError(f"StreamBlock: {heads} heads of a width of 1024, the attention takes 64 (16 heads) or 128 (8) channels")
        self.dim = self.width // heads
        if int8_cache and fp8_cache:
            raise ValueError("StreamBlock: a cache is int8 or FP8")
        for name, n in (("window", window), ("sinks", sinks)):
            if not hasattr(n, "__index__") or not 0 <= n < 1 << 63:
                raise ValueError(f"StreamBlock: {name} {n} is not a number of tokens")
        self.window, self.sinks = window, sinks
        empty = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=device)
        byte = lambda n: empty(n, dtype=torch.uint8)
        self.linears = {lin.name: lin for lin in configs.block_linears()}
        self.Wq, self.ws = {}, {}
        for name, lin in self.linears.items():
            self.Wq[name] = empty(lin.N, lin.K // 2, dtype=torch.uint8)
            self.ws[name] = empty(lin.N, lin.K // GROUP, dtype=torch.float32)
            qv.qv_pack_weights_grouped(weights[name].contiguous(), None, GROUP, self.Wq[name], self.ws[name])
        each = -(-capacity // page_size)
        self.pooled = pages is not None
        shape = (pages if self.pooled else sequences * each, heads, page_size, self.dim)
        # NaN (int8: under scales of NaN), so that a token that was not stored shows in whatever attends to it.
        nan = float("nan")
        scales = [None, None]
        if int8_cache or fp8_cache:
            scales = [torch.full(shape[:3] if int8_cache else shape[:2] + (1,), nan, device=device) for _ in range(2)]
        content = [torch.full(shape, 0 if int8_cache else nan, dtype=torch.int8 if int8_cache else torch.bfloat16, device=device)
                   for _ in range(2)]
        if fp8_cache:
            content = [x.to(torch.float8_e4m3fn) for x in content]
        self.cache = qv.QVKVCache(*content, *scales)
        if self.pooled:
            self.table = torch.full((sequences, each), -1, dtype=torch.int32, device=device)
            self.free = torch.arange(pages, dtype=torch.int32, device=device)
            self.count = torch.full((1,), pages, dtype=torch.int32, device=device)
            self.left = pages  # the host's copy of count
            self.ones = torch.ones(sequences, dtype=torch.int32, device=device)
        else:
            self.table = torch.arange(sequences * each, dtype=torch.int32, device=device).view(sequences, each)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.held = [0] * sequences  # the host's copy of lens
        self.axes = axes
        self.position = torch.zeros((sequences, axes), dtype=torch.int32, device=device)
        w = self.dim // axes
        angle = torch.arange(positions, device=device)[:, None] * base ** (-torch.arange(0, w, 2, device=device) / w)
        self.cos, self.sin = angle.cos(), angle.sin()
        self.one = self._buffers(sequences, empty, byte, few=True)
        self.frame = self._buffers(frame_tokens, empty, byte, few=False)

    def _buffers(self, rows, empty, byte, few: bool):
        import torch

        qv = self.qv
        b = {name: empty(rows, lin.N) for name, lin in self.linears.items()}
        b["q"], b["o"] = empty(rows, self.heads, self.dim), empty(rows, self.heads, self.dim)
        size = qv.qv_w4a16_linear_workspace_size if few else lambda M, K: qv.qv_w4a4_linear_grouped_workspace_size(M, K, GROUP)
        if self.pooled or not few:  # of qv_page_tables
            number = lambda n, dtype=torch.int32: empty(n, dtype=dtype)
            b["map"] = [number(self.B + 1), number(rows), number(rows), number(rows, torch.int64), number(self.B)]
        b["work"] = byte(max(size(rows, lin.K) for lin in self.linears.values()))
        if few:
            room = self.table.shape[1] * self.cache.page_size
            b["parts"] = byte(qv.qv_run_attention_workspace_size(rows, rows, 1, self.heads, self.heads, self.dim, room))
        return b

    def _linear(self, name, x, b, few: bool):
        lin, qv = self.linears[name], self.qv
        if few:
            qv.qv_w4a16_linear(x, None, self.Wq[name], self.ws[name], GROUP, None, b[name], b["work"], lin.epi)
        else:
            qv.qv_w4a4_linear_grouped(x, None, GROUP, self.Wq[name], self.ws[name], None, b[name], b["work"], lin.epi)
        return b[name]

    def _pages(self, tokens: int) -> int:
        return -(-tokens // self.cache.page_size)

    def _need_room(self, runs) -> int:
        """The pages that runs[s] more tokens of each sequence s take from the pool; ValueError where there is no room."""
        room, need = self.table.shape[1] * self.cache.page_size, 0
        for s, n in enumerate(runs):
            if self.held[s] + n > room:
                raise ValueError(f"StreamBlock: sequence {s} holds {self.held[s]} tokens and has no room for {n} more in {room}")
            need += self._pages(self.held[s] + n) - self._pages(self.held[s])
        if not self.pooled:
            return 0
        if need > self.left:
            raise ValueError(f"StreamBlock: {need} pages needed, {self.left} of {self.cache.pages} are free")
        return need

    def _check_positions(self, position, rows: int) -> None:
        """ValueError unless the append takes the positions of ``rows`` tokens: what it refuses comes before they have places."""
        import torch

        if position is None and self.axes == 1:
            return  # the places themselves
        if (not torch.is_tensor(position) or position.dtype != torch.int32 or tuple(position.shape) != (rows, self.axes)
                or not position.is_contiguous() or position.device != self.lens.device):
            what = f"{position.dtype} {list(position.shape)} on {position.device}" if torch.is_tensor(position) else type(position).__name__
            raise ValueError(f"StreamBlock: position is {what}, expected dense int32 [{rows}, {self.axes}] on {self.lens.device}")

    def _count(self, runs, need: int) -> None:
        self.held = [n + m for n, m in zip(self.held, runs)]
        if self.pooled:
            self.left -= need

    def reserve(self) -> None:
        """Counts one token of every sequence, or raises ValueError where one has no room: to be called before each replay
        of a captured step, which the host does not see.  (Who sets ``lens`` sets ``held`` as well.)"""
        runs = [1] * self.B
        self._count(runs, self._need_room(runs))

    def _places(self, runs, rows: int, b):
        """Rows of the new tokens, runs [B] int32 of each sequence: (starts, sequence and place of each row); the pages that
        they need join the table, and the lengths grow."""
        starts, seq, index, slots, status = b["map"]
        self.qv.qv_page_tables(runs, self.lens, self.free, self.count, self.cache.page_size, self.table, starts, self.lens,
                               self.count, seq[:rows], index[:rows], slots[:rows], status)
        return starts, seq[:rows], index[:rows]

    def end(self, sequence: int) -> None:
        """The sequence is over: it has no tokens, its pages hold NaN as at the start and are free again where they are shared."""
        import torch

        n = self._pages(self.held[sequence])
        pages = self.table[sequence, :n].long()
        for content, scales in ((self.cache.k_pages, self.cache.k_scale), (self.cache.v_pages, self.cache.v_scale)):
            if content.dtype == torch.float8_e4m3fn:
                content.view(torch.uint8)[pages] = 0x7F  # NaN
            (content if scales is None else scales)[pages] = float("nan")
        if self.pooled:
            self.free[self.left:self.left + n] = self.table[sequence, :n]
            self.table[sequence, :n] = -1
            self.left += n
            self.count.fill_(self.left)
        self.lens[sequence] = 0
        self.held[sequence] = 0

    def _norm(self, x):
        import torch

        return torch.nn.functional.layer_norm(x, (self.width,))

    def _heads(self, qkv):
        qkv = qkv.view(-1, 3, self.heads, self.dim)
        return qkv[:, 0], qkv[:, 1], qkv[:, 2]

    def take_frame(self, x, sequence: int, position) -> None:
        """Keys and values of a frame's tokens x [T, 1024] join ``sequence`` (position [T, axes] int32).  take_runs()
        has the attention inside a frame."""
        T = x.shape[0]
        if not 0 <= sequence < self.B:
            raise ValueError(f"StreamBlock: sequence {sequence} of {self.B}")
        if T > len(self.frame["qkv"]):
            raise ValueError(f"StreamBlock: a frame of {T} tokens, the block was made for frames of up to {len(self.frame['qkv'])}")
        runs = [T if s == sequence else 0 for s in range(self.B)]
        if self.pooled:
            self._take(x, runs, position, None)
            return
        import torch

        b = {name: t[:T] if name in self.linears else t for name, t in self.frame.items()}
        self._check_positions(position, T)
        self._need_room(runs)
        q, k, v = self._heads(self._linear("qkv", self._norm(x), b, few=False))
        index = self.lens[sequence] + torch.arange(T, dtype=torch.int32, device=x.device)
        owner = torch.full_like(index, sequence)
        self.qv.qv_kv_append(self.cache, self.table, owner, index, k, v, self.cos, self.sin, position)
        self.lens[sequence] += T
        self._count(runs, 0)

    def take_runs(self, x, runs, position, causal: bool = True):
        """New tokens of many sequences at once, prompts, frames or chunks of them: x [T, 1024] bf16 has runs[s] rows of each
        sequence s, one behind the other (position [T, axes] int32).  They join the cache and attend to it, to those before
        them alone (``causal``) or to all of their run; returns the block's output [T, 1024]."""
        runs = [int(n) for n in runs]
        if len(runs) != self.B or min(runs) < 0 or sum(runs) != x.shape[0]:
            raise ValueError(f"StreamBlock: runs {runs} of {self.B} sequences for {x.shape[0]} tokens")
        if x.shape[0] > len(self.frame["qkv"]):
            raise ValueError(f"StreamBlock: {x.shape[0]} tokens, the block was made for frames of up to {len(self.frame['qkv'])}")
        return self._take(x, runs, position, bool(causal))

    def _take(self, x, runs, position, causal):
        import torch

        qv, T = self.qv, x.shape[0]
        b = {name: t[:T] if name in self.linears or name in ("q", "o") else t for name, t in self.frame.items()}
        self._check_positions(position, T)
        need = self._need_room(runs)
        if causal is not None:  # before the tokens have places: there may be no memory for it
            room = self.table.shape[1] * self.cache.page_size
            size = qv.qv_run_attention_workspace_size(T, self.B, max(runs), self.heads, self.heads, self.dim, room)
            parts = torch.empty(size, dtype=torch.uint8, device=x.device)
        q, k, v = self._heads(self._linear("qkv", self._norm(x), b, few=False))
        if self.pooled:
            starts, seq, index = self._places(torch.tensor(runs, dtype=torch.int32, device=x.device), T, b)
        else:
            number = lambda values: torch.tensor(values, dtype=torch.int32, device=x.device)
            starts = number([sum(runs[:s]) for s in range(self.B + 1)])
            seq = number([s for s, n in enumerate(runs) for _ in range(n)])
            index = number([self.held[s] + i for s, n in enumerate(runs) for i in range(n)])
            self.lens += number(runs)
        self._count(runs, need)
        queries = (None, None) if causal is None else (q, b["q"])
        qv.qv_kv_append(self.cache, self.table, seq, index, k, v, self.cos, self.sin, position, *queries)
        if causal is None:
            return None
        qv.qv_run_attention(b["q"], starts, max(runs), self.cache, self.table, self.lens, b["o"], parts, window=self.window,
                            sinks=self.sinks, causal=causal)
        y = x + self._linear("proj", b["o"].view(T, self.width), b, few=False)
        # The linears' rounding to 4 bits takes finite rows.  A token that was not stored makes every channel of every head NaN.
        y.masked_fill_(b["o"][:, 0, :1].isnan(), float("nan"))
        return y + self._linear("fc2", self._linear("fc1", self._norm(y), b, few=False), b, few=False)

    def step(self, x):
        """One new token x [B, 1024] bf16 of every sequence, at ``self.position`` [B, axes]; returns the block's output.
        ValueError where a sequence has no room for it."""
        import torch

        qv, b = self.qv, self.one
        captured = torch.cuda.is_current_stream_capturing()  # runs later, see reserve()
        runs = [1] * self.B
        self._check_positions(self.position, self.B)
        need = 0 if captured else self._need_room(runs)
        q, k, v = self._heads(self._linear("qkv", self._norm(x), b, few=True))
        if self.pooled:
            _, seq, index = self._places(self.ones, self.B, b)
        else:
            seq, index = None, self.lens
        qv.qv_kv_append(self.cache, self.table, seq, index, k, v, self.cos, self.sin, self.position, q, b["q"])
        if not self.pooled:
            self.lens += 1
        if not captured:
            self._count(runs, need)
        qv.qv_run_attention(b["q"], None, 1, self.cache, self.table, self.lens, b["o"], b["parts"], window=self.window,
                            sinks=self.sinks)
        y = x + self._linear("proj", b["o"].view(self.B, self.width), b, few=True)
        return y + self._linear("fc2", self._linear("fc1", self._norm(y), b, few=True), b, few=True)
