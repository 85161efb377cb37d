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

    The block has no biases, no weights in its norms and no smoothing.

    The cache for ``sequences`` sequences of up to ``capacity`` tokens (rounded up to whole pages), the workspaces and the
    linears' and the attention's outputs are allocated here, so a step can be captured in a graph.  The norms and residual
    sums are torch's and allocate theirs (under capture from the graph's pool), and so does take_frame().

    ``positions`` places along each of ``axes`` axes have an angle; the output of a token at another one, and of those that
    come after it in its sequence, is NaN.  A frame has up to ``frame_tokens`` tokens."""

    def __init__(self, qv, weights, sequences: int, capacity: int, device, heads: int = 16, axes: int = 1,
                 positions: int = 4096, base: float = 10000.0, int8_cache: bool = False, page_size: int = 64,
                 frame_tokens: int = 0):
        import torch

        self.qv, self.B, self.heads, self.width = qv, sequences, heads, 1024
        if heads not in (8, 16):
            raise ValueError(f"StreamBlock: {heads} heads of a width of 1024, the attention takes 64 (16 heads) or 128 (8) channels")
        self.dim = self.width // heads
        empty = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=device)
        byte = lambda n: empty(n, dtype=torch.uint8)
        self.linears = {lin.name: lin for lin in configs.block_linears()}
        self.Wq, self.ws = {}, {}
        for name, lin in self.linears.items():
            self.Wq[name] = empty(lin.N, lin.K // 2, dtype=torch.uint8)
            self.ws[name] = empty(lin.N, lin.K // GROUP, dtype=torch.float32)
            qv.qv_pack_weights_grouped(weights[name].contiguous(), None, GROUP, self.Wq[name], self.ws[name])
        pages = -(-capacity // page_size)
        shape = (sequences * pages, heads, page_size, self.dim)
        kind = torch.int8 if int8_cache else torch.bfloat16
        # NaN (int8: under scales of NaN), so that a token that was not stored shows in whatever attends to it.
        nan = float("nan")
        scales = [torch.full(shape[:3], nan, device=device) for _ in range(2)] if int8_cache else [None, None]
        self.cache = qv.QVKVCache(*(torch.full(shape, 0 if int8_cache else nan, dtype=kind, device=device) for _ in range(2)),
                                  *scales)
        self.table = torch.arange(sequences * pages, dtype=torch.int32, device=device).view(sequences, pages)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.held = [0] * sequences  # the host's copy of lens
        self.position = torch.zeros((sequences, axes), dtype=torch.int32, device=device)
        w = self.dim // axes
        angle = torch.arange(positions, device=device)[:, None] * base ** (-torch.arange(0, w, 2, device=device) / w)
        self.cos, self.sin = angle.cos(), angle.sin()
        self.one = self._buffers(sequences, empty, byte, few=True)
        self.frame = self._buffers(frame_tokens, empty, byte, few=False)

    def _buffers(self, rows, empty, byte, few: bool):
        qv = self.qv
        b = {name: empty(rows, lin.N) for name, lin in self.linears.items()}
        b["q"], b["o"] = empty(rows, self.heads, self.dim), empty(rows, self.heads, self.dim)
        size = qv.qv_w4a16_linear_workspace_size if few else lambda M, K: qv.qv_w4a4_linear_grouped_workspace_size(M, K, GROUP)
        b["work"] = byte(max(size(rows, lin.K) for lin in self.linears.values()))
        if few:
            b["parts"] = byte(qv.qv_paged_attention_workspace_size(rows, self.heads, self.heads, self.dim,
                                                                   self.table.shape[1] * self.cache.page_size))
        return b

    def _linear(self, name, x, b, few: bool):
        lin, qv = self.linears[name], self.qv
        if few:
            qv.qv_w4a16_linear(x, None, self.Wq[name], self.ws[name], GROUP, None, b[name], b["work"], lin.epi)
        else:
            qv.qv_w4a4_linear_grouped(x, None, GROUP, self.Wq[name], self.ws[name], None, b[name], b["work"], lin.epi)
        return b[name]

    def _need_room(self, tokens: int, sequences) -> None:
        room = self.table.shape[1] * self.cache.page_size
        for s in sequences:
            if self.held[s] + tokens > room:
                raise ValueError(f"StreamBlock: sequence {s} holds {self.held[s]} tokens and has no room for {tokens} more in {room}")

    def reserve(self) -> None:
        """Counts one token of every sequence, or raises ValueError where one has no room: to be called before each replay
        of a captured step, which the host does not see.  (Who sets ``lens`` sets ``held`` as well.)"""
        self._need_room(1, range(self.B))
        self.held = [n + 1 for n in self.held]

    def _norm(self, x):
        import torch

        return torch.nn.functional.layer_norm(x, (self.width,))

    def _heads(self, qkv):
        qkv = qkv.view(-1, 3, self.heads, self.dim)
        return qkv[:, 0], qkv[:, 1], qkv[:, 2]

    def take_frame(self, x, sequence: int, position) -> None:
        """Keys and values of a frame's tokens x [T, 1024] join ``sequence`` (position [T, axes] int32).  Attention
        inside a frame is not part of this class."""
        import torch

        T, b = x.shape[0], {name: t[:x.shape[0]] if name in self.linears else t for name, t in self.frame.items()}
        if not 0 <= sequence < self.B:
            raise ValueError(f"StreamBlock: sequence {sequence} of {self.B}")
        if T > len(self.frame["qkv"]):
            raise ValueError(f"StreamBlock: a frame of {T} tokens, the block was made for frames of up to {len(self.frame['qkv'])}")
        self._need_room(T, [sequence])
        q, k, v = self._heads(self._linear("qkv", self._norm(x), b, few=False))
        index = self.lens[sequence] + torch.arange(T, dtype=torch.int32, device=x.device)
        owner = torch.full_like(index, sequence)
        self.qv.qv_kv_append(self.cache, self.table, owner, index, k, v, self.cos, self.sin, position)
        self.lens[sequence] += T
        self.held[sequence] += T

    def step(self, x):
        """One new token x [B, 1024] bf16 of every sequence, at ``self.position`` [B, axes]; returns the block's output.
        ValueError where a sequence has no room for it."""
        import torch

        qv, b = self.qv, self.one
        captured = torch.cuda.is_current_stream_capturing()  # runs later, see reserve()
        if not captured:
            self._need_room(1, range(self.B))
        q, k, v = self._heads(self._linear("qkv", self._norm(x), b, few=True))
        qv.qv_kv_append(self.cache, self.table, None, self.lens, k, v, self.cos, self.sin, self.position, q, b["q"])
        self.lens += 1
        if not captured:
            self.held = [n + 1 for n in self.held]
        qv.qv_paged_attention(b["q"], self.cache, self.table, self.lens, b["o"], b["parts"])
        y = x + self._linear("proj", b["o"].view(self.B, self.width), b, few=True)
        return y + self._linear("fc2", self._linear("fc1", self._norm(y), b, few=True), b, few=True)
