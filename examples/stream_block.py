"""Frames enter a block's paged cache, then single tokens are answered from it: the few-row 4-bit linears, the append
with the position rotation and the paged attention in one captured step.

    python examples/stream_block.py [--frames 2] [--sequences 4] [--tokens 64] [--int8]
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import bit_ptq_reconstruction_amd as qv  # noqa: E402
from bit_ptq_reconstruction_amd import configs, synth  # noqa: E402
from bit_ptq_reconstruction_amd.stream import StreamBlock  # noqa: E402

GRID = 37  # a frame's patches are GRID x GRID, after its special tokens


def frame_positions(device):
    """(row, column) of a frame's tokens; the special tokens lie at the origin."""
    patch = torch.arange(GRID * GRID, device=device)
    p = torch.stack((patch // GRID + 1, patch % GRID + 1), 1)
    return torch.cat((torch.zeros((synth.SPECIAL_TOKENS, 2), device=device), p)).to(torch.int32).contiguous()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--frames", type=int, default=2)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--int8", action="store_true", help="int8 cache instead of bf16")
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    T = synth.FRAME_TOKENS
    weights = {lin.name: synth.weights_torch(lin.N, lin.K, lin.w_seed, dev) for lin in configs.block_linears()}
    block = StreamBlock(qv, weights, a.sequences, a.frames * T + a.tokens + 8, dev, axes=2, positions=GRID + 1, base=100.0,
                        int8_cache=a.int8, frame_tokens=T)
    where = frame_positions(dev)
    for s in range(a.sequences):
        for f in range(a.frames):
            block.take_frame(synth.vggt_activations_torch(T, 1024, 1000 * s + f, torch.bfloat16, dev), s, where)
    x = torch.randn((a.sequences, 1024), device=dev).to(torch.bfloat16)
    out = block.step(x)  # once eagerly, then captured
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.step(x)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.tokens):
        block.reserve()
        graph.replay()
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / a.tokens * 1e6
    assert bool(torch.isfinite(out.float()).all())
    print(f"{a.sequences} sequences of {a.frames} frames, {'int8' if a.int8 else 'bf16'} cache: "
          f"{us:.1f} us a step, lengths {block.lens.tolist()}")
    return block, out


if __name__ == "__main__":
    main()
