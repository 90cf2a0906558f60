"""A video transformer's self-attention, generated frame by frame: quantized projections, rotary
positions over (time, height, width), an 8-bit key/value cache of the frames so far, and attention
over it.  Each step takes the tokens of some new frames; every token sees its own and earlier frames.

    python examples/streaming_video_attention.py                # 1536 wide, 12 heads, 21 frames of 30 x 52 tokens
    python examples/streaming_video_attention.py --frames 6 --chunk 2 --height 8 --width 12

Weights and activations are random (this repository has no trained ones); the sizes are those of the
video layers in workloads/.  The normalisation of q and k that such layers have before the rotary
positions is left out (video_transformer_block.py has it, in the append).
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import calibration_free_w4a4_amd as orbq  # noqa: E402
import workloads  # noqa: E402


class StreamingAttention:
    """One layer for one sequence: d = heads * head_dim, W4A4 projections, int8 cache for up to max_tokens."""

    def __init__(self, d: int, heads: int, max_tokens: int, tokens_per_frame: int, dims=(44, 42, 42), block: int = 128,
                 bits: int = 4, page_tokens: int = 64, seed: int = 7):
        dev = torch.device("cuda", torch.cuda.current_device())
        self.d, self.heads, self.hd, self.frame = d, heads, d // heads, tokens_per_frame
        perm, signs = workloads.rotation(d)
        self.rot = orbq.Rotation.create(d, block, perm, signs)
        self.cb = orbq.Codebook.lloyd_max(d, bits)
        weights = lambda m, s: torch.from_numpy(workloads.weights(m, d, s).view(np.int16)).view(torch.bfloat16).to(dev)  # noqa: E731
        self.qkv = orbq.fold_weights(weights(3 * d, seed), self.rot, self.cb)
        self.out = orbq.fold_weights(weights(d, seed + 1), self.rot, self.cb)
        self.rope = orbq.Rope.create(dims)
        pages = (max_tokens + page_tokens - 1) // page_tokens
        self.cache = orbq.KVCache.create(pages, heads, self.hd, page_tokens)
        self.table = torch.arange(pages, dtype=torch.int32, device=dev)[None]
        self.held = torch.zeros(1, dtype=torch.int32, device=dev)   # on the GPU: a step never waits for the host

    def step(self, x, positions):
        """x bf16 [n, d], the tokens of whole frames in order; positions float32 [n, 3]."""
        n = x.shape[0]
        qkv = orbq.linear(x, self.rot, self.cb, *self.qkv, self.cb, out_dtype=torch.bfloat16).view(n, 3, self.heads, self.hd)
        q, k, v = qkv.unbind(1)                                      # parts of one tensor: nothing is copied
        orbq.rope(self.rope, positions, q, k, out=(q, k))
        orbq.kv_append(self.cache, k, v, self.table, self.held)
        self.held += n
        o = orbq.kv_attention(self.cache, q, self.table, self.held, causal_block=self.frame)
        return orbq.linear(o.view(n, self.d), self.rot, self.cb, *self.out, self.cb, out_dtype=torch.bfloat16)


def grid_positions(frames: range, height: int, width: int, device="cuda"):
    """(time, height, width) of each token of some frames, float32 [tokens, 3]."""
    return torch.cartesian_prod(torch.arange(frames.start, frames.stop, dtype=torch.float32, device=device),
                                torch.arange(height, dtype=torch.float32, device=device),
                                torch.arange(width, dtype=torch.float32, device=device)).reshape(-1, 3)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--width-d", type=int, default=1536, help="model width")
    ap.add_argument("--heads", type=int, default=12)
    ap.add_argument("--frames", type=int, default=21)
    ap.add_argument("--chunk", type=int, default=3, help="frames a step")
    ap.add_argument("--height", type=int, default=30)
    ap.add_argument("--width", type=int, default=52)
    a = ap.parse_args()
    frame = a.height * a.width
    layer = StreamingAttention(a.width_d, a.heads, a.frames * frame, frame)
    gen = torch.Generator(device="cuda").manual_seed(0)
    for f in range(0, a.frames, a.chunk):
        frames = range(f, min(f + a.chunk, a.frames))
        x = torch.randn((len(frames) * frame, a.width_d), generator=gen, device="cuda").bfloat16()
        pos = grid_positions(frames, a.height, a.width)
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = layer.step(x, pos)
        torch.cuda.synchronize()
        print(f"frames {frames.start}-{frames.stop - 1}: {x.shape[0]} tokens over {frames.stop * frame} cached, "
              f"{(time.perf_counter() - t) * 1e3:.2f} ms, |y| {y.float().norm().item():.4g}", flush=True)


if __name__ == "__main__":
    main()
