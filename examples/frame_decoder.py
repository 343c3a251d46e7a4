"""Generate latent frames token by token and upsample them: the decoding-step operators and
ConvTranspose together.

A small decoder-only model (random weights) answers one frame of 128 channels per stream and
step; the frames, stacked to [streams, 128, frames], are the input of the audio decoder's 1-D
upsampler (kernel 8, stride 4, padding 2). A step is, for each layer,

    rms_norm (residual, e4m3)  ->  q4_matvec: q, k, v  ->  cache_write  ->  decode_attention
    ->  q4_matvec  ->  rms_norm (residual, e4m3)  ->  q4_matvec, SiLU, q4_matvec

and is captured once into a graph: positions, lengths and slots advance on the device.

    python examples/frame_decoder.py [--streams 16] [--frames 64] [--eager]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import convt_forward_amd as C  # noqa: E402

CHANNELS = 128  # of a frame, and of the upsampler's input


class FrameDecoder:
    def __init__(self, streams: int, frames: int, width: int = 1024, layers: int = 4, heads: int = 16, kv_heads: int = 4,
                 head_dim: int = 64, page: int = 16, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim, self.page = heads, kv_heads, head_dim, page

        def weight(n, k, group=64):
            w = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
            return C.q4_quantise(w.bfloat16(), group)

        def ones():
            return torch.ones(width, device="cuda", dtype=torch.bfloat16)

        self.embed = weight(width, CHANNELS)
        self.layers = [dict(norm1=ones(), qkv=weight((heads + 2 * kv_heads) * head_dim, width), out=weight(width, heads * head_dim),
                            norm2=ones(), up=weight(4 * width, width), down=weight(width, 4 * width)) for _ in range(layers)]
        self.norm, self.head = ones(), weight(CHANNELS, width)
        # every stream has its own pages of every layer's cache, in any order
        per_stream = -(-frames // page)
        self.table = torch.randperm(streams * per_stream, generator=g, device="cuda").to(torch.int32).view(streams, per_stream)
        self.caches = [C.KVCache.new(streams * per_stream, kv_heads, page, head_dim, quantised=True) for _ in range(layers)]
        self.lengths = torch.zeros(streams, dtype=torch.int32, device="cuda")
        self.streams = torch.arange(streams, device="cuda")
        self.frame = torch.randn(streams, CHANNELS, generator=g, device="cuda").bfloat16()
        self.out = torch.empty(streams, CHANNELS, frames, device="cuda")  # the upsampler's x
        self.done = 0  # frames enqueued, known without asking the device
        self.graph = None

    def room_for(self, frames: int) -> None:
        """ValueError unless `frames` more have room: past it, indexes would leave the output and the page table."""
        if frames > self.out.shape[2] - self.done:
            raise ValueError(f"{frames} frames after {self.done}: there is room for {self.out.shape[2]}")

    def step(self) -> None:
        """Each stream's next frame, from its last one."""
        self.room_for(1)
        self.enqueue()
        self.done += 1

    def enqueue(self) -> None:
        """A step's calls, for the stream or the graph that takes them."""
        self.out.scatter_(2, self.lengths.long().view(-1, 1, 1).expand(-1, CHANNELS, 1), self.frame.float().unsqueeze(2))
        slots = C.cache_slots(self.table, self.streams, self.lengths.long(), self.page)
        self.lengths += 1
        add = C.q4_matvec(self.frame, *self.embed)
        h = torch.zeros_like(add)
        nq, nkv = self.heads, self.kv_heads
        for layer, cache in zip(self.layers, self.caches):
            y, ys, h = C.rms_norm(add, layer["norm1"], residual=h, quantise=True)
            qkv = C.q4_matvec(y, *layer["qkv"], x_scale=ys).view(-1, nq + 2 * nkv, self.head_dim)
            C.cache_write(cache, qkv[:, nq:nq + nkv], qkv[:, nq + nkv:], slots)
            att = C.decode_attention(qkv[:, :nq], cache, self.table, self.lengths)
            add = C.q4_matvec(att.flatten(1), *layer["out"])
            y, ys, h = C.rms_norm(add, layer["norm2"], residual=h, quantise=True)
            up = torch.nn.functional.silu(C.q4_matvec(y, *layer["up"], x_scale=ys))
            add = C.q4_matvec(up, *layer["down"])
        y, ys, _ = C.rms_norm(add, self.norm, residual=h, quantise=True)
        self.frame.copy_(C.q4_matvec(y, *self.head, x_scale=ys))

    def generate(self, frames: int, eager: bool = False) -> torch.Tensor:
        """The next `frames` frames; returns all so far, [streams, 128, room for frames].
        ValueError where there is no room for them; nothing is enqueued then."""
        self.room_for(frames)
        if not eager and self.graph is None and frames > 1:
            # one step outside the graph (it is a frame like any other), then the capture, which runs nothing
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.step()
            torch.cuda.current_stream().wait_stream(side)
            frames -= 1
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.enqueue()
        for _ in range(frames):
            if eager or self.graph is None:
                self.step()
            else:
                self.graph.replay()
                self.done += 1
        return self.out


def upsample(x: torch.Tensor, seed: int = 1) -> torch.Tensor:
    """The audio decoder's upsampler on the frames: [streams, 128, frames] -> [streams, 64, 4 frames]."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn(CHANNELS, 64, 8, generator=g, device="cuda") * (CHANNELS * 2) ** -0.5
    return C.conv_transpose(x, w, torch.zeros(64, device="cuda"), stride=4, padding=2)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--streams", type=int, default=16)
    ap.add_argument("--frames", type=int, default=64)
    ap.add_argument("--eager", action="store_true", help="no graph: every call from Python")
    a = ap.parse_args()
    model = FrameDecoder(a.streams, a.frames)
    warm = min(4, a.frames)
    model.generate(warm, a.eager)
    torch.cuda.synchronize()
    t = time.perf_counter()
    x = model.generate(a.frames - warm, a.eager)
    torch.cuda.synchronize()
    s = time.perf_counter() - t
    y = upsample(x)
    torch.cuda.synchronize()
    if a.frames > warm:
        print(f"{a.frames - warm} steps of {a.streams} streams: {s / (a.frames - warm) * 1e6:.1f} us a step")
    print(f"frames {tuple(x.shape)} -> {tuple(y.shape)}, finite: {bool(y.isfinite().all())}")


if __name__ == "__main__":
    main()
