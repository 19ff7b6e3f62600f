"""A sparse decode step on this library's operators, as a serving loop would run it.

For each sequence of a batch, its next token's queries and latent key (random here, in the place of a model's
projections) go through

    rope          rotary positions of the queries and of the key's last channels
    cache_write   the new token's rows into the 8-bit attention cache and the 8-bit index cache
    index_scores  scores of all cached positions
    topk_paged    the slots of the k best
    attend        attention over those slots, one latent head shared by all query heads

The step is captured in a HIP graph once and replayed for every token; lengths, positions and slots move on the device.
Run: python examples/sparse_decode.py [--batch 64 --context 32768 --steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exact_top_selection_amd as ets  # noqa: E402

LATENT, ROTATED, INDEX = 512, 64, 128  # channels: the latent part of a key, its rotated part, an index key


class SparseDecoder:
    """Caches, tables and buffers of a batch of sequences of up to `context` tokens."""

    def __init__(self, batch: int, context: int, k: int, heads: int = 128, index_heads: int = 64, page: int = 64,
                 device: str = "cuda:0", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        pages = -(-context // page)
        slots, blocks = batch * pages * page, (LATENT + ROTATED) // 32
        self.batch, self.context, self.page, self.g = batch, pages * page, page, g
        new = dict(device=device)
        self.table = torch.randperm(batch * pages, generator=g, **new).to(torch.int32).view(batch, pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, **new)
        self.codes = torch.zeros(slots, 1, LATENT + ROTATED, dtype=torch.uint8, **new).view(torch.float8_e4m3fn)
        self.scales = torch.full((slots, 1, blocks), 127, dtype=torch.uint8, **new)
        self.index_codes = torch.zeros(slots, 1, INDEX, dtype=torch.uint8, **new).view(torch.float8_e4m3fn)
        self.index_scales = torch.full((slots, 1, INDEX // 32), 127, dtype=torch.uint8, **new)
        self.inv_freq = 10000.0 ** (-torch.arange(0, ROTATED, 2, dtype=torch.float64, **new) / ROTATED)
        bf16 = dict(dtype=torch.bfloat16, **new)
        # a token's projections, which a model would write here
        self.q = torch.zeros(batch, heads, LATENT + ROTATED, **bf16)
        self.key = torch.zeros(batch, 1, LATENT + ROTATED, **bf16)
        self.index_q = torch.zeros(batch, index_heads, INDEX, **bf16)
        self.index_key = torch.zeros(batch, 1, INDEX, **bf16)
        self.index_weights = torch.zeros(batch, 1, index_heads, dtype=torch.float32, **new)
        self.scores = torch.empty(batch, self.context, dtype=torch.float32, **new)
        self.chosen = torch.empty(batch, k, dtype=torch.int32, **new)
        self.workspace = ets.new_workspace(batch, self.context, k, self.lens.device)

    def project(self) -> None:
        """Stands for the model's projections of the next token."""
        for t in (self.q, self.key, self.index_q, self.index_key):
            t.copy_(torch.randn(t.shape, generator=self.g, device=t.device))
        self.index_weights.uniform_(0, 1, generator=self.g)

    def prefill(self, tokens: int) -> None:
        """Fills the caches with `tokens` random tokens a sequence."""
        for at in range(0, tokens, 1024):
            n = min(1024, tokens - at)
            pos = torch.arange(at, at + n, device=self.lens.device)
            slots = (self.table[:, pos // self.page] * self.page + (pos % self.page).to(torch.int32)).reshape(-1)
            for codes, scales in ((self.codes, self.scales), (self.index_codes, self.index_scales)):
                x = torch.randn(self.batch * n, 1, codes.shape[2], generator=self.g, device=pos.device)
                ets.cache_write(x, slots, codes, scales)
        self.lens.fill_(tokens)

    def step(self):
        """One token for every sequence; (out [batch, heads, LATENT], lse)."""
        pos = self.lens.clone()
        page = torch.div(pos, self.page, rounding_mode="floor")
        slots = self.table.gather(1, page.long()[:, None])[:, 0] * self.page + (pos - page * self.page)
        q = ets.rope(self.q, pos, self.inv_freq, offset=LATENT)
        key = ets.rope(self.key, pos, self.inv_freq, offset=LATENT)
        ets.cache_write(key, slots, self.codes, self.scales)
        ets.cache_write(self.index_key, slots, self.index_codes, self.index_scales)
        self.lens += 1
        ets.index_scores(self.index_q[:, None], self.index_weights, self.index_codes, self.index_scales, self.table, self.lens,
                         self.page, self.context, out=self.scores)
        ets.topk_paged(self.scores, self.lens, self.table, self.chosen, self.page, workspace=self.workspace)
        out, lse = ets.attend_selected(q[:, None], self.codes, self.scales, self.codes[..., :LATENT],
                                       self.scales[..., :LATENT // 32], self.chosen[:, None])
        return out[:, 0], lse[:, 0]

    def capture(self):
        """The step as a graph, and the outputs that its replays fill; lengths are as before."""
        before = self.lens.clone()
        self.step()  # outside the graph first: the library loads its kernels
        self.lens.copy_(before)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            with torch.cuda.graph(graph, stream=stream):
                held = self.step()
        torch.cuda.current_stream().wait_stream(stream)
        self.lens.copy_(before)
        return graph, held


def main(batch: int = 64, context: int = 32768, k: int = 2048, steps: int = 20) -> float:
    """Decodes `steps` tokens behind a prompt that leaves room for them; microseconds a step."""
    decoder = SparseDecoder(batch, context, k)
    decoder.prefill(context - steps)
    decoder.project()
    graph, _ = decoder.capture()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) / steps * 1e3
    print("%d sequences, %d positions, %d selected: %.1f us a step" % (batch, context, k, us), flush=True)
    return us


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    parser.add_argument("--batch", type=int, default=64)
    parser.add_argument("--context", type=int, default=32768)
    parser.add_argument("--k", type=int, default=2048)
    parser.add_argument("--steps", type=int, default=20)
    main(**vars(parser.parse_args()))
