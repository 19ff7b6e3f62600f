"""A speculative decode step on this library's operators, over one pool of cache pages, as a serving loop would run it.

A batch of prompts is cached once, a piece at a time; each then branches into several answers that share its pages.  Each
step every answer drafts a tree of tokens (random projections and distributions here, in the place of a model's), and

    pages_extend   gives each answer pages for the tree
    rope           rotary positions of queries and keys
    block_write    the tree's rows into the 8-bit cache with one scale for a block of tokens and a head
    attend_blocks  attention of each drafted token over its sequence and its line of the tree
    verify_drafts  the tokens that stand against the target's distributions, and the next one
    block_keep     the rows of those that stand to where their sequence ends
    pages_free     pages behind them back to the pool

The step is captured in a HIP graph once and replayed; lengths, tables and counts move on the device.  At the end one
answer of each prompt stays, the others' pages go back, and the pool is drawn together.
Run: python examples/speculative_decode.py [--prompts 8 --answers 4 --prompt 2000 --steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exact_top_selection_amd as ets  # noqa: E402


class SpeculativeDecoder:
    """A pool of pages, a table of sequences, and the buffers of a step."""

    def __init__(self, prompts: int, answers: int, capacity: int, pages: int, heads: int = 32, kv_heads: int = 8, dim: int = 128,
                 drafts: int = 16, vocabulary: int = 32000, page: int = 64, block: int = 32, device: str = "cuda:0", seed: int = 0):
        new = dict(device=device)
        self.g = torch.Generator(device=device).manual_seed(seed)
        self.prompts, self.rows, self.page = prompts, prompts * answers, page
        per = -(-capacity // page)
        self.capacity = per * page
        self.refs = torch.zeros(pages, dtype=torch.int32, **new)
        self.table = torch.full((self.rows, per), -1, dtype=torch.int32, **new)
        self.lens = torch.zeros(self.rows, dtype=torch.int32, **new)
        codes = lambda: torch.zeros(pages * page, kv_heads, dim, dtype=torch.uint8, **new).view(torch.float8_e4m3fn)  # noqa: E731
        scales = lambda: torch.full((pages * page // block, kv_heads), 127, dtype=torch.uint8, **new)  # noqa: E731
        self.k, self.k_scales, self.v, self.v_scales = codes(), scales(), codes(), scales()
        self.pool = [self.k, self.k_scales, self.v, self.v_scales]
        self.inv_freq = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, **new) / dim)
        # three drafted tokens hang on each node, as far as there are tokens
        mask = [1]
        for t in range(1, drafts):
            mask.append(mask[(t - 1) // 3] | 1 << t)
        self.tree = torch.tensor(mask, dtype=torch.int64, **new).expand(self.rows, -1).contiguous()
        self.depth = torch.tensor([bin(m).count("1") - 1 for m in mask], dtype=torch.int32, **new)
        self.drafts = torch.full((self.rows,), drafts, dtype=torch.int32, **new)
        # what a model would write: projections of the tree's tokens, its distributions, drafted tokens, random numbers
        bf16 = dict(dtype=torch.bfloat16, **new)
        self.q = torch.zeros(self.rows, drafts, heads, dim, **bf16)
        self.key, self.value = (torch.zeros(self.rows, drafts, kv_heads, dim, **bf16) for _ in "kv")
        self.probs = torch.zeros(self.rows, drafts, vocabulary, dtype=torch.float32, **new)
        self.tokens = torch.zeros(self.rows, drafts, dtype=torch.int32, **new)
        self.uniform = torch.zeros(self.rows, drafts, dtype=torch.float32, **new)

    def _turned(self, x: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
        return ets.rope(x.flatten(0, 1), positions.flatten(), self.inv_freq, layout="half").view(x.shape)

    def _write(self, key, value, table, first, counts) -> None:
        ets.block_write(key, self.k, self.k_scales, table, first, counts, self.page)
        ets.block_write(value, self.v, self.v_scales, table, first, counts, self.page)

    def prefill(self, length: int, piece: int = 512) -> torch.Tensor:
        """Caches prompts of up to `length` tokens in the first rows, then branches them into all rows; the last piece's result."""
        n, heads, dim = self.prompts, self.q.shape[2], self.q.shape[3]
        lens = torch.randint(length // 2 + 1, length + 1, (n,), generator=self.g, device=self.lens.device, dtype=torch.int32)
        prompts = self.table[:n]
        if int(ets.pages_extend(self.refs, prompts, lens, self.page).sum()):
            raise RuntimeError("the pool has too few pages for the prompts")
        normal = lambda h: torch.randn((n, piece, h, dim), generator=self.g, device=lens.device).to(torch.bfloat16)  # noqa: E731
        out = None
        for at in range(0, length, piece):
            first = torch.full_like(lens, at)
            positions = first[:, None] + torch.arange(piece, device=lens.device, dtype=torch.int32)
            here = (lens - at).clamp(0, piece)
            self._write(self._turned(normal(self.k.shape[1]), positions), normal(self.k.shape[1]), prompts, first, here)
            out, _ = ets.attend_blocks(self._turned(normal(heads), positions), *self.pool, prompts, torch.minimum(lens, first + piece),
                                       self.page, self.capacity, first=first)
        # answers of a prompt: its own row, and branches of it
        parents = torch.arange(n, self.rows, dtype=torch.int32, device=lens.device) % n
        _, lacking = ets.pages_fork(self.refs, prompts, lens, self.page, parents, self.pool, out=self.table[n:])
        if int(lacking.sum()):
            raise RuntimeError("the pool has too few pages for the branches")
        self.lens.copy_(lens.repeat(self.rows // n))
        return out  # a prompt's own row goes on in its last page: branches hold copies of that one

    def project(self) -> None:
        """Stands for the draft model and the target's projections and distributions."""
        for t in (self.q, self.key, self.value):
            t.copy_(torch.randn(t.shape, generator=self.g, device=t.device))
        self.probs.copy_(torch.softmax(4 * torch.randn(self.probs.shape, generator=self.g, device=self.lens.device), -1))
        # likely tokens of the parents, the next likely one for each of the three
        best = self.probs.topk(3, -1).indices
        at = torch.arange(self.tokens.shape[1] - 1, device=self.lens.device)
        self.tokens[:, 1:] = best[:, at // 3, at % 3]
        self.uniform.copy_(torch.rand(self.uniform.shape, generator=self.g, device=self.lens.device))

    def step(self):
        """One step of all answers: (attention's result, new tokens, how many of them)."""
        first, reach = self.lens, self.lens + self.drafts
        lacking = ets.pages_extend(self.refs, self.table, reach, self.page)
        positions = first[:, None] + self.depth
        self._write(self._turned(self.key, positions), self.value, self.table, first, self.drafts)
        out, _ = ets.attend_blocks(self._turned(self.q, positions), *self.pool, self.table, reach, self.page, self.capacity, first=first,
                                   tree_mask=self.tree)
        new, path, counts = ets.verify_drafts(self.probs, self.tokens, self.uniform, tree_mask=self.tree)
        for codes, scales in ((self.k, self.k_scales), (self.v, self.v_scales)):
            ets.block_keep(codes, scales, self.table, first, path, counts, self.page)
        self.tokens[:, 0] = new.gather(1, (counts - 1).long().view(-1, 1))[:, 0]
        self.lens += counts
        ets.pages_free(self.refs, self.table, self.lens, self.page)
        return out, new, counts, lacking

    def capture(self):
        """The step as a HIP graph, and its outputs."""
        kept = [t.clone() for t in (self.refs, self.table, self.lens, self.tokens, *self.pool)]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            self.step()  # warm
        torch.cuda.current_stream().wait_stream(stream)
        for t, old in zip((self.refs, self.table, self.lens, self.tokens, *self.pool), kept):
            t.copy_(old)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            held = self.step()
        return graph, held

    def finish(self) -> torch.Tensor:
        """Keeps the first answer of each prompt, lets the others go and draws the pool together; each page's new number."""
        stay = self.lens.clone()
        stay[self.prompts:] = 0
        ets.pages_free(self.refs, self.table, stay, self.page)
        self.lens.copy_(stay)
        return ets.pages_compact(self.refs, self.table, self.pool)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompts", type=int, default=8)
    ap.add_argument("--answers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=2000, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    capacity = a.prompt + 16 * (a.steps + 1)
    d = SpeculativeDecoder(a.prompts, a.answers, capacity, pages=a.prompts * a.answers * (capacity // 64 + 2))
    d.prefill(a.prompt)
    d.project()
    graph, held = d.capture()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    total, ms = 0, 0.0
    for _ in range(a.steps):
        d.project()
        begin.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        if int(held[3].sum()):
            raise RuntimeError("the pool has run out of pages")
        total, ms = total + int(held[2].sum()), ms + begin.elapsed_time(end)
    used = int((d.refs > 0).sum())
    d.finish()
    print("%d answers, %d steps: %.2f tokens a step and answer, %.0f us a step; %d pages in use, %d after"
          % (d.rows, a.steps, total / a.steps / d.rows, 1e3 * ms / a.steps, used, int((d.refs > 0).sum())))


if __name__ == "__main__":
    main()
