"""Serving steps of one attention block over simulated ranks: a ragged batch of
prompts, then one token a sequence and step.

Every rank holds some of the heads, with their part of the projections and of
a paged cache in 4 bits. A step norms the residual stream, projects, turns the
queries by their positions, appends keys (turned on the way) and values to the
cache, attends over it, and projects back; the ranks' partial results are
summed with the ring all-reduce, and the next step's norm adds the sum to the
residual stream. Pages are given out as sequences grow, in whatever order they
are free. The single-token step is captured into a graph and replayed.

    python examples/serve_step.py [--ranks 4] [--steps 8] [--dtype bfloat16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_all_reduce_allreduce_amd as rs  # noqa: E402

EPS = 1e-5
WIDTH, HEADS, KV_HEADS, DIM, PAGE = 512, 16, 4, 64, 16


class Pages:
    """Which pages of the cache each sequence has, and where its next tokens go. Every rank's cache is laid out alike."""

    def __init__(self, pages: int, seqs: int, most: int):
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).tolist()
        self.table = [[] for _ in range(seqs)]
        self.lengths = [0] * seqs
        self.most = most

    def grow(self, counts) -> list:
        """Slots of `counts[b]` further tokens of each sequence, one after another."""
        slots = []
        for b, n in enumerate(counts):
            for at in range(self.lengths[b], self.lengths[b] + n):
                if at // PAGE == len(self.table[b]):
                    self.table[b].append(self.free.pop())
                slots.append(self.table[b][at // PAGE] * PAGE + at % PAGE)
            self.lengths[b] += n
        return slots

    def as_rows(self) -> list:
        return [t + [-1] * (self.most - len(t)) for t in self.table]


class Rank:
    """A rank's heads: projections with equal seeds for equal heads whatever the number of ranks, and its cache."""

    def __init__(self, rank: int, ranks: int, pages: int, dtype):
        self.heads, self.kv_heads = HEADS // ranks, KV_HEADS // ranks

        def made(what: int, first: int, count: int, *shape, std: float):
            parts = [torch.empty(shape).normal_(0.0, std, generator=torch.Generator().manual_seed(1000 * what + h))
                     for h in range(first, first + count)]
            return torch.stack(parts)

        q = made(1, rank * self.heads, self.heads, DIM, WIDTH, std=WIDTH ** -0.5)
        k = made(2, rank * self.kv_heads, self.kv_heads, DIM, WIDTH, std=WIDTH ** -0.5)
        v = made(3, rank * self.kv_heads, self.kv_heads, DIM, WIDTH, std=WIDTH ** -0.5)
        self.qkv = torch.cat([q, k, v]).flatten(0, 1).t().contiguous().to("cuda", dtype)
        out = made(4, rank * self.heads, self.heads, DIM, WIDTH, std=(HEADS * DIM) ** -0.5)
        self.out = out.flatten(0, 1).to("cuda", dtype)
        self.gain = torch.ones(WIDTH, device="cuda", dtype=dtype)
        self.cache = rs.kv_cache(pages, self.kv_heads, PAGE, DIM)

    def attend(self, rows, slots, positions, pages, lengths, starts, frequencies, partial):
        """This rank's part of the block's result for normed rows; `starts` is None where each sequence has one row."""
        qkv = (rows @ self.qkv).view(rows.shape[0], -1, DIM)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        rs.rotary(q, positions, frequencies, out=q)
        rs.kv_append(self.cache, k, v, slots, positions, frequencies)
        got = rs.paged_attention(q, self.cache, pages, lengths, starts=starts).out
        torch.mm(got.flatten(1), self.out, out=partial)
        return got


def serve(ranks: int = 4, steps: int = 8, prompts=(37, 1, 70, 16), dtype=torch.bfloat16):
    """(residual stream after the prompts, after each step, the ranks, the pages)."""
    most = -(-(max(prompts) + steps) // PAGE)
    pages = Pages(len(prompts) * most, len(prompts), most)
    group = [Rank(r, ranks, len(prompts) * most, dtype) for r in range(ranks)]
    frequencies = rs.rotary_frequencies(DIM, factor=4.0, method="ramp", trained=64)
    gen = torch.Generator().manual_seed(1)
    comm = rs.comm_init(ranks, 4)

    def index(values, kind):
        return torch.tensor(values, dtype=kind).to("cuda")

    def step(stream, last, slots, positions, table, lengths, starts):
        """All ranks' sum for `stream` (+ the last one's result), and the stream."""
        partial = [torch.empty_like(stream) for _ in group]
        total = [torch.empty_like(stream) for _ in group]
        for r, p in zip(group, partial):
            n = rs.rms_norm(stream, r.gain, residual=last, eps=EPS)
            r.attend(n.out, slots, positions, table, lengths, starts, frequencies, p)
        rs.allreduce(comm, partial, total, op="sum")
        return total[0], stream if last is None else n.residual

    try:
        counts = list(prompts)
        slots = index(pages.grow(counts), torch.int64)
        positions = index([i for n in counts for i in range(n)], torch.int64)
        ends = [0]
        for n in counts:
            ends.append(ends[-1] + n)
        x = torch.empty(ends[-1], WIDTH).normal_(generator=gen).to("cuda", dtype)
        last, stream = step(x, None, slots, positions, index(pages.as_rows(), torch.int32),
                            index(pages.lengths, torch.int32), index(ends, torch.int32))
        prompt_result = stream + last
        rows = index([e - 1 for e in ends[1:]], torch.int64)
        stream, last = stream[rows].contiguous(), last[rows].contiguous()

        # One token a sequence: what the captured step reads is refilled before each replay.
        slots, positions = index([0] * len(counts), torch.int64), index([0] * len(counts), torch.int64)
        table, lengths = index(pages.as_rows(), torch.int32), index([0] * len(counts), torch.int32)
        held = (stream, last, slots, positions, table, lengths)
        graph, results = torch.cuda.CUDAGraph(), []
        for i in range(steps):
            now = list(pages.lengths)
            slots.copy_(index(pages.grow([1] * len(counts)), torch.int64))
            positions.copy_(index(now, torch.int64))
            table.copy_(index(pages.as_rows(), torch.int32))
            lengths.copy_(index(pages.lengths, torch.int32))
            if i == 0:  # as it is, which warms the libraries up
                total, after = step(*held, None)
            elif i == 1:
                torch.cuda.synchronize()
                with torch.cuda.graph(graph):
                    total, after = step(*held, None)
                graph.replay()
            else:
                graph.replay()
            results.append((after + total).clone())
            # The next token's row is the block's result here; a model would have more layers and a vocabulary.
            stream.copy_(after)
            last.copy_(total)
        torch.cuda.synchronize()
        if (err := rs.get_async_error(comm)) != rs.SUCCESS:
            raise rs.RingsimError(err, "ringsim_allreduce")
    finally:
        rs.comm_destroy(comm)
    return prompt_result, results, group, pages


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=4, choices=(1, 2, 4))
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--dtype", default="bfloat16", choices=("bfloat16", "float32"))
    a = ap.parse_args()
    dtype = getattr(torch, a.dtype)
    prompt, results, group, pages = serve(a.ranks, a.steps, dtype=dtype)
    alone, alone_steps, _, _ = serve(1, a.steps, dtype=dtype)
    print(f"{prompt.shape[0]} prompt rows, sequences of {pages.lengths} tokens, "
          f"{sum(t.numel() for r in group for t in r.cache)} bytes of cache on {a.ranks} ranks")
    for i, (x, y) in enumerate(zip(results, alone_steps)):
        print(f"step {i}: row norm {float(x.float().norm(dim=-1).mean()):.3f}, "
              f"{float((x - y).float().norm() / y.float().norm()):.2e} off one rank's")


if __name__ == "__main__":
    main()
