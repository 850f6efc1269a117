"""The attention-step operators one after another, as a step uses them: on
streams, in captured graphs, from several threads, and in examples/serve_step.py."""
import importlib.util
import os
import threading

import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests import _attention_ref as ref
from tests._gpu import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADS, KV, DIM, PAGE = 12, 4, 128, 32


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("serve_step", os.path.join(ROOT, "examples", "serve_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Batch:
    """Sequences with a context in the cache; step() norms, turns, appends and attends one token of each."""

    def __init__(self, lengths, dtype, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.dtype, self.n = dtype, len(lengths)
        most = -(-(max(lengths) + 8) // PAGE)
        self.cache = rs.kv_cache(self.n * most, KV, PAGE, DIM)
        self.table = torch.randperm(self.n * most, generator=gen).view(self.n, most).int().cuda()
        self.freq = rs.rotary_frequencies(DIM)
        self.lengths = torch.tensor(lengths, dtype=torch.int32).cuda()
        rows = torch.empty(sum(lengths), HEADS + 2 * KV, DIM).normal_(generator=gen).to(dtype).cuda()
        self.starts = torch.tensor([sum(lengths[:i]) for i in range(self.n + 1)], dtype=torch.int32).cuda()
        at = torch.cat([torch.arange(n) for n in lengths]).cuda()
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lengths)]).cuda()
        self.context = (rows, self.slots(seq, at), at)
        self.weight = torch.empty(DIM).normal_(1.0, 0.1, generator=gen).cuda()
        self.x = torch.empty(self.n, HEADS + 2 * KV, DIM).normal_(generator=gen).to(dtype).cuda()
        self.out = torch.zeros(self.n, HEADS, DIM, dtype=dtype, device="cuda")
        self.seq = torch.arange(self.n).cuda()
        self.pos = self.lengths.long()
        self.slot = self.slots(self.seq, self.pos)
        self.all = self.lengths + 1

    def slots(self, seq, at):
        return self.table[seq, at // PAGE].long() * PAGE + at % PAGE

    def prompt(self):
        rows, slots, at = self.context
        q = rs.rotary(rows[:, :HEADS], at, self.freq)
        rs.kv_append(self.cache, rows[:, HEADS:HEADS + KV], rows[:, HEADS + KV:], slots, at, self.freq)
        return q, rs.paged_attention(q, self.cache, self.table, self.lengths, starts=self.starts)

    def step(self):
        h = rs.rms_norm(self.x[:, :HEADS + KV], self.weight).out  # queries and keys, each head by itself
        rs.rotary(h[:, :HEADS], self.pos, self.freq, out=h[:, :HEADS])
        rs.kv_append(self.cache, h[:, HEADS:], self.x[:, HEADS + KV:], self.slot, self.pos, self.freq)
        rs.paged_attention(h[:, :HEADS], self.cache, self.table, self.all, out=self.out)
        return h


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_prompt_and_step(dtype):
    """What each operator leaves, against the formulas, on what the one before it left."""
    say(f"step {dtype}")
    b = Batch([70, 1, 133], dtype)
    q, got = b.prompt()
    rows, slots, at = b.context
    k = ref.to_4_bits(ref.turn(rows[:, HEADS:HEADS + KV], at, b.freq, False).float())[0]
    v = ref.to_4_bits(rows[:, HEADS + KV:].cpu())[0]
    held = rs.kv_read(b.cache, slots, dtype=torch.float32)
    assert torch.equal(held.keys.double().cpu(), k) and torch.equal(held.values.double().cpu(), v)
    ends = b.starts.tolist()
    rel = ref.ONE_PART if dtype is torch.bfloat16 else None  # 204 rows a key head over three sequences: many
    want = ref.attention([q[i:j] for i, j in zip(ends, ends[1:])], b.cache, b.table, b.lengths, weight_rel=rel)
    for (o, _, bound, _), i, j in zip(want, ends, ends[1:]):
        ref.within(got.out[i:j], o, bound + ref.half_step(o, dtype), "prompt")
    h = b.step()
    want = ref.attention([x.unsqueeze(0) for x in h[:, :HEADS]], b.cache, b.table, b.all)
    for s, (o, _, bound, _) in enumerate(want):
        ref.within(b.out[s:s + 1], o, bound + ref.half_step(o, dtype), "step")
    held = rs.kv_read(b.cache, b.slot, dtype=torch.float32)
    assert torch.equal(held.values.double().cpu(), ref.to_4_bits(b.x[:, HEADS + KV:].cpu())[0])


def test_one_query_of_a_prompt_equals_the_single_token():
    """The last token of a prompt sees what the same token sees by itself: both are within their bounds of the formula."""
    b = Batch([90, 200], torch.float32)
    q, got = b.prompt()
    last = b.starts[1:].long() - 1
    one = rs.paged_attention(q[last], b.cache, b.table, b.lengths)
    want = ref.attention([x.unsqueeze(0) for x in q[last]], b.cache, b.table, b.lengths)
    for s, (o, _, bound, _) in enumerate(want):
        for x in (one.out[s:s + 1], got.out[last][s:s + 1]):
            ref.within(x, o, bound + ref.half_step(o, torch.float32), "last token")


def test_captured_steps_replayed():
    """Two graphs of two batches, replayed in turn with new inputs, eager steps and synchronizations between, each
    checked against an eager step on the same values."""
    pair = [Batch([1500, 37, 900, 0], torch.bfloat16, seed=1), Batch([64, 2000], torch.bfloat16, seed=2)]
    graphs = []
    for b in pair:
        b.prompt()
        b.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.step()
        graphs.append(g)
    for turn in range(4):
        say(f"replay {turn}")
        for b, g in zip(pair, graphs):
            b.x.normal_(generator=torch.Generator(device="cuda").manual_seed(turn))
            if turn % 2:
                torch.cuda.synchronize()
            b.step()
            want, cache = b.out.clone(), [t.clone() for t in b.cache]
            b.out.zero_()
            rs.kv_append(b.cache, -b.x[:, HEADS:HEADS + KV], b.x[:, :KV], b.slot)  # to be written anew
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(b.out, want)
            assert all(torch.equal(t, kept) for t, kept in zip(b.cache, cache))
        for b, g in zip(pair, graphs):  # one after the other without a wait
            g.replay()
    # longer sequences in the same graph: lengths, slots and positions are read at the replay
    for b, g in zip(pair, graphs):
        b.pos.add_(1)
        b.all.add_(1)
        b.slot.copy_(b.slots(b.seq, b.pos))
        g.replay()
        got = b.out.clone()
        b.step()
        assert torch.equal(got, b.out)


def test_streams_and_threads():
    """Each thread with its stream and batch; all at once give what they give alone."""
    batches = [Batch([700, 3, 1200], torch.bfloat16, seed=s) for s in range(4)]
    want = []
    for b in batches:
        b.prompt()
        b.step()
        want.append(b.out.clone())
        b.out.zero_()
    torch.cuda.synchronize()
    errors = []

    def work(b, s):
        try:
            with torch.cuda.stream(s):
                for _ in range(20):
                    b.step()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    streams = [torch.cuda.Stream() for _ in batches]
    threads = [threading.Thread(target=work, args=x) for x in zip(batches, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for b, w in zip(batches, want):
        assert torch.equal(b.out, w)


def test_rotary_gradient_in_a_captured_step():
    """The gradient of a turn, captured, with an eager autograd graph of the same leaf alive."""
    leaf = torch.randn(64, 4, 64, device="cuda", requires_grad=True)
    pos, freq = torch.arange(64).cuda(), rs.rotary_frequencies(64)
    alive = (leaf * 2).sum()  # an eager graph of the leaf
    g_out = torch.randn(64, 4, 64, device="cuda")
    want = rs.rotary_backward(g_out, pos, freq)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = rs.rotary(leaf.detach(), pos, freq)
        back = rs.rotary_backward(g_out, pos, freq)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(back, want) and torch.equal(y, rs.rotary(leaf.detach(), pos, freq))
    alive.backward()
    assert bool((leaf.grad == 2).all())


def test_example(ex):
    """Runs: rows and lengths as given, finite results, each sequence's pages written, on several ranks and in 16 bits."""
    prompt, steps, group, pages = ex.serve(ranks=4, steps=5, prompts=(20, 1, 33), dtype=torch.float32)
    assert prompt.shape == (54, ex.WIDTH) and len(steps) == 5 and pages.lengths == [25, 6, 38]
    assert all(bool(torch.isfinite(x).all()) for x in (prompt, *steps))
    for r in group:
        used = {p for t in pages.table for p in t}
        assert all(bool(r.cache.values[p].any()) for p in used)
    bf16, more, _, _ = ex.serve(ranks=2, steps=3, prompts=(20, 1, 33), dtype=torch.bfloat16)
    assert all(bool(torch.isfinite(x.float()).all()) for x in (bf16, *more))


def test_example_attention_against_the_formula(ex):
    """One rank's attention of a ragged prompt, on the rows and cache of the example."""
    pages = ex.Pages(12, 3, 4)
    rank = ex.Rank(1, 2, 12, torch.float32)
    counts = [20, 1, 33]
    slots = torch.tensor(pages.grow(counts)).cuda()
    pos = torch.cat([torch.arange(n) for n in counts]).cuda()
    table = torch.tensor(pages.as_rows(), dtype=torch.int32).cuda()
    n = torch.tensor(counts, dtype=torch.int32).cuda()
    starts = torch.tensor([0, 20, 21, 54], dtype=torch.int32).cuda()
    freq = rs.rotary_frequencies(ex.DIM)
    rows = torch.randn(54, ex.WIDTH, generator=torch.Generator().manual_seed(4)).cuda()
    partial = torch.empty(54, ex.WIDTH, device="cuda")
    got = rank.attend(rows, slots, pos, table, n, starts, freq, partial)
    qkv = (rows @ rank.qkv).view(54, -1, ex.DIM)
    q = rs.rotary(qkv[:, :rank.heads], pos, freq)
    want = ref.attention([q[:20], q[20:21], q[21:]], rank.cache, table, n)
    for (o, _, bound, _), i, j in zip(want, (0, 20, 21), (20, 21, 54)):
        ref.within(got[i:j], o, bound + ref.half_step(o, torch.float32), "example")
