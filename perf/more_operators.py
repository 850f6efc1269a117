"""Cases for the serving-step operators: rotary positions, a paged key and value cache in 4 bits, attention over it.

Four operators are measured:

  rotary     pairs of a head's columns turned by the token's position: queries and keys, the two halves of the rotated
             part against each other or neighbouring columns, the whole head or part of it.
  backward   the gradient of `rotary`.
  append     keys (turned on the way) and values rounded to 4 bits and written into pages of a cache, and read back
             as the values that the cache then holds.
  attention  softmax attention of each sequence's last tokens over its pages of the cache: single tokens while
             decoding, several tokens a sequence, prompts.

The cache holds values of 2 exponent bits and 1 mantissa bit (e2m1), two a byte with the even column's in the low
half, and for every 32 columns of a head a power of two as an exponent byte: keys and values [pages, kv_heads, page,
dim / 2], scales [pages, kv_heads, dim / 32, page].

`own` is set from outside: False computes the plain forms below with torch's elementary operations, True calls
ring_all_reduce_allreduce_amd.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
BLOCK = 32        # columns that a scale covers
TRAINED = 8192    # positions that the frequencies were made for; a `factor` above 1 stretches them


def listed():
    return [
        # One token's 32 queries and 8 keys while decoding, at a far position: all latency.
        dict(name="rotary 1x40x128", op="rotary", batch=0, tokens=1, heads=40, dim=128, turned=128, side=8,
             interleaved=False, dtype="bfloat16", factor=8.0, index="int64"),
        # A prompt of 8192 tokens, in place where the product left it: 40 of the 48 heads of a row.
        dict(name="rotary 8192x40x128", op="rotary", batch=0, tokens=8192, heads=40, dim=128, turned=128, side=8,
             interleaved=False, dtype="bfloat16", factor=1.0, index="int64"),
        # A training step's gradient: 4 sequences of 4096 tokens, heads before tokens in memory.
        dict(name="backward 4x4096x32x128", op="backward", batch=4, tokens=4096, heads=32, dim=128, turned=128, side=0,
             interleaved=False, dtype="bfloat16", factor=1.0, index="int64"),
        # Training in 32 bits with neighbouring columns paired, 50 of 100 columns turned, odd rows.
        dict(name="backward odd 777x9x100", op="backward", batch=0, tokens=777, heads=9, dim=100, turned=50, side=1,
             interleaved=True, dtype="float32", factor=1.0, index="int32"),
        # A decoding batch's keys and values, one token a sequence.
        dict(name="append 16x8x128", op="append", tokens=16, behind=0, heads=8, dim=128, turned=128, side=32,
             interleaved=False, page=64, dtype="bfloat16", factor=8.0, index="int64"),
        # A prompt of 8192 tokens.
        dict(name="append 8192x8x128", op="append", tokens=8192, behind=0, heads=8, dim=128, turned=128, side=32,
             interleaved=False, page=64, dtype="bfloat16", factor=1.0, index="int64"),
        # Odd counts, neighbouring columns, part of the head, small pages, padding rows behind the tokens.
        dict(name="append odd 1021x3x96", op="append", tokens=1021, behind=27, heads=3, dim=96, turned=32, side=1,
             interleaved=True, page=16, dtype="float32", factor=4.0, index="int32"),
        # One sequence's next token: few heads over one context, all latency.
        dict(name="attention 1x4096", op="attention", seqs=1, new=1, ragged=False, behind=0, context=4096, even=True,
             heads=32, kv_heads=8, dim=128, page=64, dtype="bfloat16", causal=True, window=0, lse=False),
        # A decoding batch of 64 sequences of very different lengths, one of its places free.
        dict(name="attention 64x16384", op="attention", seqs=64, new=1, ragged=False, behind=0, context=16384,
             even=False, heads=32, kv_heads=8, dim=128, page=64, dtype="bfloat16", causal=True, window=0, lse=False),
        # Prompts of three sequences side by side, some with tokens in the cache from before, padding rows behind.
        dict(name="attention prompts 3x2048", op="attention", seqs=3, new=2048, ragged=True, behind=37, context=6000,
             even=False, heads=32, kv_heads=8, dim=128, page=64, dtype="bfloat16", causal=True, window=0, lse=False),
        # The last 512 tokens of a long document, whose first part is in the cache.
        dict(name="attention 512 of 32768", op="attention", seqs=1, new=512, ragged=False, behind=0, context=32768,
             even=True, heads=32, kv_heads=8, dim=128, page=64, dtype="bfloat16", causal=True, window=0, lse=True),
        # Guessed tokens to be checked, 5 a sequence, one head of keys for each of queries, a window, small pages;
        # the logarithms of the sums go out too, with which ranks join parts of a context.
        dict(name="attention odd 23x5", op="attention", seqs=23, new=5, ragged=True, behind=3, context=2999,
             even=False, heads=7, kv_heads=7, dim=64, page=16, dtype="float16", causal=True, window=1500, lse=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "backward", "append", "append", "attention", "attention", "attention"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    index = rng.choice(["int32", "int64"])
    factor = rng.choice([1.0, 1.0, 4.0, 8.0])
    interleaved = rng.random() < 0.4
    if op in ("rotary", "backward"):
        dim = rng.choice([64, 96, 128, 128, 256, 2 * _spread(rng, 4, 128)])
        turned = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        heads, batch = _spread(rng, 1, 64), rng.choice([0, 0, 1, 3])
        most = max(1, (1 << 25) // (heads * dim * max(1, batch)))
        return dict(op=op, batch=batch, tokens=_spread(rng, 1, most), heads=heads, dim=dim, turned=turned,
                    side=rng.choice([0, 1, 8]), interleaved=interleaved, dtype=dtype, factor=factor, index=index)
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        heads = _spread(rng, 1, 16)
        return dict(op=op, tokens=_spread(rng, 1, max(1, (3 << 21) // (heads * dim))), behind=rng.choice([0, 0, 5, 64]),
                    heads=heads, dim=dim, turned=rng.choice([0, dim, dim, 2 * rng.randint(1, dim // 2)]),
                    side=rng.choice([0, 1, 32]), interleaved=interleaved, page=page, dtype=dtype, factor=factor,
                    index=index)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8, 16])
    kind = rng.choice(["one", "one", "few", "prompt"])
    seqs = _spread(rng, 1, 6 if kind == "prompt" else 100)
    products = (1 << 36) // (seqs * heads * dim)  # of new tokens and context
    new = {"one": 1, "few": rng.randint(2, 9), "prompt": _spread(rng, 10, min(2048, math.isqrt(products)))}[kind]
    most = min((1 << 29) // (seqs * kv_heads * dim), products // new, 32768)
    return dict(op=op, seqs=seqs, new=new, ragged=new > 1 and rng.random() < 0.7, behind=rng.choice([0, 0, 19]),
                context=_spread(rng, max(16, new), most), even=rng.random() < 0.3, heads=heads, kv_heads=kv_heads,
                dim=dim, page=page, dtype=dtype, causal=new == 1 or rng.random() < 0.85,
                window=rng.choice([0, 0, 0, _spread(rng, 16, 4096)]), lse=rng.random() < 0.4)


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _counts(case):
    """(new tokens, tokens in the cache with them) of every sequence."""
    r = random.Random(1009 * case["seqs"] + 31 * case["new"] + case["context"])
    n, new, top = case["seqs"], case["new"], case["context"]
    fresh = [r.randint(1, new) if case["ragged"] and i else new for i in range(n)]
    lens = [top if case["even"] else f + int((top - f) * r.random()) for f in fresh]
    lens[-1] = top
    if n >= 8 and not case["even"]:
        lens[1] = 0  # a free place of the batch: its tokens see nothing
    return fresh, lens


def _frequencies(case):
    """Radians a position, slowest last. A stretched context divides the slow ones by the factor, leaves the fast
    ones (32 turns and more over the trained positions) as they are, and blends between."""
    n = case["turned"] // 2
    f = 10000.0 ** (-torch.arange(n, device=DEVICE, dtype=torch.float64) / max(n, 1))
    if case["factor"] > 1:
        keep = ((TRAINED * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / case["factor"])
    return f


def _heads(case, gen, tokens):
    """[tokens, heads, dim] (or [batch, tokens, heads, dim]) with `side` more heads between one row and the next."""
    dtype, batch = getattr(torch, case["dtype"]), case.get("batch", 0)
    if batch:  # heads before tokens in memory
        t = torch.empty(batch, case["heads"] + case["side"], tokens, case["dim"], device=DEVICE, dtype=dtype)
        return t.normal_(0.0, 1.0, generator=gen)[:, :case["heads"]].transpose(1, 2)
    t = torch.empty(tokens, case["heads"] + case["side"], case["dim"], device=DEVICE, dtype=dtype)
    return t.normal_(0.0, 1.0, generator=gen)[:, :case["heads"]]


def _empty_cache(pages, case, heads):
    """What a program keeps of pages that other sequences used before: any finite values."""
    dim, page = case["dim"], case["page"]
    made = [torch.full((pages, heads, page, dim // 2), 0x5a, device=DEVICE, dtype=torch.uint8) for _ in range(2)]
    made += [torch.full((pages, heads, dim // BLOCK, page), 125, device=DEVICE, dtype=torch.uint8) for _ in range(2)]
    return made  # keys, values, scales of the keys, scales of the values


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    s = dict(case)
    if case["op"] != "attention":
        n = case["tokens"]
        index = getattr(torch, case["index"])
        first = torch.randint(0, max(1, int(TRAINED * case["factor"]) - n), (), device=DEVICE, generator=gen)
        s["positions"] = (torch.arange(n, device=DEVICE) + first).to(index)
        s["freqs"] = _frequencies(case)
    if case["op"] in ("rotary", "backward"):
        s["x"] = _heads(case, gen, case["tokens"])
        return s
    if case["op"] == "append":
        rows = case["tokens"] + case["behind"]
        s["k"], s["v"] = _heads(case, gen, rows), _heads(case, gen, rows)
        # A key's columns differ in size: some are several times the others.
        s["k"].mul_(torch.empty(case["dim"], device=DEVICE).normal_(0.0, 0.7, generator=gen).exp_())
        pages = -(-case["tokens"] // case["page"]) + 2
        s["cache"] = _empty_cache(pages, case, case["heads"])
        # Tokens of one sequence after another, its pages anywhere in the cache, the first one begun.
        table = torch.randperm(pages, device=DEVICE, generator=gen)
        at = torch.arange(case["tokens"], device=DEVICE) + case["page"] // 2
        slots = table[at // case["page"]] * case["page"] + at % case["page"]
        behind = torch.full((case["behind"],), -1, device=DEVICE, dtype=slots.dtype)
        s["slots"] = torch.cat([slots, behind]).to(index)
        s["positions"] = torch.cat([s["positions"], s["positions"].new_zeros(case["behind"])])
        return s
    fresh, lens = _counts(case)
    page, dim = case["page"], case["dim"]
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 3
    s["cache"] = _empty_cache(pages, case, case["kv_heads"])
    widths = torch.empty(2, case["kv_heads"], 1, dim, device=DEVICE).normal_(0.0, 0.5, generator=gen).exp_()
    some = max(1, (1 << 25) // (case["kv_heads"] * page * dim))
    for at in range(0, pages, some):
        for i in range(2):
            x = torch.empty(min(some, pages - at), case["kv_heads"], page, dim, device=DEVICE)
            codes, scales = _to_4_bits(x.normal_(0.0, 1.0, generator=gen).mul_(widths[i]))
            s["cache"][i][at:at + some] = codes
            s["cache"][i + 2][at:at + some] = scales.transpose(-1, -2)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).tolist()
    table, at = [], 0
    for n in used:
        table.append(order[at:at + n] + [-1] * (max(used) - n))
        at += n
    s["pages"] = torch.tensor(table, device=DEVICE, dtype=torch.int32)
    s["lengths"] = torch.tensor(lens, device=DEVICE, dtype=torch.int32)
    dtype = getattr(torch, case["dtype"])
    if case["ragged"]:
        ends = [0]
        for n in fresh:
            ends.append(ends[-1] + n)
        s["starts"] = torch.tensor(ends, device=DEVICE, dtype=torch.int32)
        rows = ends[-1] + case["behind"]
        q = torch.empty(rows, case["heads"], dim, device=DEVICE, dtype=dtype)
    else:
        s["starts"] = None
        q = torch.empty(case["seqs"], case["new"], case["heads"], dim, device=DEVICE, dtype=dtype)
    s["q"] = q.normal_(0.0, 1.5, generator=gen)
    # Rows behind the last sequence stay as they are.
    s["out"] = torch.zeros_like(q)
    s["sums"] = torch.zeros(q.shape[:-1], device=DEVICE) if case["lse"] else None
    return s


# ---- plain forms ----------------------------------------------------------------------------------------------------

def _turn(x, positions, freqs, interleaved, back=False):
    """The rotation in the type of `x`; angles in 64 bits."""
    angle = positions.double().unsqueeze(-1) * freqs
    cos, sin = torch.cos(angle).to(x.dtype).unsqueeze(-2), torch.sin(angle).to(x.dtype).unsqueeze(-2)
    if back:
        sin = -sin
    n = freqs.numel()
    head = x[..., :2 * n]
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., :n], head[..., n:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _to_4_bits(x):
    """(codes, two a byte, and exponent bytes) of fp32 `x`: the smallest power of two that takes the block's largest
    magnitude to at most 7, from where every value is within half a step of its code."""
    w = x.unflatten(-1, (-1, BLOCK))
    top = w.abs().amax(-1).view(torch.int32)
    byte = (((top + 0x1fffff) >> 23) - 2).clamp_min(1)
    u = w.abs() / (byte << 23).view(torch.float32).unsqueeze(-1)
    code = ((u > 0.25).to(torch.uint8) + (u >= 0.75) + (u > 1.25) + (u >= 1.75) + (u > 2.5) + (u >= 3.5) + (u > 5.0)
            + 8 * torch.signbit(w).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, byte.to(torch.uint8)


def _from_4_bits(codes, scales):
    """fp32 values of packed codes [..., dim / 2] with exponent bytes [..., dim / 32]."""
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    levels = torch.cat([levels, -levels])
    x = torch.stack([levels[(codes & 15).int()], levels[(codes >> 4).int()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, BLOCK)) * (scales.int() << 23).view(torch.float32).unsqueeze(-1)).flatten(-2)


def _rotary_plain(s):
    return _turn(s["x"].float(), s["positions"], s["freqs"], s["interleaved"], s["op"] == "backward").to(s["x"].dtype)


def _append_plain(s):
    n = s["tokens"]
    slots = s["slots"][:n].long()
    page, off = slots // s["page"], slots % s["page"]
    # Turned in 64 bits: a last bit may decide between two codes.
    k = _turn(s["k"][:n].double(), s["positions"][:n], s["freqs"], s["interleaved"]).float()
    got = {}
    for i, x, name in ((0, k, "keys"), (1, s["v"][:n].float(), "values")):
        codes, scales = _to_4_bits(x)
        s["cache"][i][page, :, off] = codes
        s["cache"][i + 2][page, :, :, off] = scales
        got[name] = torch.zeros(s["k"].shape, device=DEVICE, dtype=torch.bfloat16)
        got[name][:n] = _from_4_bits(s["cache"][i][page, :, off], s["cache"][i + 2][page, :, :, off])
    return got


def _rows_of(s):
    """Rows of q that belong to each sequence [seqs, new], and how many count."""
    new, seqs = s["new"], s["seqs"]
    i = torch.arange(new, device=DEVICE)
    if s["starts"] is None:
        return i + new * torch.arange(seqs, device=DEVICE).unsqueeze(1), s["lengths"].new_full((seqs,), new)
    starts = s["starts"].long()
    counts = starts[1:] - starts[:-1]
    return torch.minimum(starts[:-1, None] + i, starts[1:, None] - 1), counts


def _attention_plain(s):
    H, G, dim = s["kv_heads"], s["heads"] // s["kv_heads"], s["dim"]
    q = s["q"].reshape(-1, s["heads"], dim)
    rows, counts = _rows_of(s)
    pages = s["pages"].long().clamp_min(0)
    kv = [_from_4_bits(s["cache"][i][pages], s["cache"][i + 2][pages].transpose(-1, -2)).transpose(1, 2).flatten(2, 3)
          for i in range(2)]  # [seqs, kv_heads, tokens, dim]
    qs = q[rows].float().unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [seqs, kv_heads, new * G, dim]
    score = torch.matmul(qs, kv[0].transpose(-1, -2)) * dim ** -0.5
    j = torch.arange(kv[0].shape[2], device=DEVICE)
    at = (s["lengths"] - counts).unsqueeze(1) + torch.arange(s["new"], device=DEVICE)  # positions [seqs, new]
    seen = (j < s["lengths"].view(-1, 1, 1)).expand(-1, s["new"], -1)
    if s["causal"]:
        seen = seen & (j <= at.unsqueeze(-1))
    if s["window"]:
        seen = seen & (j > at.unsqueeze(-1) - s["window"])
    score = score.unflatten(2, (s["new"], G)).masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[1]) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + top  # minus infinity where nothing is seen
    # Back to rows of q; places past a sequence's count write nothing.
    o, lse = (t.unflatten(2, (s["new"], G)).permute(0, 2, 1, 3, 4).flatten(2, 3) for t in (o, lse))
    real = torch.arange(s["new"], device=DEVICE) < counts.unsqueeze(1)
    to = torch.where(real, rows, q.shape[0]).flatten()
    out = torch.zeros(q.shape[0] + 1, s["heads"], dim, device=DEVICE, dtype=q.dtype)
    out[to] = o.flatten(0, 1).to(q.dtype)
    got = {"out": out[:-1].view(s["q"].shape)}
    if s["lse"]:
        sums = torch.zeros(q.shape[0] + 1, s["heads"], device=DEVICE)
        sums[to] = lse.flatten(0, 1).squeeze(-1)
        got["lse"] = sums[:-1].view(s["q"].shape[:-1])
    return got


def run(s):
    if not own:
        return {"rotary": _rotary_plain, "backward": _rotary_plain, "append": _append_plain,
                "attention": _attention_plain}[s["op"]](s)
    import ring_all_reduce_allreduce_amd as rs

    if s["op"] == "rotary":
        return rs.rotary(s["x"], s["positions"], s["freqs"], interleaved=s["interleaved"])
    if s["op"] == "backward":
        return rs.rotary_backward(s["x"], s["positions"], s["freqs"], interleaved=s["interleaved"])
    cache = rs.KvCache(*s["cache"])
    if s["op"] == "append":
        rs.kv_append(cache, s["k"], s["v"], s["slots"], s["positions"], s["freqs"], interleaved=s["interleaved"])
        keys, values = rs.kv_read(cache, s["slots"], dtype=torch.bfloat16)
        return {"keys": keys, "values": values}
    rs.paged_attention(s["q"], cache, s["pages"], s["lengths"], starts=s["starts"], causal=s["causal"],
                       window=s["window"], max_length=s["context"], out=s["out"], lse=s["sums"])
    return {"out": s["out"], "lse": s["sums"]} if s["lse"] else {"out": s["out"]}


# ---- work and exact values ------------------------------------------------------------------------------------------

_BYTES = {"float32": 4, "bfloat16": 2, "float16": 2, "int32": 4, "int64": 8}


def _seen(case, fresh, length):
    """(pairs of a token and one that it sees, cached tokens that any of them sees) of one sequence."""
    pairs, low, high = 0, length, 0
    for i in range(fresh):
        at = length - fresh + i
        end = min(length, at + 1) if case["causal"] else length
        begin = max(0, at - case["window"] + 1) if case["window"] else 0
        if end > begin:
            pairs += end - begin
            low, high = min(low, begin), max(high, end)
    return pairs, max(0, high - low)


def work(case):
    dim, heads = case["dim"], case["heads"]
    e = _BYTES[case["dtype"]]
    if case["op"] == "attention":
        fresh, lens = _counts(case)
        seen = [_seen(case, f, n) for f, n in zip(fresh, lens)]
        cached = sum(t for _, t in seen) * case["kv_heads"] * 2 * (dim // 2 + dim // BLOCK)
        rows = sum(fresh) * heads
        return {"bytes": cached + rows * (2 * dim * e + 4 * case["lse"]) + 4 * case["seqs"],
                "flops": 4 * dim * heads * sum(p for p, _ in seen)}
    n = case["tokens"] * max(1, case.get("batch", 0)) * heads * dim
    steer = case["tokens"] * _BYTES[case["index"]] + 4 * case["turned"]
    if case["op"] == "append":
        # k and v in, codes and scales out, and read again for the values in 16 bits.
        packed = 2 * (n // 2 + n // BLOCK)
        return {"bytes": 2 * n * e + 2 * packed + 2 * n * 2 + 3 * steer, "flops": 8 * n}
    return {"bytes": 2 * n * e + steer, "flops": 3 * n}


def _exact_turn(x, positions, freqs, interleaved, back):
    """Pairs as complex numbers, multiplied with exp(i * angle)."""
    n = freqs.numel()
    angle = positions.double()[:, None, None] * freqs
    z = torch.polar(torch.ones_like(angle), -angle if back else angle)
    y = x.double().clone(memory_format=torch.contiguous_format)
    part = y[..., :2 * n]
    part = part.unflatten(-1, (n, 2)) if interleaved else part.unflatten(-1, (2, n)).transpose(-1, -2)
    part.copy_(torch.view_as_real(torch.complex(part[..., 0], part[..., 1]) * z))  # a view of y
    return y


def _exact_4_bits(x):
    """Each value of `x` as the nearest that 4 bits hold, with one power of two for 32 of them; ties to even codes."""
    w = x.unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(w.abs().amax(-1, keepdim=True))  # the largest is m * 2^e, m in [1/2, 1)
    unit = torch.ldexp(torch.ones_like(m), torch.clamp(e - 3 + (m > 0.875).to(e.dtype), min=-126))
    u = w / unit
    size = u.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0)).to(u.dtype)
    return ((u / step).round() * step).clamp(-6.0, 6.0).mul(unit).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rotary", "backward"):
        return _exact_turn(s["x"], s["positions"], s["freqs"], s["interleaved"], case["op"] == "backward")
    if case["op"] == "append":
        n = case["tokens"]
        k = _exact_turn(s["k"][:n], s["positions"][:n], s["freqs"], s["interleaved"], False)
        got = {"keys": torch.zeros(s["k"].shape, device=DEVICE, dtype=torch.float64)}
        got["values"] = torch.zeros_like(got["keys"])
        got["keys"][:n] = _exact_4_bits(k)
        got["values"][:n] = _exact_4_bits(s["v"][:n].double())
        return got
    fresh, lens = _counts(case)
    dim, heads = case["dim"], case["heads"]
    q = s["q"].reshape(-1, heads, dim)
    out = torch.zeros(q.shape, device=DEVICE, dtype=torch.float64)
    lse = torch.zeros(q.shape[:2], device=DEVICE, dtype=torch.float64)
    levels = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=DEVICE,
                          dtype=torch.float64)
    row = 0
    for b, (n, length) in enumerate(zip(fresh, lens)):
        mine = slice(row, row + n)
        row += n
        if length == 0:
            lse[mine] = -math.inf
            continue
        at = torch.arange(length, device=DEVICE)
        page, off = s["pages"][b].long()[at // case["page"]], at % case["page"]
        i = torch.arange(length - n, length, device=DEVICE).unsqueeze(1)
        hidden = torch.zeros(n, length, device=DEVICE, dtype=torch.bool)
        if case["causal"]:
            hidden |= at > i
        if case["window"]:
            hidden |= at <= i - case["window"]
        for h in range(heads):
            g = h // (heads // case["kv_heads"])
            kv = []
            for c in range(2):
                byte = s["cache"][c][page, g, off]
                x = torch.empty(length, dim, device=DEVICE, dtype=torch.float64)
                x[:, 0::2], x[:, 1::2] = levels[(byte % 16).long()], levels[(byte // 16).long()]
                power = torch.exp2(s["cache"][c + 2][page, g, :, off].double() - 127.0)
                kv.append(x * power.repeat_interleave(BLOCK, -1))
            score = (q[mine, h].double() @ kv[0].t()) / math.sqrt(dim)
            score.masked_fill_(hidden, -math.inf)
            sums = torch.logsumexp(score, -1)
            p = torch.exp(score - sums.unsqueeze(-1)).masked_fill_(torch.isneginf(sums).unsqueeze(-1), 0.0)
            out[mine, h] = p @ kv[1]
            lse[mine, h] = sums
    got = {"out": out.view(s["q"].shape)}
    if case["lse"]:
        got["lse"] = lse.view(s["q"].shape[:-1])
    return got
