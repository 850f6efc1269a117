"""The attention-step operators' formulas in 64 bits on the host, and the
error bounds their tests use. Kept apart from the kernels' ways: the cache is
read through a table of levels, values are rounded by dividing and rounding,
attention goes row by row over the positions that the row sees."""
import math

import torch

U = 2.0 ** -24  # a rounding of fp32
LEVELS = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
#: Relative error of a weight held in two or three bf16 parts (one part: half a step, 2^-8).
WEIGHT_REL = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -16, torch.float32: 2.0 ** -24}
ONE_PART = 2.0 ** -8
#: Queries are split into 8-bit parts of 4 bits and 5 each further one, from the row's largest (in [128, 256)) down. What the last part leaves of a column, relative to that largest: half its smallest step, 2^-10 * 32^-(parts-1)
#: of 128 (bf16 2 parts, fp16 3), or for fp32's 24 bits in 5 parts 8 * 32^-4 of 256.
QUERY_REL = {torch.bfloat16: 2.0 ** -22, torch.float16: 2.0 ** -27, torch.float32: 2.0 ** -24}


def half_step(want, dtype):
    f = torch.finfo(dtype)
    return want.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def turn(x, positions, frequencies, interleaved, inverse=False, scale=1.0):
    """The rotation of x [..., heads, dim] in 64 bits; positions of x's leading shape."""
    x = x.double().cpu()
    n = frequencies.numel()
    t = positions.double().cpu()[..., None, None] * frequencies.cpu()
    c, s = torch.cos(t) * scale, torch.sin(t) * scale * (-1 if inverse else 1)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = a * c - b * s, b * c + a * s
    return y


def turn_bound(x, want, positions, frequencies, interleaved, scale, dtype):
    """cos and sin in fp32 (2 ulp of their own, one rounding of the angle in half turns below 1, worth pi * 2^-24
    and pi * 2^-25, and one of the scale), two products, one addition: 8 roundings of |a| + |b| cover them."""
    n = frequencies.numel()
    x = x.double().cpu().abs()
    both = torch.zeros_like(x)
    if interleaved:
        s = x[..., 0:2 * n:2] + x[..., 1:2 * n:2]
        both[..., 0:2 * n:2] = both[..., 1:2 * n:2] = s
    else:
        both[..., :n] = both[..., n:2 * n] = x[..., :n] + x[..., n:2 * n]
    out = half_step(want, dtype)
    out[..., 2 * n:] = 0.0  # copied
    return out + 8 * U * abs(scale) * both


def to_4_bits(x):
    """(values that the cache holds for x in 64 bits, exponent bytes). x is what fp32 rounds it to."""
    w = x.double().unflatten(-1, (-1, 32))
    top = w.abs().amax(-1)
    bad = ~torch.isfinite(w).all(-1)
    m, e = torch.frexp(torch.where(bad, 0.0, top))
    e = (e - 3 + (m > 0.875).to(e.dtype)).clamp(-126, 125)
    e = torch.where(top == 0, -126, e)
    unit = torch.ldexp(torch.ones_like(top), e).unsqueeze(-1)
    u = w / unit
    step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0)).double()
    q = ((u / step).round() * step).clamp(-6, 6) * unit
    q = torch.where(bad.unsqueeze(-1), math.nan, q)
    return q.flatten(-2), torch.where(bad, 255, e + 127).to(torch.uint8)


def from_cache(cache, which):
    """[pages, heads, page_size, dim] in 64 bits."""
    codes, scales = cache[which].cpu(), cache[which + 2].cpu()
    x = torch.stack([LEVELS[(codes & 15).long()], LEVELS[(codes >> 4).long()]], -1).flatten(-2)
    unit = torch.exp2(scales.double() - 127.0).transpose(-1, -2).repeat_interleave(32, -1)
    unit = torch.where(scales.transpose(-1, -2).repeat_interleave(32, -1) == 255, math.nan, unit)
    return x * unit


def seen(length, count, i, causal, window, end):
    """Positions that token i of the last `count` sees; `end`: those from there on are left out."""
    p = length - count + i
    hi = min(end, p + 1) if causal else end
    lo = max(0, p - window + 1) if window else 0
    return lo, max(lo, hi)


def attention(q, cache, pages, lengths, causal=True, window=0, scale=None, max_length=None, weight_rel=None):
    """q: a list of [count, heads, dim] a sequence. Returns for each (out, lse, bound of out before its rounding, bound
    of lse) in 64 bits."""
    keys, values = from_cache(cache, 0), from_cache(cache, 1)
    n_pages, kv_heads, page, dim = keys.shape
    table, lengths = pages.cpu().tolist(), lengths.cpu().tolist()
    scale = dim ** -0.5 if scale is None else scale
    got = []
    for b, x in enumerate(q):
        dtype = x.dtype
        x = x.double().cpu()
        count, heads = x.shape[:2]
        length = max(0, lengths[b])
        cap = len(table[b]) * page
        if max_length is not None:
            cap = min(cap, max_length)
        end = min(length, cap)
        place = [(j, table[b][j // page], j % page) for j in range(end)]
        place = [p for p in place if 0 <= p[1] < n_pages]
        at = torch.tensor([p[0] for p in place], dtype=torch.long)
        pg = torch.tensor([p[1] for p in place], dtype=torch.long)
        off = torch.tensor([p[2] for p in place], dtype=torch.long)
        out = torch.zeros(count, heads, dim, dtype=torch.float64)
        lse = torch.full((count, heads), -math.inf, dtype=torch.float64)
        bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
        for i in range(count):
            lo, hi = seen(length, count, i, causal, window, end)
            pick = (at >= lo) & (at < hi)
            if not bool(pick.any()):
                continue
            for g in range(kv_heads):
                k, v = keys[pg[pick], g, off[pick]], values[pg[pick], g, off[pick]]
                h = slice(g * (heads // kv_heads), (g + 1) * (heads // kv_heads))
                s = x[i, h] @ k.t() * scale
                lse[i, h] = torch.logsumexp(s, -1)
                w = torch.exp(s - lse[i, h].unsqueeze(-1))
                o = w @ v
                out[i, h] = o
                # A score sums dim products of up to 5 parts, each addition off by up to 2 u of the magnitudes; the
                # exponent's argument adds 3 roundings of itself and of the reference (the reference is at most the
                # row's largest score, and at least that less 8 log 2); exp2 2 ulp.
                size = (x[i, h].abs() @ k.abs().t()) * scale
                top = s.abs().amax(-1, keepdim=True)
                most = x[i, h].abs().amax(-1, keepdim=True)
                kept = most * k.abs().sum(-1) * scale * QUERY_REL[dtype]
                rel = kept + 2 * (5 * dim + 8) * U * size + 4 * U * (s.abs() + top + 8) + 4 * U
                # Sums over n positions: each pass of 32 is one chain, then splits and waves; 2 u an addition. The
                # weights' own rounding is in both sums.
                n = int(pick.sum())
                chain = 2 * (n + 64) * U
                err = rel + (WEIGHT_REL[dtype] if weight_rel is None else weight_rel) + chain
                # Weights lie relative to a reference that is at most the row's largest score, so their sum is at least
                # 1; parts of them (up to three) below the smallest normal value, 2^-126, may become 0.
                tiny = 3 * 2.0 ** -126 * v.abs().sum(0)
                bound[i, h] = (w * err) @ v.abs() + (w * err).sum(-1, keepdim=True) * o.abs() + tiny
                lse_bound[i, h] = (w * err).sum(-1) + 4 * U * (lse[i, h].abs() + 8)
        got.append((out, lse, bound, lse_bound))
    return got


def within(got, want, bound, what):
    """Every element of `got` within `bound` of `want`; NaN and infinities in the same places."""
    got = got.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: other places are finite"
    odd = ~fine
    assert torch.equal(torch.isnan(got[odd]), torch.isnan(want[odd])), f"{what}: NaN elsewhere"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: other infinities"
    off = ((got - want).abs() - bound)[fine]
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 0.0, f"{what}: {worst} beyond the bound, {int((off > 0).sum())} of {off.numel()} elements"
