"""Cases for the training-step operators that stand next to the collectives.

Four operators are measured:

  norm      y = h / sqrt(mean(h^2) + eps) * w with h = x (+ residual), the way a
            block of a language model starts; with `quant`, y in 8 bits (e4m3)
            with one scale a row or a group of columns.
  backward  the gradients of `norm`: of its input and of its weight.
  gnorm     the 2-norm of all gradients of a model together.
  clip      the gradients scaled to a mean over ranks and to at most `max_norm`.

`own` is set from outside: False computes the plain forms below with torch's
elementary operations, True calls ring_all_reduce_allreduce_amd.
"""
import math
import random

import torch

own = False

EPS = 1e-5          # under the root of the norm
CLIP_EPS = 1e-6     # beside the gradients' norm
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
DEVICE = "cuda"


def listed():
    return [
        # One token's residual stream between two blocks while serving: the smallest call, all latency.
        dict(name="norm 1x4096", op="norm", rows=1, heads=1, cols=4096, pad=0, dtype="bfloat16", weight="bfloat16",
             residual=True, quant="", group=0),
        # 8 ranks' worth of 512 tokens at width 4096, the shape of this repository's expert exchange.
        dict(name="norm 4096x4096", op="norm", rows=4096, heads=1, cols=4096, pad=0, dtype="bfloat16",
             weight="bfloat16", residual=True, quant="", group=0),
        # Queries of 32 heads of 128 inside rows of 48 heads (queries, keys and values side by side), each head
        # normed by itself: short rows with two strides, weight kept in 32 bits.
        dict(name="norm heads 2048x32x128", op="norm", rows=2048, heads=32, cols=128, pad=2048, dtype="bfloat16",
             weight="float32", residual=False, quant="", group=0),
        # An odd width in rows that are further apart than they are long: no row but the first is aligned.
        dict(name="norm odd 1021x5119", op="norm", rows=1021, heads=1, cols=5119, pad=2, dtype="float16",
             weight="float16", residual=True, quant="", group=0),
        # A small decoding batch whose next product takes 8 bits: one scale a token.
        dict(name="norm e4m3 16x4096", op="norm", rows=16, heads=1, cols=4096, pad=0, dtype="bfloat16",
             weight="bfloat16", residual=True, quant="e4m3", group=0),
        # A long prompt, wide model: scales for groups of 128 columns.
        dict(name="norm e4m3 8192x8192", op="norm", rows=8192, heads=1, cols=8192, pad=0, dtype="bfloat16",
             weight="bfloat16", residual=True, quant="e4m3", group=128),
        # Training in 32 bits at an odd size: few rows, so the weight's gradient is a sum over few workgroups.
        dict(name="backward 777x1111", op="backward", rows=777, heads=1, cols=1111, pad=0, dtype="float32",
             weight="float32", residual=True),
        # A training step of 16384 tokens at width 4096.
        dict(name="backward 16384x4096", op="backward", rows=16384, heads=1, cols=4096, pad=0, dtype="bfloat16",
             weight="bfloat16", residual=True),
        # A small model's gradients: 96 tensors of very different lengths, one of them empty, 1 M elements in all.
        dict(name="gnorm 96 tensors", op="gnorm", tensors=96, total=1 << 20, even=False, dtype="float32", ranks=4),
        # This repository's data-parallel workload: 40 buckets of 25 MiB, summed over 8 ranks.
        dict(name="gnorm 40 buckets", op="gnorm", tensors=40, total=40 * 13_107_200, even=True, dtype="bfloat16",
             ranks=8),
        # 291 tensors side by side in flat buffers, half of them 16-bit: few start on a 16-byte boundary.
        dict(name="clip 291 tensors", op="clip", tensors=291, total=40_000_003, even=False, dtype="mixed", ranks=8,
             max_norm=1.0),
        # The buckets again, clipped.
        dict(name="clip 40 buckets", op="clip", tensors=40, total=40 * 13_107_200, even=True, dtype="bfloat16",
             ranks=8, max_norm=1.0),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "backward", "backward", "gnorm", "clip"])
    if op in ("gnorm", "clip"):
        total = _spread(rng, 1 << 12, 1 << 28)
        c = dict(op=op, tensors=_spread(rng, 1, 400), total=total, even=rng.random() < 0.3,
                 dtype=rng.choice(["float32", "bfloat16", "float16", "mixed"]), ranks=rng.choice([1, 2, 4, 8, 16]))
        if op == "clip":
            c["max_norm"] = rng.choice([0.1, 1.0, 1.0, 1e6])
        return c
    cols = _spread(rng, 32, 16384)
    if rng.random() < 0.5:
        cols = -(-cols // 64) * 64
    rows = _spread(rng, 1, max(1, min(32768, (1 << 26) // cols)))
    heads = 1
    if cols <= 256 and rng.random() < 0.5:
        heads = rng.choice([2, 5, 8, 32])
        rows = max(1, rows // heads)
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    c = dict(op="norm" if op == "quant" else op, rows=rows, heads=heads, cols=cols,
             pad=rng.choice([0, 0, 1, 8, 64]), dtype=dtype, weight=rng.choice([dtype, "float32", "none"]),
             residual=rng.random() < 0.6)
    if c["op"] == "norm":
        c["quant"] = "e4m3" if op == "quant" else ""
        c["group"] = rng.choice([0, 32, 64, 128]) if op == "quant" else 0
    return c


def _sizes(case):
    """The tensors' lengths: equal ones, or lengths that spread over some orders of magnitude, one of them 0."""
    n, total = case["tensors"], case["total"]
    if case["even"]:
        return [total // n + (i < total % n) for i in range(n)]
    r = random.Random(1_000_003 * n + total)
    share = [math.exp(r.gauss(0.0, 2.0)) for _ in range(n)]
    sizes = [int(total * s / sum(share)) for s in share]
    if n > 1:
        sizes[n // 2] = 0
    sizes[0] += total - sum(sizes)
    return sizes


def _types(case):
    n = case["tensors"]
    if case["dtype"] != "mixed":
        return [getattr(torch, case["dtype"])] * n
    return [(torch.float32, torch.bfloat16)[i % 2] for i in range(n)]


def _views(flats, sizes, types):
    """The tensors, one after the other in the flat buffer of their type."""
    at, views = {t: 0 for t in flats}, []
    for n, t in zip(sizes, types):
        views.append(flats[t][at[t]:at[t] + n])
        at[t] += n
    return views


def _rows(case, gen, std=1.0):
    """A [rows, cols] or [rows, heads, cols] tensor, `pad` elements apart in memory from row to row."""
    dtype, heads, cols = getattr(torch, case["dtype"]), case["heads"], case["cols"]
    flat = torch.empty(case["rows"], heads * cols + case["pad"], device=DEVICE, dtype=dtype)
    flat.normal_(0.0, std, generator=gen)
    t = flat[:, :heads * cols]
    return t.unflatten(1, (heads, cols)) if heads > 1 else t


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("norm", "backward"):
        # An activation's columns differ in size: some are several times the others.
        s["x"] = _rows(case, gen).mul_(torch.empty(case["cols"], device=DEVICE).normal_(0.0, 0.5, generator=gen).exp_())
        s["residual"] = _rows(case, gen, 2.0) if case["residual"] else None
        s["w"] = None
        if case["weight"] != "none":
            s["w"] = torch.empty(case["cols"], device=DEVICE).normal_(1.0, 0.2, generator=gen)
            s["w"] = s["w"].to(getattr(torch, case["weight"]))
        if case["op"] == "backward":
            s["dy"] = _rows(case, gen, 1e-2)
        return s
    sizes, types = _sizes(case), _types(case)
    flats = {}
    for t in dict.fromkeys(types):
        flats[t] = torch.empty(sum(n for n, u in zip(sizes, types) if u == t), device=DEVICE, dtype=t)
        flats[t].normal_(0.0, 0.03, generator=gen)
    s["flats"] = flats
    s["grads"] = _views(flats, sizes, types)
    if case["op"] == "clip":
        s["out_flats"] = {t: torch.zeros_like(f) for t, f in flats.items()}
        s["outs"] = _views(s["out_flats"], sizes, types)
    return s


def _norm_plain(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    if s["w"] is not None:
        y = y * s["w"].float()
    out = {}
    if s["residual"] is not None:
        out["residual"] = h.to(s["x"].dtype)
    if not s["quant"]:
        out["y"] = y.to(s["x"].dtype)
        return out
    g = s["group"] or s["cols"]
    full = torch.nn.functional.pad(y, (0, -s["cols"] % g)).unflatten(-1, (-1, g))
    scales = (full.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = (full / scales.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2)[..., :s["cols"]]
    out["q"] = q.to(torch.float8_e4m3fn)
    out["scales"] = scales
    return out


def _backward_plain(s):
    h, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    g = dy if s["w"] is None else dy * s["w"].float()
    dh = r * g - h * (r.pow(3) * (g * h).mean(-1, keepdim=True))
    if s["residual"] is not None:
        dh = dh + s["residual"].float()
    out = {"dx": dh.to(s["x"].dtype)}
    if s["w"] is not None:
        out["dw"] = (dy * h * r).flatten(0, -2).sum(0).to(s["w"].dtype)
    return out


def _gnorm_plain(s):
    # Over the flat buffers, which hold the tensors without gaps: fewer and larger passes than one a tensor.
    sums = torch.stack([f.float().square().sum() for f in s["flats"].values()])
    return sums.sum().sqrt() / s["ranks"]


def _clip_plain(s):
    norm = _gnorm_plain(s)
    factor = (s["max_norm"] / (norm + CLIP_EPS)).clamp_max(1.0) / s["ranks"]
    return {"norm": norm, "grads": [(f.float() * factor).to(t) for t, f in s["flats"].items()]}


def run(s):
    if not own:
        return {"norm": _norm_plain, "backward": _backward_plain, "gnorm": _gnorm_plain, "clip": _clip_plain}[s["op"]](s)
    import ring_all_reduce_allreduce_amd as rs

    if s["op"] == "norm":
        r = rs.rms_norm(s["x"], s["w"], residual=s["residual"], eps=EPS,
                        out_dtype="float8_e4m3" if s["quant"] else None, group=s["group"])
        out = {"q": r.out, "scales": r.scales} if s["quant"] else {"y": r.out}
        if s["residual"] is not None:
            out["residual"] = r.residual
        return out
    if s["op"] == "backward":
        r = rs.rms_norm_backward(s["dy"], s["x"], s["w"], grad_residual=s["residual"], eps=EPS)
        return {"dx": r.grad_in} if s["w"] is None else {"dx": r.grad_in, "dw": r.grad_weight}
    if s["op"] == "gnorm":
        return rs.grad_norm(s["grads"], scale=1.0 / s["ranks"])
    norm = rs.clip_grads(s["grads"], s["max_norm"], outs=s["outs"], scale=1.0 / s["ranks"], eps=CLIP_EPS)
    return {"norm": norm, "grads": list(s["out_flats"].values())}


_BYTES = {"float32": 4, "bfloat16": 2, "float16": 2, "none": 0}


def work(case):
    if case["op"] in ("norm", "backward"):
        n, e, w = case["rows"] * case["heads"] * case["cols"], _BYTES[case["dtype"]], _BYTES[case["weight"]]
        if case["op"] == "backward":
            return {"bytes": n * e * (3 + case["residual"]) + 2 * case["cols"] * w, "flops": 12 * n}
        made = n * e
        if case["quant"]:
            made = n + 4 * case["rows"] * case["heads"] * (-(-case["cols"] // (case["group"] or case["cols"])))
        return {"bytes": n * e * (1 + 2 * case["residual"]) + made + case["cols"] * w, "flops": 6 * n}
    each = sum(n * torch.finfo(t).bits // 8 for n, t in zip(_sizes(case), _types(case)))
    clip = case["op"] == "clip"
    return {"bytes": each * (2 if clip else 1) + 4, "flops": case["total"] * (3 if clip else 2)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("gnorm", "clip"):
        total = sum(torch.dot(p.double(), p.double()) for f in s["flats"].values() for p in f.split(1 << 26))
        norm = torch.sqrt(total) / case["ranks"]
        if case["op"] == "gnorm":
            return norm
        top = case["max_norm"] / (float(norm) + CLIP_EPS)
        return {"norm": norm, "grads": [f.double().mul_(min(1.0, top) / case["ranks"]) for f in s["flats"].values()]}
    w = 1.0 if s["w"] is None else s["w"].double()
    x = s["x"].double()
    more = None if s["residual"] is None else s["residual"].double()
    if case["op"] == "norm":
        h = x if more is None else x + more
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["cols"] + EPS) * w
        out = {} if more is None else {"residual": h}
        if not case["quant"]:
            return {**out, "y": y}
        width = case["group"] or case["cols"]
        parts = y.split(width, -1)
        scales = torch.stack([p.abs().amax(-1) for p in parts], -1).div(E4M3_MAX).clamp_min(SCALE_MIN)
        q = torch.cat([p / scales[..., i:i + 1] for i, p in enumerate(parts)], -1)
        return {**out, "q": q, "scales": scales}
    # y = h / d * w with d = sqrt(mean(h^2) + eps): dh = (w dy - (h / d) mean(w dy h / d)) / d.
    dy = s["dy"].double()
    d = torch.sqrt((x * x).sum(-1, keepdim=True) / case["cols"] + EPS)
    unit = x / d
    dx = (w * dy - unit * (w * dy * unit).sum(-1, keepdim=True) / case["cols"]) / d
    out = {"dx": dx if more is None else dx + more}
    if s["w"] is not None:
        out["dw"] = (dy * unit).reshape(-1, case["cols"]).sum(0)
    return out
