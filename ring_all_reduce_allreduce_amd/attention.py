"""Attention-step operators: what a rank runs between the norm in front of its
projections and the all-reduce behind them.

The calls of the C ABI in ``include/ringsim_attention.h``, which defines what
every one of them computes:

    rotary(x, positions, frequencies, *, interleaved=False, scale=1.0, ...) -> tensor
    rotary_backward(grad_out, positions, frequencies, *, interleaved=False, scale=1.0, ...) -> tensor
    rotary_frequencies(columns, *, base=10000.0, ...) -> float64 tensor
    kv_cache(pages, heads, page_size, dim) -> KvCache(keys, values, key_scales, value_scales)
    kv_append(cache, k, v, slots, positions=None, frequencies=None, ...)
    kv_read(cache, slots, *, dtype=torch.bfloat16, ...) -> KvValues(keys, values)
    paged_attention(q, cache, pages, lengths, *, starts=None, causal=True, window=0, ...) -> Attention(out, lse)

What holds for the step operators (:mod:`.operators`) holds here: device
tensors of the current device; calls asynchronous on ``stream`` (default: the
current torch stream), from whose memory results and workspaces come; nothing
recorded for autograd; written tensors advance their version; wrong arguments
raise TypeError or ValueError before anything is enqueued, codes of the
library RingsimError.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from .operators import _b, _on

KV_BLOCK = 32
KV_DIMS = (64, 96, 128, 192, 256)
_VALUE_TYPES = {torch.float32: 2, torch.bfloat16: 3, torch.float16: 16}


class KvCache(NamedTuple):
    """A paged cache of keys and values in 4 bits, as uint8 tensors: ``keys``
    and ``values`` of shape (pages, heads, page_size, dim / 2), and for every
    32 columns an exponent byte in ``key_scales`` and ``value_scales`` of shape
    (pages, heads, dim / 32, page_size). Pages and heads may be apart in memory
    (multiples of 16 bytes), as where a program holds the caches of all layers
    in one tensor; the last two dimensions are contiguous."""

    keys: torch.Tensor
    values: torch.Tensor
    key_scales: torch.Tensor
    value_scales: torch.Tensor


class KvValues(NamedTuple):
    keys: torch.Tensor
    values: torch.Tensor


class Attention(NamedTuple):
    """``lse``: the logarithm of each row's sum of weights, with which outputs
    over parts of a context are joined; None where it was not wanted."""

    out: torch.Tensor
    lse: torch.Tensor | None


def rotary_frequencies(columns: int, *, base: float = 10000.0, factor: float = 1.0, method: str = "linear",
                       trained: int | None = None, low: float = 1.0, high: float = 32.0, device="cuda") -> torch.Tensor:
    """Radians a position of ``columns`` / 2 pairs, base^(-2 i / columns), as a
    float64 tensor; stretched by ``factor`` for contexts longer than the
    ``trained`` one:

    ``"linear"``  every frequency divided by the factor;
    ``"base"``    the base raised so that the slowest pair is divided by the
                  factor and the fastest one kept;
    ``"ramp"``    pairs that make ``high`` turns and more over the trained
                  context kept, those of ``low`` turns and fewer divided by the
                  factor, between them a blend linear in the turns."""
    if columns < 0 or columns % 2:
        raise ValueError("columns must be even and not negative")
    if not (factor > 0 and math.isfinite(factor) and base > 0 and math.isfinite(base)):
        raise ValueError("factor and base must be above 0")
    if method not in ("linear", "base", "ramp"):
        raise ValueError(f"unknown method {method!r}")
    i = torch.arange(columns // 2, dtype=torch.float64)
    if method == "base" and columns > 2:
        base = base * factor ** (columns / (columns - 2))
    f = torch.tensor(base, dtype=torch.float64) ** (-2.0 * i / max(columns, 1))
    if method == "linear":
        f = f / factor
    elif method == "ramp":
        if trained is None or trained < 1 or not high > low:
            raise ValueError("a ramp needs the trained context and low below high")
        keep = ((trained * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f.to(device)


def rotary(x, positions, frequencies, *, interleaved: bool = False, scale: float = 1.0, out=None, stream=None):
    """Turns the first 2 * len(frequencies) columns of every head of ``x`` by
    the token's position; the others are copied.

    ``x``: (tokens, heads, dim) or (outer, inner, heads, dim) of float32,
    bfloat16 or float16, any strides but a contiguous last dimension, so a view
    of queries and keys inside wider rows, or of heads that lie before tokens.
    ``positions``: int32 or int64, one a token, or (inner,) for all of the
    outer dimension. ``frequencies``: float64, in radians a position. Column i
    goes with column i + len(frequencies), or 2 i with 2 i + 1 if
    ``interleaved``. ``scale`` multiplies the turned columns. ``out`` may be
    ``x`` itself."""
    if stream is not None:
        with _on(stream):
            return _b.rotary(x, positions, frequencies, interleaved, False, scale, out)
    return _b.rotary(x, positions, frequencies, interleaved, False, scale, out)


def rotary_backward(grad_out, positions, frequencies, *, interleaved: bool = False, scale: float = 1.0, grad_in=None,
                    stream=None):
    """Gradient of :func:`rotary`: ``grad_out`` turned back. ``grad_in`` may be
    ``grad_out`` itself."""
    if stream is not None:
        with _on(stream):
            return _b.rotary(grad_out, positions, frequencies, interleaved, True, scale, grad_in)
    return _b.rotary(grad_out, positions, frequencies, interleaved, True, scale, grad_in)


def kv_cache(pages: int, heads: int, page_size: int, dim: int, *, device="cuda") -> KvCache:
    """A cache of zeros. ``page_size``: a power of two from 16 to 1024;
    ``dim``: one of 64, 96, 128, 192, 256."""
    if dim not in KV_DIMS:
        raise ValueError(f"dim must be one of {KV_DIMS}, not {dim}")
    if page_size < 16 or page_size > 1024 or page_size & (page_size - 1):
        raise ValueError(f"page_size must be a power of two from 16 to 1024, not {page_size}")
    if pages < 1 or heads < 1:
        raise ValueError("a cache has at least one page and one head")
    data = [torch.zeros(pages, heads, page_size, dim // 2, dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.full((pages, heads, dim // KV_BLOCK, page_size), 127, dtype=torch.uint8, device=device)
              for _ in range(2)]
    return KvCache(*data, *scales)


def kv_append(cache: KvCache, k, v, slots, positions=None, frequencies=None, *, interleaved: bool = False,
              scale: float = 1.0, stream=None) -> None:
    """Stores tokens in the cache: ``k``, turned as by :func:`rotary` where
    there are frequencies, and ``v``, each rounded to 4 bits with an exponent
    for every 32 columns. ``k`` and ``v``: (tokens, heads, dim) or (outer,
    inner, heads, dim) of the cache's heads; ``slots``: int32 or int64, page *
    page_size + place for each token, none of them twice. Slots below 0 or
    beyond the cache are left out."""
    if stream is not None:
        with _on(stream):
            return _b.kv_append(cache, k, v, slots, positions, frequencies, interleaved, scale)
    return _b.kv_append(cache, k, v, slots, positions, frequencies, interleaved, scale)


def kv_read(cache: KvCache, slots, *, dtype=torch.bfloat16, keys=None, values=None, stream=None) -> KvValues:
    """The values that the cache holds in ``slots`` (one or two dimensions), of
    shape ``slots.shape + (heads, dim)``; zeros for slots below 0 or beyond the
    cache. ``keys`` and ``values`` may be given."""
    if dtype not in _VALUE_TYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    code = _VALUE_TYPES[dtype]
    if stream is not None:
        with _on(stream):
            return KvValues._make(_b.kv_read(cache, slots, code, keys, values))
    return KvValues._make(_b.kv_read(cache, slots, code, keys, values))


def paged_attention(q, cache: KvCache, pages, lengths, *, starts=None, causal: bool = True, window: int = 0,
                    scale: float | None = None, max_length: int | None = None, out=None, lse=None,
                    need_lse: bool = False, stream=None) -> Attention:
    """Softmax attention of each sequence's last tokens over its cached keys
    and values, those of the tokens themselves among them (append first).

    ``q``: (seqs, heads, dim) for single tokens, (seqs, n, heads, dim) for n
    tokens a sequence, or with ``starts`` (tokens, heads, dim), where sequence
    b has rows starts[b] to starts[b + 1]; rows of no sequence are left as they
    are in ``out`` and ``lse`` (and undefined where the call made those).
    Query heads are a multiple of the cache's: neighbouring ones share a key
    head. ``pages``: int32 (seqs, most pages), the page numbers of each
    sequence in order; ``lengths``: int32 (seqs,); ``starts``: int32
    (seqs + 1,), not decreasing.

    ``window`` > 0 limits a token to the last ``window`` positions, its own
    among them; ``scale`` is 1 / sqrt(dim) unless given, and above 0;
    ``max_length``, where a program knows it, says that no sequence is longer
    (default: all that a row of ``pages`` holds) and so into how many parts
    contexts are split. A token that sees nothing gets zeros, and minus
    infinity in ``lse``, which is returned if given or ``need_lse``; it is
    formed in fp32 from weights that are not rounded, whatever ``q``'s type.
    Wanting it may change the last bits of ``out`` in 16 bits."""
    if stream is not None:
        with _on(stream):
            return Attention._make(_b.paged_attention(q, cache, pages, lengths, starts, causal, window, scale,
                                                      max_length, out, lse, need_lse))
    return Attention._make(_b.paged_attention(q, cache, pages, lengths, starts, causal, window, scale, max_length, out,
                                              lse, need_lse))
