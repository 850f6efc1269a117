"""What the cache holds in positions that a token does not see stays out of its
result, whatever the bytes there are: exponent bytes from 253 on take the larger
codes past fp32's range (253: 4 and 6; 254: 2 and more), 255 is NaN."""
import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests import _attention_ref as ref
from tests._gpu import say
from tests.test_gpu_paged_attention import TYPES, _cache, _q, _ragged

pytestmark = pytest.mark.gpu

#: (tokens of each sequence, their lengths, key heads, queries a key head, window): a call's rows of a key head decide
#: whether waves share rows or have their own, the number of tiles and positions whether workgroups share a context.
CALLS = {
    "single tokens": ([1, 1, 1], [50, 17, 5], 2, 2, 0),
    "single tokens, window": ([1, 1], [150, 300], 1, 5, 33),
    "some tokens": ([1, 3, 2], [50, 70, 200], 2, 2, 0),
    "some tokens, window": ([2, 4], [90, 130], 1, 3, 20),
    "prompts": ([90, 70], [100, 200], 2, 2, 0),
    "prompts, window": ([150, 100], [210, 333], 1, 2, 140),
    "prompts, short window": ([100], [150], 2, 2, 33),
    "prompts over a shared context": ([61, 80], [4200, 4499], 1, 2, 0),
}
#: (byte, codes): infinite, infinite of either sign beside what is finite, and NaN
BLOCKS = ((253, 0x76), (254, 0xf5), (254, 0x12), (255, 0x21))


def _taint(cache, page, off, byte, codes, heads=slice(None)):
    for data, scales in ((cache.keys, cache.key_scales), (cache.values, cache.value_scales)):
        data[page, heads, off] = codes
        scales[page, heads, :, off] = byte


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_any_bytes_may_stand_where_no_row_looks(dtype, call):
    """Behind the ends, in pages of no sequence, behind a token in causal order and before its window. Rows that do see
    such a place are not compared: exponents of 253 and 254 stand for nothing."""
    counts, lengths, kv_heads, group, window = CALLS[call]
    page = 16
    starts, rows = _ragged(counts, 0)
    at = starts.tolist()
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    rel = ref.ONE_PART if dtype is torch.bfloat16 else None  # what the kernels with the fewest parts hold
    for dim in (64, 128, 192):
        clean, table = _cache(lengths, page, kv_heads, dim, seed=dim)
        q = _q((rows, kv_heads * group, dim), dtype, std=1.5)
        want = ref.attention([q[a:b] for a, b in zip(at, at[1:])], clean, table, n, window=window, weight_rel=rel)
        free = sorted(set(range(clean.keys.shape[0])) - {int(i) for i in table.flatten()})
        # a place inside: of the last sequence, seen by its last row and no other one, or where there is one row by none
        inner = [None, lengths[-1] - 1 if counts[-1] > 1 else None, lengths[-1] - window - 1 if window else None]
        for byte, codes in BLOCKS:
            for place in dict.fromkeys(inner):
                say(f"{call} {dtype} {dim} {byte} {codes:x} {place}")
                cache = rs.KvCache(*(t.clone() for t in clean))
                for b, length in enumerate(lengths):
                    if length % page:
                        _taint(cache, int(table[b, length // page]), slice(length % page, page), byte, codes)
                for i in free:
                    _taint(cache, i, slice(0, page), byte, codes)
                if place is not None:
                    _taint(cache, int(table[-1, place // page]), place % page, byte, codes)
                # single tokens without starts, for which there is a kernel of their own
                got = rs.paged_attention(q, cache, table, n, starts=None if max(counts) == 1 else starts, window=window,
                                         need_lse=True)
                for b, (o, l, bound, l_bound) in enumerate(want):
                    blind = torch.ones(counts[b], dtype=torch.bool)
                    if place is not None and b == len(counts) - 1:
                        for i in range(counts[b]):
                            lo, hi = ref.seen(lengths[b], counts[b], i, True, window, lengths[b])
                            blind[i] = not lo <= place < hi
                    mine = slice(at[b], at[b + 1])
                    what = f"{call} {dim} {byte} {codes:x} {place}, sequence {b}"
                    ref.within(got.out[mine][blind], o[blind], (bound + ref.half_step(o, dtype))[blind], what)
                    ref.within(got.lse[mine][blind], l[blind], l_bound[blind], what + ", lse")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_one_call_with_all_of_them(dtype):
    """A NaN that some rows see beside infinities that none sees: NaN in those rows' 32 columns alone."""
    counts, lengths, dim, page = [80, 75], [100, 139], 64, 16
    starts, rows = _ragged(counts, 0)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    cache, table = _cache(lengths, page, 1, dim, seed=5)
    q = _q((rows, 2, dim), dtype)
    cache.value_scales[int(table[0, 60 // page]), 0, 1, 60 % page] = 255
    want = ref.attention([q[:80], q[80:]], cache, table, n,
                         weight_rel=ref.ONE_PART if dtype is torch.bfloat16 else None)
    for b, length in enumerate(lengths):
        _taint(cache, int(table[b, length // page]), slice(length % page, page), 254, 0x77)
    got = rs.paged_attention(q, cache, table, n, starts=starts)
    for mine, (o, _, bound, _) in zip((slice(0, 80), slice(80, 155)), want):
        ref.within(got.out[mine], o, torch.nan_to_num(bound) + ref.half_step(o, dtype), f"rows {mine}")
    nan = torch.isnan(got.out[:80])
    assert bool(nan[40:, :, 32:].all()) and not bool(nan[:40].any()) and not bool(nan[:, :, :32].any())
