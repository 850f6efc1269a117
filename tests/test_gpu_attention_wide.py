"""Attention of many rows with a window, where each wave has rows of its own:
what the plan's check pins as such (attention_plan_check.cpp), with and without
lse, which in 16 bits are different kernels."""
import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests import _attention_ref as ref
from tests._gpu import say
from tests.test_gpu_paged_attention import TYPES, _cache, _q, _ragged

pytestmark = pytest.mark.gpu


def _check(q, counts, cache, table, n, starts, dtype, what, lse, **how):
    """`starts` may leave rows in front and behind: those stay as they are."""
    out = torch.full_like(q, 3.0)
    sums = torch.full(q.shape[:2], 3.0, device="cuda") if lse else None
    rs.paged_attention(q, cache, table, n, starts=starts, out=out, lse=sums, **how)
    at = starts.tolist()
    rel = ref.ONE_PART if dtype is torch.bfloat16 else None
    want = ref.attention([q[a:b] for a, b in zip(at, at[1:])], cache, table, n, weight_rel=rel, **how)
    for b, (o, l, bound, l_bound) in enumerate(want):
        mine = slice(at[b], at[b + 1])
        ref.within(out[mine], o, torch.nan_to_num(bound) + ref.half_step(o, dtype), f"{what}: out of sequence {b}")
        if lse:
            ref.within(sums[mine], l, torch.nan_to_num(l_bound), f"{what}: lse of sequence {b}")
    for t in (out, sums) if lse else (out,):
        assert bool((t[:at[0]] == 3.0).all()) and bool((t[at[-1]:] == 3.0).all()), f"{what}: rows of no sequence"
    return out


@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_windows(dim, dtype, lse):
    """Rows of a tile before, across and behind a window's ends; sequences with fewer tokens in the cache than here."""
    for counts, lengths, page, group, windows, causal in (([70, 50], [333, 210], 16, 2, (1, 27, 129, 300), True),
                                                          ([49, 0, 35], [350, 40, 20], 64, 4, (128, 200), True),
                                                          ([30, 20], [64, 200], 16, 5, (33, 190), False)):
        starts, rows = _ragged(counts, 5, before=2)
        cache, table = _cache(lengths, page, 1, dim, seed=dim)
        q, n = _q((rows, group, dim), dtype, std=1.5), torch.tensor(lengths, dtype=torch.int32).cuda()
        for window in windows:
            say(f"{dim} {dtype} {lse} {counts} {window}")
            _check(q, counts, cache, table, n, starts, dtype, f"window {window}", lse, window=window, causal=causal)


@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_nan_before_the_window_and_behind_the_end(dtype, lse):
    counts, lengths, dim, page = [100, 130], [190, 261], 128, 16
    starts, rows = _ragged(counts, 0)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    for window in (33, 150):
        cache, table = _cache(lengths, page, 2, dim, seed=window)
        q = _q((rows, 4, dim), dtype)
        for b, length in enumerate(lengths):
            for t in (cache.key_scales, cache.value_scales):
                t[int(table[b, length // page]), :, :, length % page:] = 255
        # seen by none (where there are so many), by the first rows, by all but the last one, by the last ones
        for place in (None, lengths[1] - counts[1] - window, lengths[1] - counts[1] - 3, lengths[1] - window - 1,
                      lengths[1] - 5):
            if place is not None and place < 0:
                continue
            say(f"{dtype} {lse} {window} {place}")
            if place is not None:
                for t in (cache.key_scales, cache.value_scales):
                    t[int(table[1, place // page]), 1, 2, place % page] = 255
            got = _check(q, counts, cache, table, n, starts, dtype, f"window {window}, place {place}", lse, window=window)
            if place is None or place == lengths[1] - counts[1] - window:
                assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_the_longest_lengths(dtype, lse):
    """Prompts at the end of 2^31 positions, whose pages repeat: windows of few and of some more positions."""
    most = 2 ** 31 - 1
    cache, table = _cache([4096], 1024, 1, 64)
    table = torch.randint(0, cache.keys.shape[0], (1, 2 ** 21), generator=torch.Generator().manual_seed(6)).int().cuda()
    q = _q((1, 100, 1, 64), dtype)
    rel = ref.ONE_PART if dtype is torch.bfloat16 else None
    for window in (100, 250):
        for length in (most - 1023, most - 1100, most):
            say(f"{dtype} {lse} {window} {length}")
            n = torch.tensor([length], dtype=torch.int32).cuda()
            got = rs.paged_attention(q, cache, table, n, window=window, need_lse=lse)
            gone = (length - 400) // 1024  # pages that the window cannot reach
            (out, sums, bound, l_bound), = ref.attention([q[0]], cache, table[:, gone:], n - gone * 1024, window=window,
                                                         max_length=2 ** 31 - 1024 - gone * 1024, weight_rel=rel)
            ref.within(got.out[0], out, bound + ref.half_step(out, dtype), f"length {length}: out")
            if lse:
                ref.within(got.lse[0], sums, l_bound, f"length {length}: lse")
