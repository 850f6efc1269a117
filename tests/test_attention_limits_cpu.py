"""The C entries of the attention-step operators at the ends of their arguments'
ranges. Needs no GPU: a call is refused before anything is enqueued, and sizes of
workspaces are the host's."""
import ctypes

import pytest

import ring_all_reduce_allreduce_amd as rs

from tests.test_attention_cpu import BAD, OK, L, _append, _attention, _host, _rotary  # noqa: F401

MOST = 2 ** 63 - 1


def _bytes(L, **over):  # noqa: F811
    n = ctypes.c_size_t(12345)
    assert L.ringsim_paged_attention_workspace(_attention(**over), n) == OK
    return n.value


@pytest.mark.parametrize("sizes", [dict(tokens=1, seqs=1, max_pages=512), dict(tokens=64, seqs=64, max_pages=256),
                                   dict(tokens=512, seqs=1, max_pages=512), dict(tokens=3 * 2048, seqs=3, max_pages=94)],
                         ids=str)
def test_windows_past_every_position_cut_a_call_as_none_does(L, sizes):  # noqa: F811
    want = _bytes(L, **sizes)
    for window in (1 << 31, 1 << 40, MOST - 1000, MOST - 1, MOST):
        assert _bytes(L, window=window, **sizes) == want


@pytest.mark.parametrize("pairs", [1 << 62, (1 << 62) + 1, (1 << 62) + (1 << 20), MOST, -(1 << 62), -MOST - 1])
def test_pairs_beyond_a_head_are_refused(L, pairs):  # noqa: F811
    """2 * pairs does not fit 64 bits: it must not look like a small number. Calls without tokens, which enqueue nothing."""
    assert L.ringsim_rotary(_rotary(pairs=pairs, outer=0), None) == BAD
    assert L.ringsim_kv_append(_append(pairs=pairs, outer=0), None) == BAD
    assert L.ringsim_rotary(_rotary(outer=0), None) == OK and L.ringsim_kv_append(_append(outer=0), None) == OK


@pytest.mark.parametrize("cache", [dict(page_size=1 << 62), dict(page_size=MOST), dict(page_size=2048), dict(page_size=48),
                                   dict(dim=80), dict(dim=1 << 40), dict(dim=MOST)], ids=str)
def test_workspaces_of_impossible_caches_are_refused(L, cache):  # noqa: F811
    """As the call itself refuses them: sizes whose products leave 64 bits have no workspace."""
    n = ctypes.c_size_t(0)
    assert L.ringsim_paged_attention_workspace(_attention(cache), n) == BAD


def test_workspaces_do_not_depend_on_the_number_of_pages(L):  # noqa: F811
    n, want = ctypes.c_size_t(0), _bytes(L)
    for pages in (0, 1, MOST):
        assert L.ringsim_paged_attention_workspace(_attention(dict(pages=pages)), n) == OK and n.value == want


def test_numbers_out_of_range_are_values_refused():
    """Of the binding: TypeError or ValueError, as for other wrong arguments."""
    cache, x, i, f, pages, lengths = _host()
    for call in (lambda: rs.paged_attention(x, cache, pages, lengths, window=1 << 70),
                 lambda: rs.paged_attention(x, cache, pages, lengths, max_length=-(1 << 70)),
                 lambda: rs.paged_attention(x, cache, pages, lengths, scale=10 ** 400),
                 lambda: rs.rotary(x, i, f, scale=10 ** 400), lambda: rs.kv_append(cache, x, x, i, scale=-10 ** 400)):
        with pytest.raises(ValueError, match="out of range"):
            call()
