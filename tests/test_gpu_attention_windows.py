"""Windows that reach past every position are none."""
import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests._gpu import say
from tests.test_gpu_paged_attention import TYPES, _cache, _q, _ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("counts,lengths", [([1, 1], [3000, 5]), ([4, 3], [700, 2]), ([90, 70], [200, 33]),
                                            ([61, 80], [4200, 20])], ids=str)
def test_the_same_bits(counts, lengths, dtype, causal):
    """Sequences with fewer tokens in the cache than in the call among them, whose first ones stand before position 0."""
    say(f"{counts} {dtype} {causal}")
    starts, rows = _ragged(counts, 0)
    cache, table = _cache(lengths, 64, 1, 64, seed=2)
    q, n = _q((rows, 2, 64), dtype), torch.tensor(lengths, dtype=torch.int32).cuda()
    want = rs.paged_attention(q, cache, table, n, starts=starts, causal=causal, need_lse=True)
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 63 - 1000, 2 ** 63 - 1):
        got = rs.paged_attention(q, cache, table, n, starts=starts, causal=causal, window=window, need_lse=True)
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse), window
