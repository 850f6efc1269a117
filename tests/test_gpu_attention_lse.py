"""lse is the logarithm of the sum of the weights themselves, in fp32, also where
the weights that go into the second product are rounded to fewer bits."""
import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests._gpu import say
from tests.test_gpu_paged_attention import TYPES

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

#: (sequences, tokens of each, queries a key head, pages in a row of the table): waves that share rows and workgroups
#: that share a context; a workgroup a tile, as there are more than 512 of them; waves with rows of their own.
CALLS = {
    "single tokens": (7, 1, 16, 64),
    "many single tokens": (520, 1, 16, 9),
    "some tokens": (5, 4, 4, 64),
    "many of some tokens": (520, 2, 8, 9),
    "prompt": (1, 128, 1, 25),
    "prompts": (2, 150, 2, 30),
    "prompt over a shared context": (1, 200, 1, 400),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_two_positions(dtype, call):
    """Every row sees a position of score 0 and one of score x (the others' weights are exp(-190) and less): lse is
    log(1 + exp(x)). x is one column's product with 1, so exact. Near the first position x is below 0, so that its
    weight is rounded beside one of 1; further behind it is above 0, where the weight of 1 stays the reference.

    Roundings, in units of 2^-24 (s the larger of x and 0, lse >= s): scale * log2(e) and the product with it, 2 of |x|
    or less, which counts by the weight's share, so by less than lse; exp2, 2; the sums 4; its logarithm 2 of at most
    lse + 0.7; the reference's, ln 2's and the last product's roundings, 1 of lse each. 8 * lse + 10 in all."""
    seqs, tokens, group, most = CALLS[call]
    for dim in (64, 128):
        for place in (1, 32, 128):
            if place // 16 >= most:
                continue
            say(f"{call} {dtype} {dim} {place}")
            cache = rs.kv_cache(2, 1, 16, dim)
            cache.keys[:, 0, :, 0], cache.key_scales[:, 0, 0] = 0x0f, 133  # -6 * 2^6
            cache.keys[0, 0, 0, 0] = 0
            page, off = (0, place) if place < 16 else (1, place % 16)
            cache.keys[page, 0, off, 0], cache.key_scales[page, 0, 0, off] = 2, 127  # 1
            table = torch.full((seqs, most), -1, dtype=torch.int32)
            table[:, 0] = 0
            if page:
                table[:, place // 16] = 1
            gen = torch.Generator().manual_seed(place + dim)
            x = torch.rand(seqs, tokens, group, generator=gen)
            x = (-0.69 * x if place < 16 else 0.5 + 5 * x).to(dtype)
            q = torch.zeros(seqs, tokens, group, dim, dtype=dtype)
            q[..., 0] = x
            n = torch.full((seqs,), place + 1, dtype=torch.int32).cuda()
            q, table = q.cuda(), table.cuda()
            got = rs.paged_attention(q if tokens > 1 else q[:, 0], cache, table, n, causal=False, scale=1.0,
                                     need_lse=True).lse.view(x.shape)
            want = torch.log1p(torch.exp(x.double()))
            off_by = ((got.double().cpu() - want).abs() - U * (8 * want + 10))
            assert float(off_by.max()) <= 0.0, \
                f"{call} {dim} {place}: {float(off_by.max())} beyond the bound, {int((off_by > 0).sum())} of {x.numel()}"


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_small_columns_of_many_rows_over_few_positions(dim, dtype):
    """Many rows of a key head that see 128 positions at most lose nothing of a score's small columns: all keys are ones,
    so that a row of c positions with columns 1 and +-2^-e has an lse of 1 +- 2^-e + log(c).

    Roundings, in units of 2^-24: five of the score (scale * log2(e), its product, ln 2, the product with it, the sum
    with a logarithm); exp2, 2; sums, one for each of 4 positions, 8 over lanes and waves; the logarithm's 2, ln 2's,
    the product's and the sum's, 6 of log(c); 2 more of the weights' arguments beside 0."""
    least = 16 if dtype == torch.bfloat16 else 20
    x = torch.zeros(3 * 2 * least, dim)
    for i, other in enumerate((1, 7, 15)):
        for e in range(1, least + 1):
            for j, sign in enumerate((1, -1)):
                x[(i * least + e - 1) * 2 + j, 0] = 1.0
                x[(i * least + e - 1) * 2 + j, other] = sign * 2.0 ** -e
    rows, x = x.shape[0], x.to(dtype)
    cache = rs.kv_cache(1, 1, 16, dim)
    cache.keys.fill_(0x22)
    score = x.double().sum(-1)
    for length, window, pages in ((rows, 0, 8), (128, 0, 8), (700, 128, 44), (700, 27, 44), (3, 0, 1)):
        say(f"{dim} {dtype} {length} {window}")
        n = torch.tensor([length], dtype=torch.int32).cuda()
        table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
        causal = length >= rows
        got = rs.paged_attention(x.cuda().view(1, rows, 1, dim), cache, table, n, scale=1.0, window=window, causal=causal,
                                 need_lse=True).lse.view(-1)
        count = torch.arange(length - rows + 1, length + 1).clamp(max=window or length) if causal else torch.full((rows,), 3)
        want = score + torch.log(count.double())
        bound = U * (5 * score.abs() + 12 + count / 4 + 6 * torch.log(count.double()))
        off_by = (got.double().cpu() - want).abs() - bound
        assert float(off_by.max()) <= 0.0, f"{dim} {length} {window}: {float(off_by.max())} beyond the bound"
