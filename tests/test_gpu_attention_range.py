"""The range of values that attention's sums hold: below 2^119 over the positions that a token sees."""
import pytest
import torch

from tests import _attention_ref as ref
from tests._gpu import say
from tests.test_gpu_paged_attention import _cache, _q, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 192])
def test_large_and_small_values(dim, dtype):
    """Blocks of up to 6 * 2^e with 6 * 2^e * n < 2^119, where the weights grow by their full slack of 2^8 (scores of
    many sizes, in any order); and of down to 2^-101, whose products with the smallest weights that count, 2^-24, are
    normal."""
    rel = ref.ONE_PART if dtype is torch.bfloat16 else None
    for length, shape in ((60, (1, 4, dim)), (2000, (1, 4, dim)), (200, (1, 90, 2, dim))):
        top = 119 - 3 - (length - 1).bit_length()  # 6 < 2^3
        for e in (top, -100):
            say(f"{dim} {dtype} {length} {e}")
            cache, table = _cache([length], 16, 1, dim, seed=length, scale_byte=(126, 129))
            cache.value_scales.copy_(torch.randint(127 + e - 1, 127 + e + 1, cache.value_scales.shape,
                                                   generator=torch.Generator().manual_seed(e + 200), dtype=torch.uint8))
            _run(_q(shape, dtype, std=3.0), cache, table, [length], f"2^{e}", weight_rel=rel)
