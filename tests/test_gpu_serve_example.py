"""The serving example gives on several ranks what it gives on one."""
import importlib.util
import os

import pytest
import torch

from tests._gpu import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("serve_step", os.path.join(ROOT, "examples", "serve_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("ranks", [2, 4])
def test_ranks_agree(ex, ranks):
    """In fp32 the projections of other shapes add in other orders: 512 terms, off by up to 512 * 2^-24 = 3e-5 of their
    magnitudes. That may move a key or value that lies as near to one of the 14 borders between codes over it, so at
    most 14 * 2 * 3e-5 = 1e-3 of them, by a step of at most 2/6 of the block's largest, which is about 2.5 times the
    root mean square: the square root of 1e-3 times 5/6 is 2.6% of a cache's norm, and no more of what attention reads
    out of it. Behind a step that much of the block's results may be different, and the next step begins with it.
    A head taken from another rank, a slot or position past the right one, a replay over old inputs or a part missing
    from the sum changes the block's results by half of their norm and more."""
    prompts = (20, 1, 33)
    say(f"ranks {ranks}")
    prompt, steps, _, pages = ex.serve(ranks=ranks, steps=5, prompts=prompts, dtype=torch.float32)
    alone, alone_steps, _, alone_pages = ex.serve(ranks=1, steps=5, prompts=prompts, dtype=torch.float32)
    assert pages.lengths == alone_pages.lengths and pages.table == alone_pages.table
    x = torch.empty(sum(prompts), ex.WIDTH).normal_(generator=torch.Generator().manual_seed(1)).cuda()
    last = [sum(prompts[:i + 1]) - 1 for i in range(len(prompts))]
    before, before_alone = x, x
    for i, (got, want) in enumerate(zip((prompt, *steps), (alone, *alone_steps))):
        block, block_alone = got - before, want - before_alone  # what this call added to the residual stream
        off = float((block - block_alone).norm() / block_alone.norm())
        assert off <= 0.026 * (i + 1), f"call {i}: {off} of the block's result"
        before, before_alone = (got, want) if i else (got[last], want[last])
