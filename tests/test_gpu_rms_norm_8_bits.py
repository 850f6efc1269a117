"""The 8-bit values of the norm against y / scale in 64 bits. y is taken from
the same call without 8 bits, in fp32, where it is not rounded again."""
import pytest
import torch

import ring_all_reduce_allreduce_amd as rs

pytestmark = pytest.mark.gpu
#: Roundings of the reciprocal and of the product, 2^-24 each, and of this
#: test's own way to e4m3 through fp32, 2^-24.
NEAR = 2.0 ** -22


def e4m3(v):
    return v.float().to(torch.float8_e4m3fn).float()


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows, cols", [(4096, 4096), (1, 449), (333, 1000), (20, 30000), (9000, 100)])
def test_values_are_nearest_to_y_over_scale(rows, cols, group):
    """Every q is what y / scale rounds to; next to the middle of two 8-bit
    values, either of them."""
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.empty(rows, cols, device="cuda").normal_(generator=gen)
    x[0] = torch.arange(cols, device="cuda") - cols // 3  # many ties
    w = torch.full((cols,), 448.0, device="cuda")
    y = rs.rms_norm(x, w, eps=0.0).out
    got = rs.rms_norm(x, w, eps=0.0, out_dtype="float8_e4m3", group=group)
    spread = got.scales.double().repeat_interleave(group or cols, -1)[:, :cols]
    ideal = y.double() / spread
    q = got.out.float()
    low, high = e4m3(ideal.abs() * (1 - NEAR)), e4m3(ideal.abs() * (1 + NEAR))
    assert bool(((q.abs() >= low) & (q.abs() <= high)).all())
    assert bool((q * ideal >= 0).all())
    # Nothing beyond the largest value, which the largest of a group takes.
    top = q.abs().amax(-1) if group == 0 else q.abs()[:, :group].amax(-1)
    assert bool((top == 448.0).all())


def test_scales_are_the_largest_over_448():
    x = torch.randn(50, 1000, device="cuda")
    y = rs.rms_norm(x).out
    got = rs.rms_norm(x, out_dtype="float8_e4m3", group=128)
    want = torch.stack([p.abs().amax(-1) for p in y.split(128, -1)], -1).double() / 448.0
    assert torch.equal(got.scales, want.float())
