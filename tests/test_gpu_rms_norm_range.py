"""The norm's gradients over the range of values that the forward pass takes:
rows far above and far below 1, on every layout of a row, against the formula
in 64 bits. The cube of the reciprocal root would leave fp32's range here."""
import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests import _ops_ref as ref
from tests._gpu import say

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# A part of a wave, a wave, two packs of it, whole waves, and 1024 lanes with two, four and eight packs.
COLS = (40, 250, 700, 1500, 6000, 9000, 20000, 32768)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("scale, eps", [(1e13, 1e-5), (1e14, 1e-5), (1e15, 0.0), (1e17, 1e-5), (3e4, 1e-5),
                                        (1e-12, 0.0), (1e-13, 0.0), (1e-15, 0.0), (1e-15, 1e-30)])
def test_backward_large_and_small_rows(scale, eps, cols):
    for name, dtype in DTYPES.items():
        for with_residual in (False, True):
            say(f"backward {name} rows of {scale} x {cols} eps {eps} residual {with_residual}")
            gen = torch.Generator().manual_seed(cols)
            h = (torch.empty(5, cols).normal_(generator=gen) * scale).to(dtype)
            # As large as grad_in, so that the sum of the two hides neither.
            dy = torch.empty(5, cols).normal_(generator=gen).to(dtype)
            r = (torch.empty(5, cols).normal_(generator=gen) / scale).to(dtype) if with_residual else None
            w = torch.empty(cols).normal_(1.0, 0.3, generator=gen).to(dtype)
            got = rs.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), grad_residual=None if r is None else r.cuda(), eps=eps)
            dx, dw, bound, terms = ref.backward(dy, h, w, r, eps)
            ref.within(got.grad_in, dx, bound + ref.half_step(dx, dtype), f"grad_in of {scale}")
            # Five rows: a chain of five additions and the joins of lanes that share a column.
            ref.within(got.grad_weight, dw, terms * (5 + 16 + ref.SUM / 2 + 8) * ref.U + ref.half_step(dw, dtype),
                       f"grad_weight of {scale}")


@pytest.mark.parametrize("cols", (333, 1500, 9000))
def test_rows_of_every_size_side_by_side(cols):
    """Rows from 1e-15 to 1e17 in one call: each has its own gradient."""
    gen = torch.Generator().manual_seed(1)
    scales = torch.logspace(-15, 17, 33)[:, None]
    h = torch.empty(33, cols).normal_(generator=gen) * scales
    dy = torch.empty(33, cols).normal_(generator=gen)
    got = rs.rms_norm_backward(dy.cuda(), h.cuda(), None, eps=0.0)
    dx, _, bound, _ = ref.backward(dy, h, None, None, 0.0)
    ref.within(got.grad_in, dx, bound + ref.half_step(dx, torch.float32), "grad_in")
