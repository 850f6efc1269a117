"""The step operators' formulas in 64 bits on the host, and the error bounds
their tests use.

A result is rounded once to its type, off by at most half a step:
finfo.eps / 2 relative, or half the smallest subnormal. Before that, arithmetic
is in fp32 (u = 2^-24 a rounding). A row's sum is a chain of at most 32 fused
additions a lane, 6 joins inside a wave and up to 15 over waves, so sums of
positive terms are off by at most SUM u relative with SUM = 64; the
reciprocal root halves that and adds its own 2 ulp (4 u)."""
import torch

U = 2.0 ** -24
SUM = 64


def half_step(want, dtype):
    """Half a step of the type around `want` (64-bit values)."""
    f = torch.finfo(dtype)
    return want.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def norm(x, residual, weight, eps):
    """(h, r, y) of the forward formula."""
    h = x.double() if residual is None else x.double() + residual.double()
    r = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return h, r, h * r if weight is None else h * r * weight.double()


#: Relative error of y before its rounding: half the sum's and of the mean's
#: and eps's roundings, the root's, and one each for h and the two products.
Y_REL = (SUM / 2 + 2 + 4 + 3) * U


def scales(y, group):
    """e4m3 scales, one for each `group` columns (0: a row)."""
    parts = y.split(group or y.shape[-1], -1)
    return torch.stack([p.abs().amax(-1) for p in parts], -1).div(448.0).clamp_min(2.0 ** -126)


def backward(dy, h, weight, residual, eps):
    """(grad_in, grad_weight, bound of grad_in's fp32 arithmetic, sum of the
    magnitudes that grad_weight adds)."""
    dy, h = dy.double(), h.double()
    r = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    g = dy if weight is None else dy * weight.double()
    m = (g * h).mean(-1, keepdim=True)
    dx = r * g - h * r.pow(3) * m
    # r is off by SUM/2 + 6, r^3 by three times that and 2 roundings, the mean
    # by SUM + 3 of its terms' magnitudes; each product and the subtraction add one.
    bound = (r * g).abs() * (SUM / 2 + 6 + 2) * U + \
        (h * r.pow(3)).abs() * (g * h).abs().mean(-1, keepdim=True) * (3 * (SUM / 2 + 6) + SUM + 8) * U + dx.abs() * U
    if residual is not None:
        dx = dx + residual.double()
        bound = bound + dx.abs() * U
    terms = (dy * h * r).reshape(-1, h.shape[-1])
    return dx, terms.sum(0), bound, terms.abs().sum(0)


def within(got, want, bound, what):
    """Every element of `got` within `bound` of `want`; NaN and infinities in
    the same places."""
    got = got.double().cpu()
    same = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), same), f"{what}: other places are finite"
    odd = ~same
    assert torch.equal(torch.isnan(got[odd]), torch.isnan(want[odd])), f"{what}: NaN elsewhere"
    off = (got - want).abs()[same] - bound.expand_as(want)[same]
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 0.0, f"{what}: {worst} beyond the bound, {int((off > 0).sum())} of {off.numel()} elements"
