"""Views with several leading dimensions as rows of the norm and of its
gradients: which ones are taken, which refused, and that every row is read and
written where the view has it. Dimensions of size 1, whose strides mean
nothing, stand at every place."""
import itertools
import os
import random

import pytest
import torch

from ring_all_reduce_allreduce_amd import build

if not (os.path.exists(build.LIB) and os.path.exists(build.BINDING)):
    build.build()
import ring_all_reduce_allreduce_amd as rs  # noqa: E402
from tests import _ops_ref as ref  # noqa: E402

EPS = 1e-5

#: (shape of the memory, the view of it): rows that two strides cannot
#: describe, most with a dimension of size 1 that stands before the gap.
GAPPED = {
    "five, gap behind a one": ((2, 1, 8, 4, 16), lambda t: t[:, :, :5]),
    "five, no one": ((2, 3, 8, 4, 16), lambda t: t[:, :, :5]),
    "four, gap": ((2, 3, 8, 16), lambda t: t[:, :2, :5]),
    "repeated behind a one": ((1, 3, 3, 4, 16), lambda t: t.expand(4, 3, 3, 4, 16)[:, :1]),
    "two ones": ((2, 1, 1, 8, 4, 16), lambda t: t[:, :, :, :5]),
    "repeated batch": ((1, 5, 4, 16), lambda t: t.expand(3, 5, 4, 16)),
}
#: Rows that two strides do describe, though a dimension of size 1 has a
#: stride that does not fit its neighbours.
REGULAR = {
    "one head of several": ((4, 8, 3, 16), lambda t: t[:, :1]),
    "one token of a padded batch": ((6, 48, 16), lambda t: t[:, :32].unsqueeze(1)),
    "five, without a gap": ((2, 1, 5, 4, 16), lambda t: t),
    "a one in front": ((1, 7, 4, 16), lambda t: t[:, 1:6]),
    "a one inside": ((5, 9, 4, 16), lambda t: t[:, 3:4, :3]),
    "a one last": ((5, 4, 3, 16), lambda t: t[:, :, 1:2]),
    "ones everywhere": ((1, 5, 1, 4, 1, 16), lambda t: t[:, :, :, :3]),
    "only ones": ((1, 3, 1, 16), lambda t: t[:, 2:3]),
    "any two strides": ((3, 1, 7, 16), lambda t: t.transpose(0, 2)),
    "no rows": ((2, 3, 8, 4, 16), lambda t: t[:, :0, :5]),
    "a vector": ((16,), lambda t: t),
}


def describable(shape, strides):
    """Whether outer and inner strides reach every row: the definition, by
    the rows' offsets."""
    dims = [(n, s) for n, s in zip(shape[:-1], strides[:-1]) if n != 1]
    if any(n == 0 for n, _ in dims) or len(dims) < 2:
        return True
    inner_n, inner_s = dims[-1]
    outer = [sum(i * s for i, (_, s) in zip(at, dims[:-1])) for at in itertools.product(*(range(n) for n, _ in dims[:-1]))]
    step = outer[1] - outer[0]
    return outer == [i * step for i in range(len(outer))]


def taken(view):
    """Whether the binding takes a view of host memory as far as its strides
    go: it is then refused for where it lies."""
    with pytest.raises(ValueError) as e:
        rs.rms_norm(view)
    text = str(e.value)
    assert "on the current device" in text or "leading dimensions" in text, text
    return "on the current device" in text


@pytest.mark.parametrize("name", GAPPED)
def test_gapped_views_are_refused(name):
    shape, view = GAPPED[name]
    v = view(torch.zeros(shape))
    assert not describable(v.shape, v.stride()) and not taken(v)


@pytest.mark.parametrize("name", REGULAR)
def test_regular_views_are_taken(name):
    shape, view = REGULAR[name]
    v = view(torch.zeros(shape))
    assert describable(v.shape, v.stride()) and taken(v)


def test_random_views():
    """Slices of random memory with up to six dimensions, dimensions permuted
    and repeated: taken exactly where two strides reach every row."""
    rng = random.Random(5)
    seen = set()
    for _ in range(4000):
        n = rng.randint(1, 5)
        t = torch.zeros([rng.choice((1, 1, 2, 3)) for _ in range(n)] + [4])
        if rng.random() < 0.3:
            order = list(range(n))
            rng.shuffle(order)
            t = t.permute(*order, n)
        for d in range(n):
            if rng.random() < 0.3:
                at = rng.randrange(t.shape[d])
                t = t.narrow(d, at, rng.randint(1, t.shape[d] - at))
        if rng.random() < 0.2:
            t = t.expand([rng.choice((1, 3)) if s == 1 else s for s in t.shape[:-1]] + [4])
        want = describable(t.shape, t.stride())
        assert taken(t) == want, (tuple(t.shape), t.stride())
        seen.add((want, t.dim()))
    assert {(w, d) for w in (True, False) for d in (4, 5, 6)} <= seen


# ---------------------------------------------------------------------------
# On the device
# ---------------------------------------------------------------------------


def filled(shape, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.empty(shape).normal_(generator=gen).to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("name", REGULAR)
def test_rows_lie_where_the_view_has_them(name):
    """Inputs and outputs through each view; what lies between the rows stays."""
    shape, view = REGULAR[name]
    w = filled((16,), 1)
    x, r, dy = (filled(shape, i) for i in (2, 3, 4))
    xd, rd, dyd, wd = (t.cuda() for t in (x, r, dy, w))
    outs = [torch.full(shape, 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    q = torch.full(shape, 9.0, device="cuda").to(torch.float8_e4m3fn)
    got = rs.rms_norm(view(xd), wd, residual=view(rd), eps=EPS, out=view(outs[0]), residual_out=view(outs[1]))
    h, _, y = ref.norm(view(x), view(r), w, EPS)
    ref.within(got.out, y, y.abs() * ref.Y_REL + ref.half_step(y, x.dtype), name + " out")
    ref.within(got.residual, h, h.abs() * ref.U + ref.half_step(h, x.dtype), name + " residual")
    assert torch.equal(view(outs[0]), got.out) and torch.equal(view(outs[1]), got.residual)
    assert torch.equal(rs.rms_norm(view(xd), wd, residual=view(rd), eps=EPS).out, got.out)
    whole = rs.rms_norm(view(xd).contiguous(), wd, eps=EPS, out_dtype="float8_e4m3")
    part = rs.rms_norm(view(xd), wd, eps=EPS, out_dtype="float8_e4m3", out=view(q))
    assert torch.equal(part.out.float(), whole.out.float()) and torch.equal(part.scales, whole.scales)
    back = rs.rms_norm_backward(view(dyd), view(xd), wd, grad_residual=view(rd), eps=EPS, grad_in=view(outs[2]))
    dx, dw, bound, terms = ref.backward(view(dy), view(x), w, view(r), EPS)
    ref.within(view(outs[2]), dx, bound + ref.half_step(dx, x.dtype), name + " grad_in")
    # A column adds at most 64 rows here.
    ref.within(back.grad_weight, dw, terms * (64 + 64 + ref.SUM / 2 + 8) * ref.U + ref.half_step(dw, w.dtype),
               name + " grad_weight")
    for t in outs:
        view(t).fill_(9.0)
        assert bool((t == 9.0).all()), "written outside the view"
    view(q).copy_(torch.full(view(q).shape, 9.0, device="cuda"))
    assert bool((q.float() == 9.0).all()), "written outside the view"


@pytest.mark.gpu
@pytest.mark.parametrize("name", GAPPED)
def test_gapped_views_are_refused_on_the_device(name):
    """As every argument, before anything is written."""
    shape, view = GAPPED[name]
    t = torch.full(shape, 3.0, device="cuda")
    bad, q = view(t), view(torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn))
    good = torch.ones(bad.shape, device="cuda")
    for call in (lambda: rs.rms_norm(bad), lambda: rs.rms_norm(good, residual=bad), lambda: rs.rms_norm(good, out=bad),
                 lambda: rs.rms_norm(good, residual=good, residual_out=bad),
                 lambda: rs.rms_norm(good, out_dtype="float8_e4m3", out=q),
                 lambda: rs.rms_norm_backward(bad, good), lambda: rs.rms_norm_backward(good, bad),
                 lambda: rs.rms_norm_backward(good, good, grad_residual=bad),
                 lambda: rs.rms_norm_backward(good, good, grad_in=bad)):
        with pytest.raises(ValueError, match="leading dimensions"):
            call()
    torch.cuda.synchronize()
    assert bool((t == 3.0).all())
