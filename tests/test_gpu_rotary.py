"""Rotary positions and their gradient against the formula in 64 bits."""
import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests import _attention_ref as ref
from tests._gpu import say

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _x(shape, dtype, seed=0, side=0):
    """[..., heads, dim] inside rows of `side` more heads."""
    gen = torch.Generator().manual_seed(seed)
    wide = torch.empty(*shape[:-2], shape[-2] + side, shape[-1]).normal_(generator=gen).to(dtype).cuda()
    return wide[..., :shape[-2], :]


def _check(x, pos, freq, interleaved, scale, what, inverse=False, out=None):
    call = rs.rotary_backward if inverse else rs.rotary
    before = x.clone()
    y = call(x, pos, freq, interleaved=interleaved, scale=scale,
             **({} if out is None else {"grad_in" if inverse else "out": out}))
    assert out is None or y is out
    full = pos.cpu().expand(x.shape[:-2])
    want = ref.turn(before, full, freq, interleaved, inverse, scale)
    ref.within(y, want, ref.turn_bound(before, want, full, freq, interleaved, scale, x.dtype), what)
    if out is None:
        assert torch.equal(x, before)
    return y


# (tokens, heads, dim, pairs): whole packs, single pairs, odd ends, one of everything, many heads, long heads
SHAPES = [(1, 1, 2, 1), (1, 40, 128, 64), (7, 5, 128, 64), (33, 3, 80, 40), (5, 2, 96, 16), (130, 1, 64, 32),
          (17, 9, 100, 25), (3, 4, 7, 2), (6, 3, 33, 16), (2, 70, 256, 128), (4, 2, 24, 0), (1, 3, 2048, 1024),
          (300, 2, 16, 3)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rotary(shape, interleaved, dtype):
    tokens, heads, dim, pairs = shape
    say(f"rotary {shape} {interleaved} {dtype}")
    freq = rs.rotary_frequencies(2 * pairs)
    gen = torch.Generator().manual_seed(tokens)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=gen).cuda()
    x = _x((tokens, heads, dim), dtype, side=1)
    _check(x, pos, freq, interleaved, 1.0, "forward")
    _check(x, pos.int(), freq, interleaved, 0.75, "32-bit positions, scaled")
    _check(x, pos, freq, interleaved, 1.25, "backward", inverse=True)
    y = _x((tokens, heads, dim), dtype, seed=5)
    _check(y, pos, freq, interleaved, 1.0, "in place", out=y)
    _check(y, pos, freq, interleaved, 1.0, "backward in place", inverse=True, out=y)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_views(dtype):
    """Heads before tokens, positions shared by a batch, strided positions, odd addresses, negative positions."""
    freq = rs.rotary_frequencies(64)
    say(f"views {dtype}")
    t = _x((2, 5, 11, 64), dtype)  # [batch, heads, tokens, dim]
    pos = torch.arange(-3, 8).cuda()
    _check(t.transpose(1, 2), pos, freq, False, 1.0, "heads before tokens")
    _check(t.transpose(1, 2), pos.expand(2, 11), freq, True, 1.0, "expanded positions")
    both = torch.arange(44).cuda().view(2, 22)[:, ::2]
    _check(t.transpose(1, 2), both, freq, False, 1.0, "strided positions")
    flat = torch.randn(6 * 3 * 65 + 1).to(dtype).cuda()
    odd = flat[1:].as_strided((6, 3, 64), (3 * 65, 65, 1), 1)
    _check(odd, torch.arange(6).cuda(), freq, False, 1.0, "odd addresses")
    _check(odd, torch.arange(6).cuda(), freq, True, 1.0, "odd addresses, neighbours")
    out = torch.zeros(6 * 3 * 70, device="cuda", dtype=dtype).as_strided((6, 3, 64), (70, 6 * 70, 1), 3)
    _check(odd, torch.arange(6).cuda(), freq, False, 1.0, "into strided heads", out=out)
    _check(_x((1, 9, 3, 64), dtype), torch.arange(9).cuda(), freq, False, 1.0, "a batch of one")


def test_nothing_beside_the_output_is_written():
    freq = rs.rotary_frequencies(32)
    for dtype, dim in ((torch.bfloat16, 48), (torch.float32, 41), (torch.float16, 32)):
        wide = torch.full((9, 5, dim + 6), 7.0, device="cuda", dtype=dtype)
        rs.rotary(_x((9, 4, dim), dtype), torch.arange(9).cuda(), freq, out=wide[:, :4, 3:3 + dim])
        wide[:, :4, 3:3 + dim] = 7.0
        assert bool((wide == 7.0).all())


def test_far_positions_keep_their_angles():
    """Positions beyond 2^31: the angle's error is that of 64 bits, position * frequency * 2^-52."""
    freq = rs.rotary_frequencies(32)
    pos = torch.tensor([2 ** 24 + 1, 2 ** 31 - 1, 2 ** 33 + 12345]).cuda()
    x = _x((3, 2, 32), torch.float32)
    y = rs.rotary(x, pos, freq)
    want = ref.turn(x, pos, freq, False)
    bound = ref.turn_bound(x, want, pos, freq, False, 1.0, torch.float32)
    angle = pos.double().cpu()[:, None, None] * freq.cpu() * 2.0 ** -51
    ref.within(y, want, bound + torch.cat([angle, angle], -1) * 8, "far")


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    """The forward pass is linear in x, so <g, rotary(d)> = <rotary_backward(g), d> up to roundings: each side sums
    n products of values off by at most 10 roundings of at most |a| + |b|."""
    freq = rs.rotary_frequencies(24, base=500.0)
    pos = torch.arange(5).cuda() * 31
    d, g = _x((5, 3, 40), torch.float32, 1), _x((5, 3, 40), torch.float32, 2)
    left = (g.double() * rs.rotary(d, pos, freq, interleaved=interleaved, scale=1.5).double()).sum()
    right = (rs.rotary_backward(g, pos, freq, interleaved=interleaved, scale=1.5).double() * d.double()).sum()
    size = float((g.double().abs().sum(-1) * d.double().abs().sum(-1)).sum())
    assert abs(float(left - right)) <= 20 * ref.U * 1.5 * size


def test_special_values_stay_in_their_pair():
    freq = rs.rotary_frequencies(16)
    x = torch.ones(2, 2, 24, device="cuda")
    x[0, 1, 3], x[1, 0, 20] = float("nan"), float("inf")
    y = rs.rotary(x, torch.arange(2).cuda() + 1, freq)
    bad = ~torch.isfinite(y)
    assert bad.nonzero().tolist() == [[0, 1, 3], [0, 1, 11], [1, 0, 20]]


def test_many_tokens_and_heads():
    """More workgroups than a launch holds at once, and heads cut over workgroups; every element once."""
    freq = rs.rotary_frequencies(8)
    for shape in ((70001, 3, 8), (3, 4001, 8), (1, 65535, 4)):
        say(f"many {shape}")
        f = rs.rotary_frequencies(shape[2])
        x = _x(shape, torch.bfloat16)
        _check(x, torch.arange(shape[0]).cuda(), f, False, 1.0, str(shape))
    assert freq.numel() == 4


def test_no_tokens():
    freq = rs.rotary_frequencies(8)
    for shape in ((0, 3, 8), (2, 0, 3, 8), (3, 0, 8)):
        x = torch.zeros(shape, device="cuda")
        pos = torch.zeros(shape[:-2], device="cuda", dtype=torch.int64)
        assert rs.rotary(x, pos, freq).shape == x.shape


def test_stream_and_version():
    freq = rs.rotary_frequencies(64)
    x, pos = _x((64, 8, 64), torch.bfloat16), torch.arange(64).cuda()
    want = rs.rotary(x, pos, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rs.rotary(x, pos, freq, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    y = x.contiguous()
    version = y._version
    rs.rotary(y, pos, freq, out=y)
    assert y._version > version and torch.equal(y, want)


def test_frequencies():
    f = rs.rotary_frequencies(8, base=100.0)
    assert f.dtype is torch.float64 and torch.allclose(f.cpu(), torch.tensor([100.0 ** (-i / 4) for i in range(4)]).double())
    assert torch.allclose(rs.rotary_frequencies(8, factor=4.0), rs.rotary_frequencies(8) / 4)
    raised, plain = rs.rotary_frequencies(8, factor=4.0, method="base"), rs.rotary_frequencies(8)
    assert float(raised[0]) == 1.0 and abs(float(raised[-1] / plain[-1]) - 0.25) < 1e-12
    ramp = rs.rotary_frequencies(64, factor=8.0, method="ramp", trained=4096, low=1.0, high=32.0)
    plain = rs.rotary_frequencies(64)
    turns = 4096 * plain / (2 * torch.pi)
    assert torch.equal(ramp[turns >= 32], plain[turns >= 32])
    assert torch.allclose(ramp[turns <= 1], plain[turns <= 1] / 8, rtol=1e-12)
    between = (turns > 1) & (turns < 32)
    assert bool(((ramp < plain) & (ramp > plain / 8))[between].all())
