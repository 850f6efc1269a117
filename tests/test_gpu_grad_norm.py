"""grad_norm, scale_grads and clip_grads on the device against the formulas in
64 bits: lists of every kind, types, alignment, special values, streams and
graphs."""
import math

import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests import _ops_ref as ref
from tests._gpu import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def tensors(sizes, types, seed, std=0.03, gap=0):
    """Host values, and device tensors of them that lie `gap` elements apart
    in one buffer a type (so most start at odd addresses)."""
    gen = torch.Generator().manual_seed(seed)
    host = [torch.empty(n).normal_(0.0, std, generator=gen).to(t) for n, t in zip(sizes, types)]
    flats = {t: torch.full((sum(n + gap for n, u in zip(sizes, types) if u == t) + gap,), 7.0, dtype=t, device=DEV)
             for t in set(types)}
    at = dict.fromkeys(flats, gap)
    dev = []
    for h, t in zip(host, types):
        v = flats[t][at[t]:at[t] + h.numel()]
        v.copy_(h)
        at[t] += h.numel() + gap
        dev.append(v)
    return host, dev, flats


def norm_of(host):
    return math.sqrt(sum(float(h.double().square().sum()) for h in host))


def check_norm(got, host, scale, what):
    want = abs(scale) * norm_of(host)
    # fp64 sums, one rounding to fp32 (and scale's own to fp32).
    assert got.shape == () and abs(float(got) - want) <= want * 3 * ref.U + 2.0 ** -149, (what, float(got), want)


def check_scaled(got, host, scale, max_norm, eps, what):
    c = min(1.0, max_norm / (abs(scale) * norm_of(host) + eps))
    for i, (g, h) in enumerate(zip(got, host)):
        want = h.double() * (scale * c)
        # the norm's, the factor's and scale's roundings, then the product's in fp32 and in the type
        ref.within(g, want, want.abs() * 6 * ref.U + 2.0 ** -150 + ref.half_step(want, h.dtype), f"{what} tensor {i}")


LISTS = {
    "one element": ([1], [F32]),
    "one bf16": ([1], [BF16]),
    "seven": ([7], [F16]),
    "a tile": ([8192], [BF16]),
    "a tile and one": ([4097], [F32]),
    "tile borders": ([8191, 8192, 8193, 16384, 16385], [BF16, F16, BF16, F16, BF16]),
    "16 short tiles": ([512 * 15, 255], [BF16, F32]),
    "17 short tiles": ([512 * 16 + 1], [F16]),
    "64 short tiles": ([512 * 30 + 7, 256 * 20, 100, 512 * 11 + 1], [F16, F32, F32, BF16]),
    "65 short tiles": ([1] * 65, [BF16] * 65),
    "192 short tiles": ([512] * 100 + [256] * 91 + [3], [F16] * 100 + [F32] * 92),
    "192 KiB": ([49152], [F32]),
    "192 KiB and one": ([98305], [BF16]),
    "193 short tiles": ([512] * 193, [BF16] * 193),
    "16 whole tiles": ([4096 * 16], [F32]),
    "17 tiles": ([8192 * 16 + 1], [F16]),
    "16 small ones": ([i % 9 for i in range(1, 17)], [F32, BF16, F16, BF16] * 4),
    "17 small ones": ([i % 8 + 1 for i in range(17)], [F32, BF16, F16] * 5 + [F32, BF16]),
    "empty ones": ([0, 5, 0, 0, 1000, 0], [F32, F32, BF16, F16, BF16, F32]),
    "all empty": ([0, 0], [F32, BF16]),
    "mixed": ([100_003, 17, 65_536, 3, 250_001], [F32, BF16, F16, F32, BF16]),
    "196 tensors": ([600 + i for i in range(196)], [F32, BF16] * 98),
    "197 tensors": ([600 + i for i in range(197)], [F16] * 197),
    "330 tensors": ([5 * i + 1 for i in range(330)], [BF16, F32] * 165),
    "331 tensors": ([9000 - 20 * i for i in range(331)], [F32] * 331),
    "128 tensors": ([i * 7 + 1 for i in range(128)], [F32, BF16] * 64),
    "129 tensors": ([i * 7 for i in range(129)], [BF16] * 129),
    "600 tensors": ([(i * 37) % 900 for i in range(600)], [F32, F16, BF16] * 200),
    "many tiles": ([40_000_001, 11], [BF16, F32]),
}


@pytest.mark.parametrize("gap", [0, 1])
@pytest.mark.parametrize("name", LISTS)
def test_lists(name, gap):
    sizes, types = LISTS[name]
    say(f"gradients {name} gap {gap}")
    host, dev, flats = tensors(sizes, types, 3, gap=gap)
    total = norm_of(host)
    check_norm(rs.grad_norm(dev), host, 1.0, name)
    check_norm(rs.grad_norm(dev, scale=-0.125), host, -0.125, name)
    for scale, top in ((1.0, 0.5 * total + 1e-3), (0.125, 0.01), (1.0, 2 * total + 1)):
        _, outs, out_flats = tensors(sizes, types, 4, gap=gap)
        norm = rs.clip_grads(dev, top, outs=outs, scale=scale)
        check_norm(norm, host, scale, name)
        check_scaled(outs, host, scale, top, 1e-6, f"{name} outs")
        apart, again, _ = tensors(sizes, types, 3, gap=gap)
        rs.scale_grads(dev, norm, top, outs=again, scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(outs, again))
        _, mine, my_flats = tensors(sizes, types, 3, gap=gap)
        assert float(rs.clip_grads(mine, top, scale=scale)) == float(norm)
        assert all(torch.equal(a, b) for a, b in zip(outs, mine))
        if gap:  # nothing between the tensors is written
            for fl, views in ((out_flats, outs), (my_flats, mine)):
                for v in views:
                    v.fill_(7.0)
                assert all(bool((f == 7.0).all()) for f in fl.values())
    assert all(torch.equal(d.cpu(), h) for d, h in zip(dev, host)), "gradients changed"


def test_no_tensors():
    assert float(rs.grad_norm([])) == 0.0
    assert float(rs.clip_grads([], 1.0)) == 0.0


def test_shapes_and_given_norm():
    g = [torch.ones(3, 4, 5, device=DEV), torch.ones((), device=DEV, dtype=BF16)]
    norm = torch.zeros(1, device=DEV)
    assert rs.grad_norm(g, norm=norm) is norm and abs(float(norm) - math.sqrt(61)) < 1e-5
    assert rs.clip_grads(g, 1e9, norm=norm) is norm
    assert float(g[0].sum()) == 60.0


def test_inactive_clipping_changes_no_bit():
    host, dev, _ = tensors([1000, 333], [F32, BF16], 1)
    rs.clip_grads(dev, 1e6)
    assert all(torch.equal(d.cpu(), h) for d, h in zip(dev, host))
    outs = [torch.zeros_like(d) for d in dev]
    rs.clip_grads(dev, 1e6, outs=outs)
    assert all(torch.equal(d.cpu(), h) for d, h in zip(outs, host))


def test_values_whose_squares_leave_fp32():
    """Squares above 2^128 and below 2^-149, and the largest value."""
    for v, n in ((1e30, 1000), (1e-30, 1000), (2.0 ** -149, 4096), (torch.finfo(F32).max, 1)):
        t = torch.full((n,), v, device=DEV)
        want = float(t[:1].double()) * math.sqrt(n)
        assert abs(float(rs.grad_norm([t])) - want) <= want * 2 * ref.U, v
    t = torch.full((4,), 3e38, device=DEV)  # the norm itself is beyond fp32
    assert float(rs.grad_norm([t])) == math.inf
    big = torch.full((1000,), 1e30, device=DEV)
    rs.clip_grads([big], 1.0)
    assert abs(float(big.double().square().sum().sqrt()) - 1.0) < 1e-5


def test_more_than_2_to_the_31_elements():
    """One tensor of 2^31 + 9 elements: its norm, and what is written at its
    start, at its end and where 32 bits wrap."""
    n = (1 << 31) + 9
    t = torch.full((n,), 0.5, dtype=BF16, device=DEV)
    t[-1] = 256.0
    want = math.sqrt(0.25 * (n - 1) + 65536.0)
    assert abs(float(rs.grad_norm([t])) - want) <= want * 2 * ref.U
    norm = rs.clip_grads([t], want / 2, eps=0.0)
    assert abs(float(norm) - want) <= want * 2 * ref.U
    assert float(t[-1]) == 128.0
    for lo in (0, (1 << 30) - 50, (1 << 31) - 50, n - 101):
        assert bool((t[lo:min(lo + 100, n - 1)] == 0.25).all()), lo
    assert abs(float(rs.grad_norm([t])) - want / 2) <= want * 2 * ref.U


def test_special_values():
    """An infinite norm leaves 0 in finite places and NaN in infinite ones; a
    NaN norm makes everything NaN."""
    for dtype in (F32, BF16, F16):
        a, b = torch.ones(100, dtype=dtype, device=DEV), torch.ones(9000, dtype=dtype, device=DEV)
        b[8500] = -math.inf
        assert float(rs.clip_grads([a, b], 1.0)) == math.inf
        assert not a.any() and int(torch.isnan(b).sum()) == 1 and bool(torch.isnan(b[8500]))
        a, b = torch.ones(100, dtype=dtype, device=DEV), torch.ones(9000, dtype=dtype, device=DEV)
        b[1] = math.nan
        assert math.isnan(float(rs.grad_norm([a, b])))
        assert math.isnan(float(rs.clip_grads([a, b], 1.0)))
        assert bool(torch.isnan(a).all()) and bool(torch.isnan(b).all())
    zeros = torch.zeros(50, device=DEV)
    assert float(rs.clip_grads([zeros], 1.0)) == 0.0 and not zeros.any()


def test_same_bits_every_time():
    _, dev, _ = tensors([1_000_001, 77, 500_000], [BF16, F32, F16], 9)
    first = rs.grad_norm(dev)
    for _ in range(5):
        assert torch.equal(rs.grad_norm(dev), first)


def test_norm_of_shards_is_the_norm_of_the_whole():
    """After a reduce-scatter every rank holds one block: the blocks of all
    ranks give the norm of the whole gradient."""
    n, ranks = 10_000, 4
    gen = torch.Generator().manual_seed(2)
    send = [torch.empty(ranks * n).normal_(generator=gen).to(DEV) for _ in range(ranks)]
    recv = [torch.empty(n, device=DEV) for _ in range(ranks)]
    comm = rs.comm_init(ranks, 2)
    try:
        rs.reduce_scatter(comm, send, recv)
        got = rs.grad_norm(recv, scale=1.0 / ranks)
        torch.cuda.synchronize()
    finally:
        rs.comm_destroy(comm)
    check_norm(got, [r.cpu() for r in recv], 1.0 / ranks, "shards")


def test_on_another_stream():
    side = torch.cuda.Stream()
    host, dev, _ = tensors([100_000, 31], [F32, BF16], 5)
    side.wait_stream(torch.cuda.current_stream())
    a = rs.grad_norm(dev, stream=side)
    b = rs.grad_norm(dev, stream=side.cuda_stream)
    c = rs.clip_grads(dev, 0.1, stream=side)
    side.synchronize()
    for got in (a, b, c):
        check_norm(got, host, 1.0, "side stream")
    check_scaled(dev, host, 1.0, 0.1, 1e-6, "side stream")


def test_captured_into_a_graph():
    """Every replay on new gradients equals the eager calls on them."""
    sizes, types = [70_001, 8, 0, 123_456], [BF16, F32, F32, F16]
    _, dev, flats = tensors(sizes, types, 1)
    outs = [torch.empty_like(d) for d in dev]
    rs.clip_grads(dev, 1.0, outs=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n1 = rs.grad_norm(dev, scale=0.5)
        n2 = rs.clip_grads(dev, 1.0, outs=outs)
    for seed in range(5):
        _, new, _ = tensors(sizes, types, 20 + seed, std=0.01 * (seed + 1))
        for d, x in zip(dev, new):
            d.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n1, rs.grad_norm(dev, scale=0.5))
        eager = [torch.empty_like(d) for d in dev]
        assert torch.equal(n2, rs.clip_grads(dev, 1.0, outs=eager))
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        torch.cuda.synchronize()


def test_binding_refuses_on_device():
    g = torch.ones(8, 8, device=DEV)
    for bad in ([g.t()[:, :4]], [g.cpu()], [g, g.cpu()]):
        with pytest.raises(ValueError):
            rs.grad_norm(bad)
    with pytest.raises(TypeError):
        rs.grad_norm([g.double()])
    for outs in ([], [g.bfloat16()], [g[:4]], [g, g]):
        with pytest.raises(ValueError):
            rs.clip_grads([g], 1.0, outs=outs)
    with pytest.raises(ValueError):
        rs.scale_grads([g], torch.ones(2, device=DEV), 1.0)
    for kw in (dict(scale=math.inf), dict(eps=-1.0)):
        with pytest.raises(rs.RingsimError):
            rs.clip_grads([g], 1.0, **kw)
    for top in (-1.0, math.nan, math.inf):
        with pytest.raises(rs.RingsimError):
            rs.clip_grads([g], top)
