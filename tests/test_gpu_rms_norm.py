"""rms_norm and rms_norm_backward on the device against the formulas in 64
bits: types, odd and ragged sizes, strides, single tokens, 8-bit outputs,
special values, streams and graphs."""
import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests import _ops_ref as ref
from tests._gpu import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
# Columns on both sides of every border: of a lane's 16 bytes, of the lanes a
# row takes (powers of two from 64 on), of whole waves, and the limit.
COLS = (1, 2, 3, 4, 5, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 512, 513, 1024, 1025, 1600, 2047, 2048,
        2049, 4096, 4097, 5119, 8192, 8193, 12300, 16384, 16385, 24576, 32767, 32768)


def make(shape, dtype, seed, std=1.0, pad=0, offset=0):
    """Host values and a device tensor of them: rows `pad` elements apart, the
    first `offset` elements into its memory."""
    gen = torch.Generator().manual_seed(seed)
    host = torch.empty(shape).normal_(0.0, std, generator=gen).to(dtype)
    rows, width = 1, shape[-1]
    for s in shape[:-1]:
        rows *= s
    flat = torch.full((offset + rows * (width + pad),), 3.0, dtype=dtype, device=DEV)
    t = flat[offset:].view(rows, width + pad)[:, :width]
    t.copy_(host.view(rows, width))
    if pad == 0:
        return host, t.view(shape)
    if len(shape) == 1:
        return host, t[0]
    return host, t.unflatten(0, shape[:-1]) if len(shape) > 2 else t


def weight_of(kind, cols, dtype, seed):
    if kind == "none":
        return None, None
    w = torch.empty(cols).normal_(1.0, 0.3, generator=torch.Generator().manual_seed(seed))
    w = w.to(torch.float32 if kind == "f32" else dtype)
    return w, w.to(DEV)


def check_norm(got, x, residual, w, eps, what):
    h, _, y = ref.norm(x, residual, w, eps)
    ref.within(got.out, y, y.abs() * ref.Y_REL + ref.half_step(y, x.dtype), what + " out")
    if residual is None:
        assert got.residual is None
    else:
        ref.within(got.residual, h, h.abs() * ref.U + ref.half_step(h, x.dtype), what + " residual")
    assert got.scales is None


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("name", DTYPES)
def test_norm_sizes_and_types(name, cols):
    dtype = DTYPES[name]
    for rows, kind, with_residual, pad, offset in ((1, "same", True, 0, 0), (3, "f32", False, 1, 1), (5, "none", True, 8, 0)):
        what = f"norm {name} {rows}x{cols} weight {kind} residual {with_residual} pad {pad} offset {offset}"
        say(what)
        x, xd = make((rows, cols), dtype, cols, pad=pad, offset=offset)
        r, rd = make((rows, cols), dtype, cols + 1, 2.0) if with_residual else (None, None)
        w, wd = weight_of(kind, cols, dtype, 7)
        got = rs.rms_norm(xd, wd, residual=rd, eps=EPS)
        check_norm(got, x, r, w, EPS, what)


@pytest.mark.parametrize("rows, cols", [(1000, 64), (4097, 130), (2500, 1000), (1111, 4100), (700, 9000)])
def test_norm_many_rows(rows, cols):
    """More rows than the launch has workgroups for at once."""
    for name in ("bf16", "f32"):
        say(f"norm {name} {rows}x{cols}")
        x, xd = make((rows, cols), DTYPES[name], rows, pad=3)
        w, wd = weight_of("same", cols, DTYPES[name], 3)
        check_norm(rs.rms_norm(xd, wd, eps=EPS), x, None, w, EPS, f"{rows}x{cols}")


def test_norm_heads_inside_a_wider_row():
    """[tokens, heads, 128] views of rows that hold more heads; the output's
    strides are another tensor's."""
    x = torch.empty(37, 12, 128).normal_(generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    wide = x.to(DEV)
    w, wd = weight_of("f32", 128, torch.bfloat16, 2)
    for lo, hi in ((0, 8), (8, 10), (11, 12)):
        out = torch.full((37, 16, 160), 9.0, dtype=torch.bfloat16, device=DEV)
        view = out[:, 2:2 + hi - lo, 16:144]
        got = rs.rms_norm(wide[:, lo:hi], wd, eps=EPS, out=view)
        check_norm(got, x[:, lo:hi], None, w, EPS, f"heads {lo}:{hi}")
        out[:, 2:2 + hi - lo, 16:144] = 9.0
        assert bool((out == 9.0).all()), "written outside the view"
    by_head = wide.transpose(0, 1)  # [heads, tokens, 128]
    got = rs.rms_norm(by_head, wd, eps=EPS)
    check_norm(got, x.transpose(0, 1), None, w, EPS, "transposed heads")


def test_norm_of_a_vector_and_of_four_dimensions():
    x, xd = make((640,), torch.float16, 5)
    check_norm(rs.rms_norm(xd, eps=EPS), x, None, None, EPS, "1-d")
    x, xd = make((2, 3, 5, 72), torch.float32, 6)
    check_norm(rs.rms_norm(xd, eps=EPS), x, None, None, EPS, "4-d")


def test_norm_in_place():
    for name, dtype in DTYPES.items():
        x, xd = make((33, 777), dtype, 1)
        r, rd = make((33, 777), dtype, 2)
        w, wd = weight_of("same", 777, dtype, 3)
        got = rs.rms_norm(xd, wd, residual=rd, eps=EPS, out=xd, residual_out=rd)
        assert got.out.data_ptr() == xd.data_ptr() and got.residual.data_ptr() == rd.data_ptr()
        check_norm(got, x, r, w, EPS, f"in place {name}")


def check_quant(got, x, residual, w, eps, group, what):
    h, _, y = ref.norm(x, residual, w, eps)
    s = ref.scales(y, group)
    ref.within(got.scales, s, s * (ref.Y_REL + 2 * ref.U) + 2.0 ** -149, what + " scales")
    width = group or y.shape[-1]
    spread = got.scales.double().cpu().repeat_interleave(width, -1)[..., :y.shape[-1]]
    stands_for = got.out.cpu().float().double() * spread
    # Half a step of e4m3: 2^-4 of the value, or half its smallest subnormal (2^-9) in units of the scale.
    bound = y.abs() * (2.0 ** -4 * (1 + 4 * ref.U) + ref.Y_REL) + spread * 2.0 ** -10 * (1 + 4 * ref.U)
    ref.within(stands_for, y, bound, what + " q")
    if residual is not None:
        ref.within(got.residual, h, h.abs() * ref.U + ref.half_step(h, x.dtype), what + " residual")


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("name", DTYPES)
def test_norm_in_8_bits(name, group):
    dtype = DTYPES[name]
    for rows, cols, pad in ((1, 4096, 0), (3, 1, 0), (5, 31, 1), (4, 33, 0), (7, 128, 8), (2, 1000, 0), (9, 2050, 3),
                            (2, 8200, 0), (1, 32767, 0), (3000, 96, 0)):
        what = f"8 bits {name} {rows}x{cols} group {group} pad {pad}"
        say(what)
        x, xd = make((rows, cols), dtype, cols, pad=pad)
        r, rd = make((rows, cols), dtype, cols + 1) if rows != 5 else (None, None)
        w, wd = weight_of("f32" if rows == 9 else "same", cols, dtype, 4)
        got = rs.rms_norm(xd, wd, residual=rd, eps=EPS, out_dtype="float8_e4m3", group=group)
        assert got.out.dtype is torch.float8_e4m3fn
        check_quant(got, x, r, w, EPS, group, what)
        again = rs.rms_norm(xd, wd, residual=rd, eps=EPS, out_dtype=torch.float8_e4m3fn, group=group)
        assert torch.equal(again.out.view(torch.uint8), got.out.view(torch.uint8))


def test_8_bit_rounding_is_to_nearest_even():
    """A row of magnitude one and no weight: q = y / scale exactly as torch
    rounds it, ties included (y * 448 / max is exact for these values)."""
    v = torch.arange(0, 449, dtype=torch.float32) / 448.0
    v = torch.cat([v, -v])
    x = v.to(DEV).reshape(1, -1)
    w = torch.full((v.numel(),), 448.0, device=DEV)
    got = rs.rms_norm(x, w, eps=0.0, out_dtype="float8_e4m3")
    y = rs.rms_norm(x, w, eps=0.0).out
    inv = 1.0 / got.scales
    assert torch.equal(got.out.float(), (y * inv).to(torch.float8_e4m3fn).float())


def test_zero_rows_and_rows_of_zeros():
    for name, dtype in DTYPES.items():
        got = rs.rms_norm(torch.empty(0, 64, dtype=dtype, device=DEV), torch.ones(64, dtype=dtype, device=DEV))
        assert got.out.shape == (0, 64)
        x = torch.zeros(4, 200, dtype=dtype, device=DEV)
        assert not rs.rms_norm(x, eps=EPS).out.any()
        got = rs.rms_norm(x, eps=EPS, out_dtype="float8_e4m3", group=64)
        assert not got.out.float().any() and bool((got.scales == 2.0 ** -126).all())
        got = rs.rms_norm_backward(x[:0], x[:0], torch.ones(200, dtype=dtype, device=DEV))
        assert got.grad_in.shape == (0, 200) and not got.grad_weight.any()


def test_special_values_stay_in_their_rows():
    """A NaN makes its row NaN; an infinity makes its place NaN and the other
    places 0; other rows are untouched. 8-bit scales of a NaN are NaN."""
    inf, nan = float("inf"), float("nan")
    for name, dtype in DTYPES.items():
        x, xd = make((6, 300), dtype, 11)
        for t in (x, xd):
            t[1, 17] = nan
            t[2, 299] = inf
            t[3, 0] = -inf
        w, wd = weight_of("same", 300, dtype, 1)
        check_norm(rs.rms_norm(xd, wd, eps=EPS), x, None, w, EPS, f"special {name}")
        got = rs.rms_norm(xd, wd, eps=EPS, out_dtype="float8_e4m3", group=128)
        q, s = got.out.float().cpu(), got.scales.cpu()
        assert bool(torch.isnan(q[1]).all()) and bool(torch.isnan(s[1]).all())
        assert torch.isnan(s[2]).tolist() == [False, False, True]
        assert not q[2, :256].any() and bool(torch.isnan(q[2, 256:]).all())
        assert torch.isnan(s[3]).tolist() == [True, False, False]
        for row in (0, 4, 5):
            assert bool(torch.isfinite(q[row]).all())


def test_large_and_small_values():
    for scale, eps in ((1e17, EPS), (1e-15, 0.0), (3e4, EPS)):
        x = (torch.empty(3, 1500).normal_(generator=torch.Generator().manual_seed(1)) * scale)
        got = rs.rms_norm(x.to(DEV), eps=eps)
        check_norm(got, x, None, None, eps, f"scale {scale}")


# ---------------------------------------------------------------------------
# Backward
# ---------------------------------------------------------------------------


def check_backward(got, dy, h, w, res, eps, what):
    dx, dw, bound, terms = ref.backward(dy, h, w, res, eps)
    ref.within(got.grad_in, dx, bound + ref.half_step(dx, h.dtype), what + " grad_in")
    if w is None:
        assert got.grad_weight is None
        return
    # A column's sum is a chain over rows and workgroups of at most rows + 64 additions,
    # its terms off by r's error and two products.
    rows = h.numel() // h.shape[-1]
    ref.within(got.grad_weight, dw, terms * (rows + 64 + ref.SUM / 2 + 8) * ref.U + ref.half_step(dw, w.dtype),
               what + " grad_weight")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("name", DTYPES)
def test_backward_sizes_and_types(name, cols):
    dtype = DTYPES[name]
    for rows, kind, with_residual, pad, offset in ((1, "same", True, 0, 0), (3, "f32", False, 1, 1), (6, "none", True, 8, 0)):
        what = f"backward {name} {rows}x{cols} weight {kind} residual {with_residual} pad {pad} offset {offset}"
        say(what)
        h, hd = make((rows, cols), dtype, cols, pad=pad, offset=offset)
        dy, dyd = make((rows, cols), dtype, cols + 1, 0.1)
        r, rd = make((rows, cols), dtype, cols + 2, 0.1, pad=pad) if with_residual else (None, None)
        w, wd = weight_of(kind, cols, dtype, 7)
        check_backward(rs.rms_norm_backward(dyd, hd, wd, grad_residual=rd, eps=EPS), dy, h, w, r, EPS, what)


@pytest.mark.parametrize("rows, cols", [(9000, 64), (5000, 130), (3000, 1000), (2777, 2100), (1111, 4100), (700, 9000),
                                        (530, 17000)])
def test_backward_many_rows(rows, cols):
    for name, kind in (("bf16", "same"), ("f32", "same"), ("f16", "f32")):
        say(f"backward {name} {rows}x{cols}")
        h, hd = make((rows, cols), DTYPES[name], rows, pad=3)
        dy, dyd = make((rows, cols), DTYPES[name], rows + 1, 0.1)
        w, wd = weight_of(kind, cols, DTYPES[name], 3)
        got = rs.rms_norm_backward(dyd, hd, wd, eps=EPS)
        check_backward(got, dy, h, w, None, EPS, f"{name} {rows}x{cols}")
        again = rs.rms_norm_backward(dyd, hd, wd, eps=EPS)
        assert torch.equal(again.grad_weight, got.grad_weight) and torch.equal(again.grad_in, got.grad_in)


@pytest.mark.parametrize("cols", [5, 100, 128, 500, 1000, 2000, 4096, 8000, 16000, 30000])
def test_backward_few_rows(cols):
    """Row counts on both sides of the border below which one workgroup takes
    all rows (4 turns of 16, 4 or 1 rows)."""
    for rows in (1, 2, 4, 5, 15, 16, 17, 63, 64, 65):
        for name, kind in (("bf16", "same"), ("f16", "f32"), ("f32", "same")):
            say(f"backward {name} {rows}x{cols} weight {kind}")
            h, hd = make((rows, cols), DTYPES[name], rows)
            dy, dyd = make((rows, cols), DTYPES[name], rows + 1, 0.1)
            w, wd = weight_of(kind, cols, DTYPES[name], 3)
            check_backward(rs.rms_norm_backward(dyd, hd, wd, eps=EPS), dy, h, w, None, EPS, f"{name} {rows}x{cols}")


@pytest.mark.parametrize("cols", [8193, 12296, 16384, 16385, 20003, 32768])
def test_backward_wide_rows(cols):
    """Rows on 1024 lanes, which load the next row while they write one: one to
    three turns a workgroup, with and without the weight and the residual's
    gradient, results in place of each input."""
    for rows in (4, 257, 600):
        for name, kind, target in (("bf16", "same", "grad_residual"), ("f16", "f32", "h"), ("f32", "none", "grad_out"),
                                   ("f32", "same", "grad_residual"), ("bf16", "none", None), ("f32", "same", None)):
            what = f"backward {name} {rows}x{cols} weight {kind} into {target}"
            say(what)
            h, hd = make((rows, cols), DTYPES[name], rows)
            dy, dyd = make((rows, cols), DTYPES[name], rows + 1, 0.1)
            r, rd = make((rows, cols), DTYPES[name], rows + 2, 0.1) if target else (None, None)
            w, wd = weight_of(kind, cols, DTYPES[name], 3)
            into = {"grad_out": dyd, "h": hd, "grad_residual": rd, None: None}[target]
            got = rs.rms_norm_backward(dyd, hd, wd, grad_residual=rd, eps=EPS, grad_in=into)
            check_backward(got, dy, h, w, r, EPS, what)


@pytest.mark.parametrize("rows, cols", [(2048, 4100), (2049, 4104), (2049, 4097), (2100, 5121), (2600, 6144), (2100, 6145)])
def test_backward_three_packs(rows, cols):
    """Both sides of the borders of rows on three or four waves."""
    for name, kind, with_residual in (("bf16", "same", True), ("f16", "f32", False)):
        what = f"backward {name} {rows}x{cols} weight {kind} residual {with_residual}"
        say(what)
        h, hd = make((rows, cols), DTYPES[name], rows, pad=1)
        dy, dyd = make((rows, cols), DTYPES[name], rows + 1, 0.1)
        r, rd = make((rows, cols), DTYPES[name], rows + 2, 0.1) if with_residual else (None, None)
        w, wd = weight_of(kind, cols, DTYPES[name], 3)
        check_backward(rs.rms_norm_backward(dyd, hd, wd, grad_residual=rd, eps=EPS), dy, h, w, r, EPS, what)


def test_backward_heads_and_in_place():
    h = torch.empty(37, 12, 128).normal_(generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    dy = torch.empty(37, 8, 128).normal_(generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    w, wd = weight_of("f32", 128, torch.bfloat16, 2)
    hd, dyd = h.to(DEV), dy.to(DEV)
    got = rs.rms_norm_backward(dyd, hd[:, 2:10], wd, eps=EPS)
    check_backward(got, dy, h[:, 2:10], w, None, EPS, "heads")
    for target in ("grad_out", "h", "grad_residual"):
        t = {"grad_out": dy.to(DEV), "h": h[:, 2:10].contiguous().to(DEV), "grad_residual": dy.flip(0).to(DEV)}
        got = rs.rms_norm_backward(t["grad_out"], t["h"], wd, grad_residual=t["grad_residual"], eps=EPS, grad_in=t[target])
        assert got.grad_in.data_ptr() == t[target].data_ptr()
        check_backward(got, dy, h[:, 2:10], w, dy.flip(0), EPS, f"into {target}")


def test_backward_without_the_weights_gradient():
    h, hd = make((40, 1030), torch.bfloat16, 1)
    dy, dyd = make((40, 1030), torch.bfloat16, 2)
    w, wd = weight_of("same", 1030, torch.bfloat16, 3)
    got = rs.rms_norm_backward(dyd, hd, wd, eps=EPS, need_grad_weight=False)
    assert got.grad_weight is None
    dx, _, bound, _ = ref.backward(dy, h, w, None, EPS)
    ref.within(got.grad_in, dx, bound + ref.half_step(dx, h.dtype), "grad_in")
    buf = torch.full((1030,), 5.0, dtype=torch.bfloat16, device=DEV)
    got = rs.rms_norm_backward(dyd, hd, wd, eps=EPS, grad_weight=buf)
    assert got.grad_weight.data_ptr() == buf.data_ptr()
    check_backward(got, dy, h, w, None, EPS, "overwrites")


def test_backward_against_differences():
    """Directional differences of the forward formula in 64 bits: for a loss
    sum(dy * y), (loss(h + t v) - loss(h - t v)) / 2t is <grad_in, v>, and the
    same for the weight. Central differences are off by t^2 times the third
    derivative, here below 1e-8 of the sums of magnitudes; fp32 gradients by
    their own bound."""
    h, hd = make((19, 333), torch.float32, 1)
    dy, dyd = make((19, 333), torch.float32, 2)
    w, wd = weight_of("same", 333, torch.float32, 3)
    got = rs.rms_norm_backward(dyd, hd, wd, eps=EPS)
    _, _, bound, terms = ref.backward(dy, h, w, None, EPS)

    def loss(hh, ww):
        y = hh / torch.sqrt(hh.square().mean(-1, keepdim=True) + EPS) * ww
        return float((dy.double() * y).sum())

    t = 1e-5
    for seed in range(4):
        gen = torch.Generator().manual_seed(seed)
        v = torch.empty(19, 333, dtype=torch.float64).normal_(generator=gen)
        u = torch.empty(333, dtype=torch.float64).normal_(generator=gen)
        dh = (loss(h.double() + t * v, w.double()) - loss(h.double() - t * v, w.double())) / (2 * t)
        prod = got.grad_in.double().cpu() * v
        slack = float(((bound + ref.half_step(got.grad_in.double().cpu(), torch.float32)) * v.abs()).sum())
        assert abs(float(prod.sum()) - dh) <= slack + 1e-6 * float(prod.abs().sum())
        dw = (loss(h.double(), w.double() + t * u) - loss(h.double(), w.double() - t * u)) / (2 * t)
        prod = got.grad_weight.double().cpu() * u
        slack = float((terms * 128 * ref.U * u.abs()).sum())
        assert abs(float(prod.sum()) - dw) <= slack + 1e-6 * float(prod.abs().sum())


def test_backward_special_values_stay_in_their_rows():
    """What a NaN or an infinity does to its row's gradient and to the columns
    of the weight's is the formula's; other rows are untouched."""
    for name, dtype in DTYPES.items():
        for cols in (300, 2000):
            h, hd = make((6, cols), dtype, 11)
            dy, dyd = make((6, cols), dtype, 12)
            w, wd = weight_of("same", cols, dtype, 1)
            for t in (h, hd):
                t[1, 17] = float("nan")
                t[2, cols - 1] = float("inf")
            for t in (dy, dyd):
                t[4, 3] = float("-inf")
            got = rs.rms_norm_backward(dyd, hd, wd, eps=EPS)
            dx, _, bound, _ = ref.backward(dy, h, w, None, EPS)
            keep = [0, 3, 5]
            ref.within(got.grad_in[keep], dx[keep], bound[keep] + ref.half_step(dx[keep], dtype), f"{name} other rows")
            for row in (1, 2, 4):
                assert not bool(torch.isfinite(got.grad_in[row]).any()), (name, row)
            assert bool(torch.isnan(got.grad_weight).all())  # row 1's root is NaN in every column


def test_rows_beyond_32_bit_offsets():
    """Rows more than 2^31 elements into their memory."""
    far = 1_200_000_000
    for name, kind in (("bf16", "same"),):
        dtype = DTYPES[name]
        flat = torch.zeros(2 * far + 4096, dtype=dtype, device=DEV)
        x, xd = make((3, 1000), dtype, 1)
        r, rd = make((3, 1000), dtype, 2)
        view = flat.as_strided((3, 1000), (far, 1))
        view.copy_(xd)
        w, wd = weight_of(kind, 1000, dtype, 3)
        got = rs.rms_norm(view, wd, residual=rd, eps=EPS, residual_out=view)
        check_norm(got, x, r, w, EPS, "far rows")
        view.copy_(xd)
        back = rs.rms_norm_backward(rd, view, wd, eps=EPS, grad_in=view)
        check_backward(back, r, x, w, None, EPS, "far rows")
        heads = flat.as_strided((3, 5, 128), (far, 200, 1))
        y, yd = make((3, 5, 128), dtype, 4)
        heads.copy_(yd)
        check_norm(rs.rms_norm(heads, None, eps=EPS, out=heads), y, None, None, EPS, "far heads")


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------


def test_on_another_stream():
    side = torch.cuda.Stream()
    x, xd = make((64, 2048), torch.bfloat16, 1)
    w, wd = weight_of("same", 2048, torch.bfloat16, 2)
    side.wait_stream(torch.cuda.current_stream())
    got = [rs.rms_norm(xd, wd, eps=EPS, stream=side), rs.rms_norm(xd, wd, eps=EPS, stream=side.cuda_stream)]
    back = rs.rms_norm_backward(xd, got[0].out, wd, eps=EPS, stream=side)
    side.synchronize()
    for g in got:
        check_norm(g, x, None, w, EPS, "side stream")
    check_backward(back, x, got[0].out.cpu(), w, None, EPS, "side stream")


def test_captured_into_a_graph():
    """Forward and backward captured together; every replay on new values
    equals the eager calls on them."""
    x, r, dy = (torch.zeros(130, 1500, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    w = torch.ones(1500, dtype=torch.bfloat16, device=DEV)

    def step():
        f = rs.rms_norm(x, w, residual=r, eps=EPS)
        q = rs.rms_norm(x, w, residual=r, eps=EPS, out_dtype="float8_e4m3", group=128)
        b = rs.rms_norm_backward(dy, f.residual, w, grad_residual=r, eps=EPS)
        return [f.out, f.residual, q.out.view(torch.uint8), q.scales, b.grad_in, b.grad_weight]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(5):
        for i, t in enumerate((x, r, dy)):
            t.copy_(make((130, 1500), torch.bfloat16, 10 * seed + i)[1])
        w.copy_(weight_of("same", 1500, torch.bfloat16, seed)[1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b), seed
        torch.cuda.synchronize()


def test_binding_refuses_on_device():
    x = torch.zeros(4, 64, device=DEV)
    with pytest.raises(ValueError):
        rs.rms_norm(x.t())
    with pytest.raises(ValueError):
        rs.rms_norm(x, residual=x[:2])
    with pytest.raises(TypeError):
        rs.rms_norm(x, residual=x.bfloat16())
    with pytest.raises(ValueError):
        rs.rms_norm(x, torch.ones(64))  # weight on the host
    with pytest.raises(ValueError):
        rs.rms_norm(x, residual_out=x)
    with pytest.raises(ValueError):
        rs.rms_norm(x, out_dtype="float8_e4m3", scales=torch.zeros(4, 2, device=DEV))
    with pytest.raises(rs.RingsimError):
        rs.rms_norm(x, eps=-1.0)
    with pytest.raises(rs.RingsimError):
        rs.rms_norm(torch.zeros(1, 40000, device=DEV))
    with pytest.raises(rs.RingsimError):
        rs.rms_norm(x, out=torch.zeros(1, 64, device=DEV).expand(4, 64))
    with pytest.raises(ValueError):
        rs.rms_norm(torch.zeros(2, 3, 2, 2, 128, device=DEV)[:, :2])  # leading dimensions with a gap
    with pytest.raises(ValueError):
        rs.rms_norm_backward(x, x, None, grad_weight=torch.zeros(64, device=DEV))
