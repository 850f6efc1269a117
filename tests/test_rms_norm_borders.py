"""The norm and its gradients where their launches change: two short rows a
group of lanes, inputs beyond the Infinity Cache, grids of two dimensions, and
row counts that one workgroup takes. Large cases are compared on the device,
with the formulas in 64 bits by torch."""
import ctypes
import os

import numpy as np
import pytest
import torch

from ring_all_reduce_allreduce_amd import build

if not (os.path.exists(build.LIB) and os.path.exists(build.BINDING)):
    build.build()
import ring_all_reduce_allreduce_amd as rs  # noqa: E402
from tests import _ops_ref as ref  # noqa: E402
from tests._gpu import say  # noqa: E402

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"f32": 2, "bf16": 3, "f16": 16}
MiB = 1 << 20

#: Rows from which on a group of 16, 32 and 64 lanes takes two, with columns
#: of such rows (of 16-bit types; half of them in fp32): whole packs, odd ones
#: and rows shorter than a pack.
TWO_ROWS = [(32768, 128), (32768, 101), (32768, 3), (16384, 256), (16384, 203), (8192, 512), (8192, 491)]


def random(shape, dtype, seed, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


def inside(got, want, bound, what):
    off = (got.double() - want).abs() - bound
    assert bool((off <= 0).all()), f"{what}: {float(off.max())} beyond the bound, {int((off > 0).sum())} elements"


def check_norm(got, x, residual, w, what, rows=1 << 16):
    """In pieces of `rows` rows."""
    for lo in range(0, x.shape[0], rows):
        s = slice(lo, lo + rows)
        h, _, y = ref.norm(x[s], None if residual is None else residual[s], w, EPS)
        inside(got.out[s], y, y.abs() * ref.Y_REL + ref.half_step(y, x.dtype), what + " out")
        if residual is not None:
            inside(got.residual[s], h, h.abs() * ref.U + ref.half_step(h, x.dtype), what + " residual")


def check_quant(got, x, residual, w, group, what):
    _, _, y = ref.norm(x, residual, w, EPS)
    s = ref.scales(y, group)
    inside(got.scales, s, s * (ref.Y_REL + 2 * ref.U) + 2.0 ** -149, what + " scales")
    spread = got.scales.double().repeat_interleave(group or y.shape[-1], -1)[..., :y.shape[-1]]
    bound = y.abs() * (2.0 ** -4 * (1 + 4 * ref.U) + ref.Y_REL) + spread * 2.0 ** -10 * (1 + 4 * ref.U)
    inside(got.out.float().double() * spread, y, bound, what + " q")


def check_grad_in(got, dy, h, w, residual, what, rows=1 << 16):
    for lo in range(0, h.shape[0], rows):
        s = slice(lo, lo + rows)
        dx, _, bound, _ = ref.backward(dy[s], h[s], w, None if residual is None else residual[s], EPS)
        inside(got[s], dx, bound + ref.half_step(dx, h.dtype), what + " grad_in")


# ---------------------------------------------------------------------------
# Forward
# ---------------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("border, cols", TWO_ROWS)
@pytest.mark.parametrize("name", DTYPES)
def test_norm_two_rows_a_group(name, border, cols):
    """Below, at and above the border; the last pair is ragged above it."""
    dtype = DTYPES[name]
    cols = cols if dtype != torch.float32 else (cols + 1) // 2
    w = random(cols, torch.float32, 1, 0.3) + 1.0
    for rows in (border - 1, border, border + 1, border + 37):
        what = f"norm {name} {rows}x{cols}"
        say(what)
        x, r = random((rows, cols), dtype, rows), random((rows, cols), dtype, rows + 1, 2.0)
        check_norm(rs.rms_norm(x, w, eps=EPS), x, None, w, what)
        xi, ri = x.clone(), r.clone()
        got = rs.rms_norm(xi, w.to(dtype), residual=ri, eps=EPS, out=xi, residual_out=ri)
        check_norm(got, x, r, w.to(dtype), what + " in place")
        for group in (0, 32, 128):
            got = rs.rms_norm(x, None, residual=r, eps=EPS, out_dtype="float8_e4m3", group=group)
            check_quant(got, x, r, None, group, f"{what} into 8 bits, group {group}")
        # Rows by themselves: the same arithmetic on one row a group.
        part = rs.rms_norm(x[rows - 50:], w, eps=EPS)
        assert torch.equal(part.out, rs.rms_norm(x, w, eps=EPS).out[rows - 50:])


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1023, 1024, 1025])
def test_norm_heads_two_rows_a_group(tokens):
    """Heads inside wider rows, into heads inside wider rows."""
    wide, out = random((tokens, 48, 128), torch.bfloat16, 3), random((tokens, 40, 130), torch.bfloat16, 4)
    kept = out.clone()
    w = random(128, torch.float32, 1, 0.3) + 1.0
    x, o = wide[:, 8:40], out[:, 1:33, 1:129]
    got = rs.rms_norm(x, w, eps=EPS, out=o)
    check_norm(got, x, None, w, f"heads of {tokens} tokens")
    o.copy_(kept[:, 1:33, 1:129])
    assert torch.equal(out, kept), "written outside the view"


#: Columns of every layout of a row; in fp32 half of them, and 32765 as well.
LAYOUTS = (125, 250, 509, 1021, 2045, 4099, 8187, 16381, 32765)


def beyond_the_cache(cols, size, tensors):
    """Rows of which a call moves a little more than 256 MiB."""
    return 256 * MiB // (cols * size * tensors) + 3


@pytest.mark.gpu
@pytest.mark.parametrize("cols", LAYOUTS)
@pytest.mark.parametrize("name", DTYPES)
def test_norm_beyond_the_cache(name, cols):
    dtype = DTYPES[name]
    widths = (cols,) if dtype != torch.float32 else ((cols + 1) // 2, 32765) if cols == LAYOUTS[-1] else ((cols + 1) // 2,)
    for c in widths:
        w = random(c, dtype, 1, 0.3) + 1.0
        for tensors in (2, 4):
            rows = beyond_the_cache(c, dtype.itemsize, tensors)
            what = f"norm {name} {rows}x{c} of {tensors} tensors"
            say(what)
            x = random((rows, c), dtype, c)
            r = random((rows, c), dtype, c + 1, 2.0) if tensors == 4 else None
            got = rs.rms_norm(x, w, residual=r, eps=EPS)
            check_norm(got, x, r, w, what, rows=max(1, (1 << 24) // c))
            few = rows // 3  # through the caches: the same bits
            again = rs.rms_norm(x[:few], w, residual=None if r is None else r[:few], eps=EPS)
            assert torch.equal(again.out, got.out[:few])
            for group in (0, 64):
                q = rs.rms_norm(x, w, residual=r, eps=EPS, out_dtype="float8_e4m3", group=group)
                part = rs.rms_norm(x[:few], w, residual=None if r is None else r[:few], eps=EPS,
                                   out_dtype="float8_e4m3", group=group)
                assert torch.equal(q.scales[:few], part.scales)
                assert torch.equal(q.out[:few].view(torch.uint8), part.out.view(torch.uint8))
                last = slice(rows - 20, rows)
                check_quant(q._replace(out=q.out[last], scales=q.scales[last]), x[last],
                            None if r is None else r[last], w, group, what + " into 8 bits")


@pytest.mark.gpu
@pytest.mark.parametrize("rows, cols", [((1 << 20) + 3, 1025), ((1 << 25) + 37, 8)])
def test_norm_in_a_grid_of_two_dimensions(rows, cols):
    """More than 2^20 workgroups, of one row and of 32."""
    say(f"norm {rows}x{cols}")
    x = random((rows, cols), torch.bfloat16, 1)
    w = random(cols, torch.bfloat16, 2, 0.3) + 1.0
    check_norm(rs.rms_norm(x, w, eps=EPS), x, None, w, f"{rows}x{cols}", rows=(1 << 25) // cols)


# ---------------------------------------------------------------------------
# Backward
# ---------------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("cols", LAYOUTS + (5000,))
@pytest.mark.parametrize("name", DTYPES)
def test_backward_beyond_the_cache(name, cols):
    dtype = DTYPES[name]
    widths = (cols,) if dtype != torch.float32 else ((cols + 1) // 2, 32765) if cols == 32765 else ((cols + 1) // 2,)
    for c in widths:
        w = random(c, dtype, 1, 0.3) + 1.0
        for tensors in (3, 4):
            rows = beyond_the_cache(c, dtype.itemsize, tensors)
            what = f"backward {name} {rows}x{c} of {tensors} tensors"
            say(what)
            h, dy = random((rows, c), dtype, c), random((rows, c), dtype, c + 1, 0.1)
            r = random((rows, c), dtype, c + 2, 0.1) if tensors == 4 else None
            got = rs.rms_norm_backward(dy, h, w, grad_residual=r, eps=EPS)
            check_grad_in(got.grad_in, dy, h, w, r, what, rows=max(1, (1 << 24) // c))
            few = rows // 3
            again = rs.rms_norm_backward(dy[:few], h[:few], w, grad_residual=None if r is None else r[:few], eps=EPS)
            assert torch.equal(again.grad_in, got.grad_in[:few])


def whole_root(cols):
    """Columns, from `cols` on, for which cols * (1 / cols) is 1 in fp32."""
    while np.float32(cols) * (np.float32(1) / np.float32(cols)) != np.float32(1):
        cols += 1
    return cols


def count_rows(name, rows, cols):
    """The weight's gradient of rows of 1 and -1, whose root is exactly 1, and
    of whole numbers: every sum is a whole number below 2^24, so that the
    result is exact in any order, and no row can be missing or counted twice."""
    dtype = DTYPES[name]
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    h = (torch.randint(0, 2, (rows, cols), generator=gen, device="cuda") * 2 - 1).to(dtype)
    dy = torch.randint(1, 9, (rows, cols), generator=gen, device="cuda").to(dtype)
    w = torch.ones(cols, device="cuda")
    what = f"backward {name} {rows}x{cols}"
    say(what)
    got = rs.rms_norm_backward(dy, h, w, eps=0.0)
    want = torch.zeros(cols, device="cuda", dtype=torch.float64)
    for lo in range(0, rows, 1 << 16):
        want += (h[lo:lo + (1 << 16)].double() * dy[lo:lo + (1 << 16)].double()).sum(0)
    assert torch.equal(got.grad_weight.double(), want), what
    return got, dy, h, w


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [5, 100, 128, 130, 250, 500, 700, 1000, 2000, 4096, 5000, 8000, 9000, 16000, 30000])
def test_weight_gradient_counts_every_row(cols):
    """Row counts on both sides of the borders below which one workgroup takes
    all rows (three turns of 16, 8, 4 or 1 rows), of the second kernel's two
    forms, and where workgroups take one, two and more turns."""
    cols = whole_root(cols)
    for rows in (1, 2, 3, 4, 5, 11, 12, 13, 23, 24, 25, 47, 48, 49, 50, 63, 64, 65, 255, 257, 513, 1025, 2049, 2500):
        for name in DTYPES:
            got, dy, h, w = count_rows(name, rows, cols)
            if rows in (3, 4, 12, 13, 24, 25, 48, 49):
                dx, _, bound, _ = ref.backward(dy, h, w, None, 0.0)
                inside(got.grad_in, dx, bound + ref.half_step(dx, h.dtype), f"{name} {rows}x{cols} grad_in")


@pytest.mark.gpu
@pytest.mark.parametrize("rows, cols", [(9000, 64), (5000, 130), (20011, 250), (9001, 700), (2777, 2100), (300_007, 100),
                                        (70_001, 509), (30_001, 1500), (9000, 4100), (9000, 5200), (5000, 9000)])
def test_weight_gradient_counts_every_one_of_many_rows(rows, cols):
    for name in DTYPES:
        count_rows(name, rows, whole_root(cols))


def test_rows_of_one_workgroup():
    """The workspace says it: none where one workgroup takes all rows."""
    f = ctypes.CDLL(rs.lib()._name).ringsim_rms_norm_backward_workspace
    f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
    n = ctypes.c_size_t()
    for name, code in CODES.items():
        pack = 4 if name == "f32" else 8
        for packs, most in ((1, 48), (16, 48), (17, 24), (32, 24), (33, 12), (64, 12), (65, 12), (128, 12), (129, 3),
                            (256, 3), (257, 3), (1024, 3), (1025, 3), (4096, 3)):
            for rows, needs in ((most, False), (most + 1, True)):
                assert f(rows, packs * pack, code, n) == 0
                assert (n.value > 0) == needs, (name, packs, rows)
