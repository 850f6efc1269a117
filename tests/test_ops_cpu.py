"""Host-side checks of the step operators (include/ringsim_ops.h) that need no
GPU: every declared function is exported, the binding's structures are the
header's, and the C entry points refuse wrong arguments before they touch a
device."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from ring_all_reduce_allreduce_amd import build

if not (os.path.exists(build.LIB) and os.path.exists(build.BINDING)):
    build.build()
from ring_all_reduce_allreduce_amd import operators as ops  # noqa: E402

OK, BAD = 0, 4
F32, BF16, F16, E4M3 = 2, 3, 16, 17


def _header():
    with open(rs.OPS_HEADER_PATH) as f:
        return f.read()


def _struct(cname):
    """A ctypes structure with the fields the header declares."""
    body = re.search(r"typedef struct \{((?:(?!typedef struct).)*?)\}\s*" + cname + ";", _header(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    types = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t, "float": ctypes.c_float}
    fields = []
    for ctype, star, name, n in re.findall(r"^\s*(?:const\s+)?([a-z_0-9]+)(\*?)\s+([a-z_0-9]+)(?:\[(\d)\])?;", body,
                                           re.M):
        t = ctypes.c_void_p if star else types[ctype]
        fields.append((name, t * int(n) if n else t))
    assert len(fields) == body.count(";"), cname
    return type(cname, (ctypes.Structure,), {"_fields_": fields})


RmsNormArgs = _struct("ringsim_rms_norm_t")
RmsNormBackwardArgs = _struct("ringsim_rms_norm_backward_t")


@pytest.fixture(scope="module")
def L():
    lib = ctypes.CDLL(rs.lib()._name)
    vp, i, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    for name, args in {
        "ringsim_rms_norm": [vp, vp],
        "ringsim_rms_norm_backward": [vp, vp],
        "ringsim_rms_norm_backward_workspace": [i64, i64, i, ctypes.POINTER(sz)],
        "ringsim_grad_norm": [i, vp, vp, vp, f32, vp, vp, sz, vp],
        "ringsim_grad_norm_workspace": [i, vp, vp, ctypes.POINTER(sz)],
        "ringsim_scale_grads": [i, vp, vp, vp, vp, f32, vp, f32, f32, vp],
        "ringsim_clip_grads": [i, vp, vp, vp, vp, f32, f32, f32, vp, vp, sz, vp],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i
    return lib


def test_exports_every_declared_function(L):
    declared = sorted(set(re.findall(r"^ringsim_result_t (ringsim_[a-z_]+)\(", _header(), re.M)))
    assert len(declared) == 7
    out = subprocess.run(["nm", "-D", "--defined-only", rs.LIB_PATH], check=True, capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(declared) <= exported
    for f in ("rms_norm", "rms_norm_backward", "grad_norm", "scale_grads", "clip_grads"):
        assert getattr(rs, f) is getattr(ops, f)
    consts = dict(re.findall(r"(RINGSIM_FLOAT16|RINGSIM_FLOAT8_E4M3|RINGSIM_NORM_MAX_COLS)\s*=?\s*(\d+)", _header()))
    assert (int(consts["RINGSIM_FLOAT16"]), int(consts["RINGSIM_FLOAT8_E4M3"])) == (F16, E4M3)
    assert int(consts["RINGSIM_NORM_MAX_COLS"]) == ops.NORM_MAX_COLS
    with pytest.raises(AttributeError):
        rs.no_such_operator


P = 1 << 20  # an address that is never read: the call is refused first


def _norm(**over):
    a = RmsNormArgs()
    v = dict(x=P, out=P, x_stride=(64, 0), out_stride=(64, 0), residual_stride=(64, 0), residual_out_stride=(64, 0),
             outer=4, inner=1, cols=64, dtype=BF16, weight_dtype=BF16, out_dtype=BF16, eps=1e-5)
    v.update(over)
    for k, x in v.items():
        setattr(a, k, type(getattr(a, k))(*x) if isinstance(x, tuple) else x)
    return ctypes.byref(a)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(out=None), dict(x=P + 1), dict(out=P + 1), dict(weight=P + 1), dict(weight=P + 2, weight_dtype=F32),
    dict(dtype=0), dict(dtype=1), dict(dtype=E4M3), dict(dtype=99), dict(out_dtype=F32), dict(out_dtype=F16),
    dict(weight_dtype=F16), dict(weight_dtype=E4M3), dict(cols=0), dict(cols=-1), dict(cols=32769, out_stride=(32769, 0)),
    dict(outer=-1), dict(inner=-1), dict(outer=1 << 31), dict(outer=1 << 40, inner=1 << 40),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(residual=P), dict(residual_out=P), dict(residual=P + 1, residual_out=P), dict(residual=P, residual_out=P + 1),
    dict(scales=P), dict(group=32), dict(out_dtype=E4M3), dict(out_dtype=E4M3, scales=P + 2),
    dict(out_dtype=E4M3, scales=P, group=16), dict(out_dtype=E4M3, scales=P, group=256),
    dict(out_stride=(63, 0)), dict(out_stride=(0, 0)), dict(inner=2, out_stride=(64, 64)),
    dict(inner=2, out_stride=(128, 63)), dict(inner=2, out_stride=(100, 64)), dict(inner=2, out_stride=(64, 100)),
    dict(x_stride=(1 << 62, 0)), dict(out_stride=(-(1 << 62), 0)),
    dict(residual=P, residual_out=P, residual_out_stride=(10, 0)),
], ids=str)
def test_norm_refuses(L, over):
    assert L.ringsim_rms_norm(_norm(**over), None) == BAD


def test_norm_without_rows_or_arguments(L):
    assert L.ringsim_rms_norm(None, None) == BAD
    assert L.ringsim_rms_norm(_norm(outer=0, x=None, out=None), None) == OK
    assert L.ringsim_rms_norm(_norm(inner=0, x=None, out=None), None) == OK


def _backward(**over):
    a = RmsNormBackwardArgs()
    v = dict(grad_out=P, h=P, grad_in=P, weight=P, grad_weight=P, workspace=P, workspace_bytes=1 << 30,
             grad_out_stride=(64, 0), h_stride=(64, 0), grad_residual_stride=(64, 0), grad_in_stride=(64, 0),
             outer=400, inner=1, cols=64, dtype=F32, weight_dtype=F32, eps=1e-5)
    v.update(over)
    for k, x in v.items():
        setattr(a, k, type(getattr(a, k))(*x) if isinstance(x, tuple) else x)
    return ctypes.byref(a)


@pytest.mark.parametrize("over", [
    dict(grad_out=None), dict(h=None), dict(grad_in=None), dict(grad_out=P + 2), dict(h=P + 1), dict(grad_in=P + 2),
    dict(grad_residual=P + 2), dict(weight=P + 2), dict(grad_weight=P + 2), dict(workspace=None),
    dict(workspace=P + 8), dict(workspace_bytes=0), dict(workspace_bytes=64 * 4 - 1), dict(dtype=0), dict(dtype=E4M3),
    dict(weight_dtype=BF16), dict(cols=0), dict(cols=32769, grad_in_stride=(32769, 0)), dict(eps=-1.0),
    dict(eps=float("nan")), dict(grad_in_stride=(63, 0)), dict(outer=1 << 31), dict(h_stride=(1 << 62, 0)),
], ids=str)
def test_backward_refuses(L, over):
    assert L.ringsim_rms_norm_backward(_backward(**over), None) == BAD


def test_backward_workspace(L):
    n = ctypes.c_size_t(0)
    for dtype in (F32, BF16, F16):
        for rows, cols in ((0, 1), (1, 1), (1, 32768), (777, 1111), (1 << 20, 4096), ((1 << 31) - 1, 64)):
            assert L.ringsim_rms_norm_backward_workspace(rows, cols, dtype, n) == OK
            # one workgroup (few rows) needs none
            assert n.value <= 4 * cols * 2048 and n.value % (4 * cols) == 0 and (n.value > 0) == (rows > 64)
    for rows, cols, dtype in ((-1, 64, F32), (4, 0, F32), (4, 32769, F32), (1 << 31, 64, F32), (4, 64, 0), (4, 64, E4M3)):
        assert L.ringsim_rms_norm_backward_workspace(rows, cols, dtype, n) == BAD
    assert L.ringsim_rms_norm_backward_workspace(4, 4, F32, None) == BAD


def _list_args(ptrs, counts, types):
    n = len(ptrs)
    return (n, (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*counts), (ctypes.c_int * n)(*types))


@pytest.mark.parametrize("ptrs, counts, types", [
    ([None], [1], [F32]), ([P + 2], [1], [F32]), ([P + 1], [1], [BF16]), ([P], [-1], [F32]), ([P], [1], [0]),
    ([P], [1], [E4M3]), ([P], [1 << 60], [F32]), ([P], [1 << 50], [BF16]), ([P, None], [1, 5], [F32, F32]),
    ([P] * 4, [1 << 43] * 4, [F32] * 4), ([1 << 48], [1], [F32]), ([P, 1 << 63], [9, 9], [BF16, F32]),
], ids=str)
def test_gradient_lists_refused(L, ptrs, counts, types):
    n, p, c, t = _list_args(ptrs, counts, types)
    big = 1 << 30
    assert L.ringsim_grad_norm(n, p, c, t, 1.0, P, P, big, None) == BAD
    assert L.ringsim_scale_grads(n, p, None, c, t, 1.0, P, 1.0, 0.0, None) == BAD
    assert L.ringsim_clip_grads(n, p, None, c, t, 1.0, 1.0, 0.0, P, P, big, None) == BAD


def test_gradient_calls_refused(L):
    n, p, c, t = _list_args([P], [1 << 20], [F32])
    nan, inf, big = float("nan"), float("inf"), 1 << 30
    need = ctypes.c_size_t(0)
    assert L.ringsim_grad_norm_workspace(1, c, t, need) == OK and need.value > 0
    for args in ((-1, c, t, need), (1, None, t, need), (1, c, None, need), (1, c, t, None),
                 (1, (ctypes.c_int64 * 1)(-1), t, need), (1, c, (ctypes.c_int * 1)(0), need)):
        assert L.ringsim_grad_norm_workspace(*args) == BAD
    few = ctypes.c_size_t(1)
    assert L.ringsim_grad_norm_workspace(0, None, None, few) == OK and few.value == 0
    assert L.ringsim_grad_norm_workspace(1, (ctypes.c_int64 * 1)(12 * 4096), t, few) == OK and few.value == 0
    for args in ((-1, p, c, t, 1.0, P, P, big), (1, None, c, t, 1.0, P, P, big), (1, p, None, t, 1.0, P, P, big),
                 (1, p, c, None, 1.0, P, P, big), (1, p, c, t, nan, P, P, big), (1, p, c, t, inf, P, P, big),
                 (1, p, c, t, 1.0, None, P, big), (1, p, c, t, 1.0, P + 2, P, big), (1, p, c, t, 1.0, P, None, big),
                 (1, p, c, t, 1.0, P, P + 8, big), (1, p, c, t, 1.0, P, P, need.value - 1)):
        assert L.ringsim_grad_norm(*args, None) == BAD, args
    bad_out = (ctypes.c_void_p * 1)(None)
    odd_out = (ctypes.c_void_p * 1)(P + 2)
    for outs, scale, norm, top, eps in ((bad_out, 1.0, P, 1.0, 0.0), (odd_out, 1.0, P, 1.0, 0.0),
                                        (None, nan, P, 1.0, 0.0), (None, 1.0, None, 1.0, 0.0),
                                        (None, 1.0, P + 1, 1.0, 0.0), (None, 1.0, P, -1.0, 0.0),
                                        (None, 1.0, P, inf, 0.0), (None, 1.0, P, nan, 0.0),
                                        (None, 1.0, P, 1.0, -1.0), (None, 1.0, P, 1.0, inf)):
        assert L.ringsim_scale_grads(1, p, outs, c, t, scale, norm, top, eps, None) == BAD
        assert L.ringsim_clip_grads(1, p, outs, c, t, scale, top, eps, norm, P, big, None) == BAD
    for ws, nbytes in ((None, big), (P + 8, big), (P, need.value - 1)):
        assert L.ringsim_clip_grads(1, p, None, c, t, 1.0, 1.0, 0.0, P, ws, nbytes, None) == BAD
    # nothing to scale
    assert L.ringsim_scale_grads(0, None, None, None, None, 1.0, P, 1.0, 0.0, None) == OK
    n, p, c, t = _list_args([None], [0], [F32])
    assert L.ringsim_scale_grads(1, p, None, c, t, 1.0, P, 1.0, 0.0, None) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    for call in (lambda: rs.rms_norm(x.to(torch.float64)), lambda: rs.rms_norm(x, torch.zeros(8, dtype=torch.bfloat16)),
                 lambda: rs.rms_norm(x, out_dtype=torch.float16), lambda: rs.rms_norm(x, out_dtype="float8_e5m2"),
                 lambda: rs.rms_norm_backward(x, x.to(torch.int32)), lambda: rs.grad_norm([x.to(torch.float64)]),
                 lambda: rs.rms_norm(1), lambda: rs.rms_norm(x, eps="a"), lambda: rs.rms_norm(x, 5)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: rs.rms_norm(x, torch.zeros(7)), lambda: rs.rms_norm(x, torch.zeros(1, 8)),
                 lambda: rs.rms_norm(x, torch.zeros(16)[::2]), lambda: rs.rms_norm(torch.zeros(())),
                 lambda: rs.rms_norm(x, group=32), lambda: rs.rms_norm(x, out_dtype="float8_e4m3", group=16),
                 lambda: rs.rms_norm(x), lambda: rs.grad_norm([x]), lambda: rs.clip_grads([x], 1.0),  # host tensors
                 lambda: rs.rms_norm_backward(x, x)):
        with pytest.raises(ValueError):
            call()
